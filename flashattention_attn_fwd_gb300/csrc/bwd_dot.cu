// D_i = sum_j P_ij dP_ij of the windowed backward with sinks, from the scores.
//
// dS = P (dP - D) cancels where a row's weight sits on one key: dP of that key
// and D are then nearly equal.  D is otherwise taken as dO . O with the output
// that the forward returned, whose bf16 rounding (2^-9 of |O|, and that of P
// before it) then is the error of the difference; rows of a few keys, which
// have little else to attend to, bring that out (score_rows in bwd.h has the
// figures and the rule).  So this kernel forms S = Q K^T and dP = dO V^T once
// more over the visible keys and sums P dP in 32 bits: P = 2^(t log2 e - L2) needs
// no running maximum, as the log-sum-exp is known.
//
// One CTA takes 64 query rows of one head, 16 per warp; keys come in tiles of 64
// through a two-stage cp.async ring; both products are warp-level m16n8k16
// tiles whose accumulators stay in registers.  Larger blocks read K and V less
// often but leave fewer of them to hide each other's waits: 128 rows in 8 warps
// and 32 rows per warp were 15 and 20 us slower at B 4 H 16 L 2048 d 64, and for
// the first rows alone 16 rows a block with the keys split over its warps: 3 us
// there, for 0.7 us less at one sequence of 600 tokens.  No
// accumulator outlives a tile, so there is nothing for TMEM to hold; bound by
// the tensor core's warp-level rate and by the exponentials.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <algorithm>
#include <cstdint>

#include "bwd.h"
#include "host.h"
#include "ptx.cuh"

namespace fl {
namespace {

constexpr int kDotKeys = 64, kDotThreads = 128;
constexpr float kDotLog2e = 1.4426950408889634f;

template <int D, int DV, int SCORE>
__global__ void __launch_bounds__(kDotThreads) attn_bwd_dot_kernel(const __grid_constant__ BwdParams p) {
  constexpr int STAGE = kDotKeys * (D + DV) * 2;
  extern __shared__ __align__(128) uint8_t dot_sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  ptx::launch_dependents();  // the other rows' kernel shares nothing with this one
  const int n_rt = (min(p.dot_rows, p.Lq) + kDotRows - 1) / kDotRows;
  const int rt = blockIdx.x % n_rt;
  const int bh = blockIdx.x / n_rt;  // (batch, query head)
  const int h = bh % p.Hq, b = bh / p.Hq;
  const int hkv = h / (p.Hq / p.Hkv);
  const int r0 = rt * kDotRows;
  const int64_t row0 = static_cast<int64_t>(bh) * p.Lq;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row0 * D;
  const __nv_bfloat16* dout = static_cast<const __nv_bfloat16*>(p.dout) + row0 * DV;
  const int64_t krow0 = (static_cast<int64_t>(b) * p.Hkv + hkv) * p.Lk;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + krow0 * D;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + krow0 * DV;

  // the rows' dQ accumulator starts at zero
  {
    const int n = min(kDotRows, p.Lq - r0) * (D / 4);
    float4* acc = reinterpret_cast<float4*>(p.dq_acc + (row0 + r0) * D);
    for (int i = tid; i < n; i += kDotThreads) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }

  // key tiles: the window's [w0, w1], then the sinks' left of it [0, ns)
  const int r1 = min(r0 + kDotRows, p.Lq) - 1;
  const int win = min(p.window, p.Lq);
  const int w0 = max(r0 - win + 1, 0) / kDotKeys, w1 = r1 / kDotKeys;
  const int ns = (min(p.sink, max(r1 - win + 1, 0)) + kDotKeys - 1) / kDotKeys;
  const int nw = w1 - w0 + 1, n_tiles = nw + ns;
  const uint32_t sm = ptx::smem_u32(dot_sm);
  auto load = [&](int i) {
    const int j0 = (i < nw ? w0 + i : i - nw) * kDotKeys;
    const uint32_t st = sm + (i & 1) * STAGE;
    for (int c = tid; c < kDotKeys * (D / 8); c += kDotThreads) {
      const int r = c / (D / 8), cc = c % (D / 8);
      const bool ok = j0 + r < p.Lk;
      ptx::cp_async16(st + chunk_at<D>(r, cc), k + static_cast<int64_t>(ok ? j0 + r : 0) * D + cc * 8, ok);
    }
    for (int c = tid; c < kDotKeys * (DV / 8); c += kDotThreads) {
      const int r = c / (DV / 8), cc = c % (DV / 8);
      const bool ok = j0 + r < p.Lk;
      ptx::cp_async16(st + kDotKeys * D * 2 + chunk_at<DV>(r, cc), v + static_cast<int64_t>(ok ? j0 + r : 0) * DV + cc * 8, ok);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  load(0);

  // this warp's 16 rows of Q and dO as A fragments (rows past the end: zero)
  uint32_t qa[D / 16][4], da[DV / 16][4];
  int row[2];
  float l2[2], slope2 = 0.f;
  bool live[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    row[e] = r0 + warp * 16 + g + 8 * e;
    live[e] = row[e] < p.Lq;
    const int64_t rr = live[e] ? row[e] : 0;
    const uint32_t* qr = reinterpret_cast<const uint32_t*>(q + rr * D);
    const uint32_t* dr = reinterpret_cast<const uint32_t*>(dout + rr * DV);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qa[kk][e] = live[e] ? __ldg(qr + 8 * kk + t4) : 0u;
      qa[kk][2 + e] = live[e] ? __ldg(qr + 8 * kk + 4 + t4) : 0u;
    }
#pragma unroll
    for (int kk = 0; kk < DV / 16; ++kk) {
      da[kk][e] = live[e] ? __ldg(dr + 8 * kk + t4) : 0u;
      da[kk][2 + e] = live[e] ? __ldg(dr + 8 * kk + 4 + t4) : 0u;
    }
    const float l = live[e] ? __ldg(p.lse + row0 + row[e]) : 0.f;
    l2[e] = l == -CUDART_INF_F ? CUDART_INF_F : l * kDotLog2e;
  }
  const float sc = p.scale * kDotLog2e;
  if (SCORE == 1) slope2 = __ldg(p.slopes + h) * kDotLog2e;

  // P = 2^(t log2 e - L2) of a raw score x, key j, row[w]
  float sum[2] = {0.f, 0.f};
  auto weight = [&](float x, int j, int w) {
    if (SCORE == 1) return ptx::ex2(fmaf(x, sc, fmaf(slope2, static_cast<float>(j - row[w]), -l2[w])));
    if (SCORE == 2) return ptx::ex2(x - l2[w]);  // x is t already
    return ptx::ex2(fmaf(x, sc, -l2[w]));
  };
  for (int i = 0; i < n_tiles; ++i) {
    if (i + 1 < n_tiles) {
      load(i + 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const uint32_t ks = sm + (i & 1) * STAGE, vs = ks + kDotKeys * D * 2;
    const int j0 = (i < nw ? w0 + i : i - nw) * kDotKeys;
    // the interval that each of this lane's two rows sees in this tile, and the
    // warp's 16 rows' smallest and largest ends
    const bool win_tile = i < nw;
    int lo[2], hi[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int first = max(row[e] - win + 1, 0);
      lo[e] = win_tile ? first : 0;
      hi[e] = !live[e] ? -1 : win_tile ? row[e] : min(p.sink, first) - 1;
    }
    const int ra = r0 + warp * 16, rz = min(ra + 15, p.Lq - 1);
    const int fa = max(ra - win + 1, 0), fz = max(rz - win + 1, 0);
    const int lo_min = win_tile ? fa : 0, lo_max = win_tile ? fz : 0;
    const int hi_min = ra + 15 >= p.Lq ? -1 : win_tile ? ra : min(p.sink, fa) - 1;
    const int hi_max = win_tile ? rz : min(p.sink, fz) - 1;
#pragma unroll 1
    for (int n2 = 0; n2 < kDotKeys / 16; ++n2) {
      // blocks that none of the warp's rows sees (a third of them at a window of
      // 256 and few sinks)
      const int jb = j0 + n2 * 16;
      if (jb > hi_max || jb + 15 < lo_min) continue;
      // 16 keys: matrices (keys 0-7 | 8-15) x (channels 0-7 | 8-15) of a k-step
      const int lr = n2 * 16 + ((lane >> 4) << 3) + (lane & 7), lc = (lane >> 3) & 1;
      float s[2][4] = {}, dp[2][4] = {}, none[1][4];
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t r[4];
        ptx::ldsm4(r, ks + chunk_at<D>(lr, 2 * kk + lc));
        ptx::mma16816(s[0], qa[kk], r[0], r[1]);
        ptx::mma16816(s[1], qa[kk], r[2], r[3]);
      }
#pragma unroll
      for (int kk = 0; kk < DV / 16; ++kk) {
        uint32_t r[4];
        ptx::ldsm4(r, vs + chunk_at<DV>(lr, 2 * kk + lc));
        ptx::mma16816(dp[0], da[kk], r[0], r[1]);
        ptx::mma16816(dp[1], da[kk], r[2], r[3]);
      }
      if constexpr (SCORE == 2) softcap_log2<2, false>(p, s, none);
      if (jb >= lo_max && jb + 15 <= hi_min) {  // all of the warp's rows see all of it
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sum[e >> 1] = fmaf(weight(s[n][e], jb + n * 8 + 2 * t4 + (e & 1), e >> 1), dp[n][e], sum[e >> 1]);
      } else {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = jb + n * 8 + 2 * t4 + (e & 1), w = e >> 1;
            const float pv = j >= lo[w] && j <= hi[w] ? weight(s[n][e], j, w) : 0.f;
            sum[w] = fmaf(pv, dp[n][e], sum[w]);
          }
      }
    }
    __syncthreads();  // the stage may be refilled
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
    if (t4 == 0 && live[e]) {
      const int64_t at = static_cast<int64_t>(bh) * p.Lq_pad + row[e];
      p.dvec[at] = sum[e] * p.dout_scale;
      p.l2[at] = l2[e];
    }
  }
}

template <int D, int DV, int SCORE>
cudaError_t launch_dot_ds(const BwdParams& p, cudaStream_t s) {
  constexpr int smem = 2 * kDotKeys * (D + DV) * 2;
  static OncePerDevice once;
  const cudaError_t attr = on_this_device(once, [] {
    return cudaFuncSetAttribute(attn_bwd_dot_kernel<D, DV, SCORE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (attr != cudaSuccess) return attr;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.Hq * ((std::min(p.dot_rows, p.Lq) + kDotRows - 1) / kDotRows));
  attn_bwd_dot_kernel<D, DV, SCORE><<<grid, kDotThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int D, int DV>
cudaError_t launch_dot_d(int score_mod, const BwdParams& p, cudaStream_t s) {
  return score_mod == 0 ? launch_dot_ds<D, DV, 0>(p, s)
         : score_mod == 1 ? launch_dot_ds<D, DV, 1>(p, s)
                          : launch_dot_ds<D, DV, 2>(p, s);
}

}  // namespace

cudaError_t launch_bwd_dot(int d, int dv, int score_mod, const BwdParams& p, cudaStream_t s) {
  if (dv != d) return launch_dot_d<64, 128>(score_mod, p, s);
  switch (d) {
    case 32: return launch_dot_d<32, 32>(score_mod, p, s);
    case 64: return launch_dot_d<64, 64>(score_mod, p, s);
    default: return launch_dot_d<128, 128>(score_mod, p, s);
  }
}

}  // namespace fl
