// Backward of the window with sinks for sequences of at most 64 tokens: all of
// dQ, dK, dV in one launch.
//
//   P = 2^(t log2 e - L2),  dP = dO V^T,  D = sum_j P dP,  dS = P (dP - D) dT/dS
//   dQ = dS K,  dK = dS^T Q,  dV = P^T dO
//
// The tiled backward makes four launches of it (D, the walks, dQ to bf16) that
// each wait for the last, and rounds P and dS to bf16 between the products,
// which few rows do not average out (2.4e-3 to 2.7e-3 from the 64-bit gradients,
// where rounding the results alone gives 1.7e-3).  Here one block takes a (batch,
// key/value head) and its query heads in turn, 16 rows a warp.  S and dP stay in
// registers from their products to dS, and D comes from them.  P and dS go into
// the second products as a sum of two bf16 parts (a high one and the rest, 2^-17
// of the value), two tensor-core products each, so that the results are the
// definition's but for their own rounding.  dV and dK of a warp's 16 keys stay in
// registers over the heads: no atomics, one order of sums.
//
// Warp-level m16n8k16 tiles: 64 rows are less than half of a tcgen05 tile, and a
// block's few products are over before its accumulators would have been read
// back.  Where blocks are few a cluster shares the query heads of a group and
// joins its dV and dK through distributed shared memory, in rank order.  Bound by
// latency, a dozen dependent phases a head.  Measured, the tiled backward's time
// second: B 1, H 2, L 64, d 64: 7 us, 12; B 2, 16 heads over 4, L 64, d 128: 15
// and 25 (34 without the cluster); B 64, H 16, L 64, d 64: 28 and 58; B 256, H 16,
// L 64, d 128: 183 and 343.  The call issues in 9 us against 14.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <cstdint>
#include <type_traits>

#include "bwd.h"
#include "host.h"
#include "ptx.cuh"

namespace fl {
namespace {

constexpr int kRows = kShortRows, kShortThreads = 128;
constexpr float kShortLog2e = 1.4426950408889634f;

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// x, y as bf16 pairs: the nearest, and what is left of each
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = ptx::pack_bf16x2(x, y);
  lo = ptx::pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

template <int D, int DV>
struct ShortLayout {
  static constexpr int K = 0, V = K + kRows * D * 2, Q = V + kRows * DV * 2, DO = Q + kRows * D * 2;
  static constexpr int PART = kRows * kRows * 2;  // one bf16 part of P or dS, [row][key]
  static constexpr int P = DO + kRows * DV * 2, DS = P + 2 * PART, BYTES = DS + 2 * PART;
  static constexpr int W = D + DV + 4;           // floats a key of a cluster's partial dV, dK
  static_assert(kRows * W * 4 <= BYTES, "partial sums over the tiles");
};

// cl: CTAs of a cluster that share a (batch, key/value head)
template <int D, int DV, int SCORE>
__global__ void __launch_bounds__(kShortThreads) attn_bwd_short_kernel(const __grid_constant__ BwdParams p, int cl) {
  using L = ShortLayout<D, DV>;
  extern __shared__ __align__(128) uint8_t short_sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int n = p.Lq;                       // rows, and keys
  const int nb = (n + 15) / 16;             // blocks of 16 of them
  const int unit = blockIdx.x / cl, rank = blockIdx.x % cl;
  const int heads = p.Hq / p.Hkv / cl;      // query heads of this block
  const int hkv = unit % p.Hkv, b = unit / p.Hkv;
  const int h0 = hkv * (p.Hq / p.Hkv) + rank * heads;
  const int64_t krow0 = (static_cast<int64_t>(b) * p.Hkv + hkv) * n;
  const uint32_t sm = ptx::smem_u32(short_sm);
  // rows [0, 16 nb) of a [n][C] matrix into a tile, zeros behind row n
  auto load = [&](auto width, uint32_t dst, const void* base, int64_t row0) {
    constexpr int C = decltype(width)::value;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(base) + row0 * C;
    for (int c = tid; c < nb * 16 * (C / 8); c += kShortThreads) {
      const int r = c / (C / 8), cc = c % (C / 8);
      const bool ok = r < n;
      ptx::cp_async16(sm + dst + chunk_at<C>(r, cc), src + static_cast<int64_t>(ok ? r : 0) * C + cc * 8, ok);
    }
  };
  load(std::integral_constant<int, D>{}, L::K, p.k, krow0);
  load(std::integral_constant<int, DV>{}, L::V, p.v, krow0);
  const float sc = p.scale * kShortLog2e;

  float dk[D / 8][4], dv[DV / 8][4];        // of this warp's 16 keys
#pragma unroll
  for (int c = 0; c < D / 8; ++c) dk[c][0] = dk[c][1] = dk[c][2] = dk[c][3] = 0.f;
#pragma unroll
  for (int c = 0; c < DV / 8; ++c) dv[c][0] = dv[c][1] = dv[c][2] = dv[c][3] = 0.f;

  for (int h = h0; h < h0 + heads; ++h) {
    const int64_t row0 = (static_cast<int64_t>(b) * p.Hq + h) * n;
    load(std::integral_constant<int, D>{}, L::Q, p.q, row0);
    load(std::integral_constant<int, DV>{}, L::DO, p.dout, row0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    int row[2];
    float l2[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      row[e] = warp * 16 + g + 8 * e;
      l2[e] = row[e] < n ? __ldg(p.lse + row0 + row[e]) * kShortLog2e : 0.f;
    }
    const float slope2 = SCORE == 1 ? __ldg(p.slopes + h) * kShortLog2e : 0.f;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    if (warp < nb) {
      // ---- S = Q K^T and dP = dO V^T of this warp's rows, in blocks of 8 keys
      float s[kRows / 8][4], dp[kRows / 8][4];
#pragma unroll
      for (int c = 0; c < kRows / 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[c][e] = dp[c][e] = 0.f;
      const int ar = warp * 16 + (lane & 15), ac = lane >> 4;
      const int br = ((lane >> 4) << 3) + (lane & 7), bc = (lane >> 3) & 1;
      auto product = [&](auto width, float (&acc)[kRows / 8][4], uint32_t a_tile, uint32_t b_tile) {
        constexpr int C = decltype(width)::value;
#pragma unroll
        for (int kk = 0; kk < C / 16; ++kk) {
          uint32_t a[4];
          ptx::ldsm4(a, sm + a_tile + chunk_at<C>(ar, 2 * kk + ac));
#pragma unroll
          for (int n2 = 0; n2 < kRows / 16; ++n2) {
            if (n2 >= nb) break;
            uint32_t r[4];
            ptx::ldsm4(r, sm + b_tile + chunk_at<C>(n2 * 16 + br, 2 * kk + bc));
            ptx::mma16816(acc[2 * n2], a, r[0], r[1]);
            ptx::mma16816(acc[2 * n2 + 1], a, r[2], r[3]);
          }
        }
      };
      product(std::integral_constant<int, D>{}, s, L::Q, L::K);
      product(std::integral_constant<int, DV>{}, dp, L::DO, L::V);
      // ---- P, D and dS (row 0 sees one key: its softmax has no gradient)
      float dsum[2] = {0.f, 0.f};
      float sech[SCORE == 2 ? kRows / 8 : 1][4];
      if constexpr (SCORE == 2) softcap_log2<kRows / 8, true>(p, s, sech);
#pragma unroll
      for (int c = 0; c < kRows / 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int w = e >> 1, i = row[w], j = 8 * c + 2 * t4 + (e & 1);
          const bool sees = i < n && j <= i && (j > i - p.window || j < p.sink);
          float t;
          if constexpr (SCORE == 2) {
            t = s[c][e] - l2[w];  // capped already
          } else if constexpr (SCORE == 1) {
            t = fmaf(s[c][e], sc, fmaf(slope2, static_cast<float>(j - i), -l2[w]));
          } else {
            t = fmaf(s[c][e], sc, -l2[w]);
          }
          s[c][e] = sees ? ptx::ex2(t) : 0.f;
          dsum[w] = fmaf(s[c][e], dp[c][e], dsum[w]);
        }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        dsum[w] += __shfl_xor_sync(0xffffffffu, dsum[w], 1);
        dsum[w] += __shfl_xor_sync(0xffffffffu, dsum[w], 2);
      }
#pragma unroll
      for (int c = 0; c < kRows / 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[c][e] * (dp[c][e] - dsum[e >> 1]);
          if constexpr (SCORE == 2) x *= sech[c][e];
          dp[c][e] = row[e >> 1] == 0 ? 0.f : x;
        }
      // ---- both, in two bf16 parts, to shared memory for the keys' products;
      // dS stays as the A operand of dQ too
      uint32_t dsa[2][kRows / 8][2];
#pragma unroll
      for (int c = 0; c < kRows / 8; ++c) {
        if (c >= 2 * nb) break;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t at = chunk_at<kRows>(row[w], c) + 4 * t4;
          uint32_t hi, lo;
          split2(s[c][2 * w], s[c][2 * w + 1], hi, lo);
          sts32(sm + L::P + at, hi);
          sts32(sm + L::P + L::PART + at, lo);
          split2(dp[c][2 * w], dp[c][2 * w + 1], dsa[0][c][w], dsa[1][c][w]);
          sts32(sm + L::DS + at, dsa[0][c][w]);
          sts32(sm + L::DS + L::PART + at, dsa[1][c][w]);
        }
      }
      // ---- dQ = scale dS K, 16 channels at a time
      __nv_bfloat16* dq = static_cast<__nv_bfloat16*>(p.dq) + row0 * D;
#pragma unroll
      for (int cc = 0; cc < D / 16; ++cc) {
        float acc[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < kRows / 16; ++kk) {
          if (kk >= nb) break;
          uint32_t r[4];
          ptx::ldsm4t(r, sm + L::K + chunk_at<D>(kk * 16 + (lane & 15), 2 * cc + (lane >> 4)));
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const uint32_t a[4] = {dsa[part][2 * kk][0], dsa[part][2 * kk][1], dsa[part][2 * kk + 1][0], dsa[part][2 * kk + 1][1]};
            ptx::mma16816(acc[0], a, r[0], r[1]);
            ptx::mma16816(acc[1], a, r[2], r[3]);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int w = 0; w < 2; ++w)
            if (row[w] < n)
              *reinterpret_cast<uint32_t*>(dq + static_cast<int64_t>(row[w]) * D + 16 * cc + 8 * x + 2 * t4) =
                  ptx::pack_bf16x2(acc[x][2 * w] * p.scale, acc[x][2 * w + 1] * p.scale);
      }
    }
    __syncthreads();  // P and dS of all rows
    if (warp < nb) {
      // ---- dV += P^T dO and dK += dS^T Q of this warp's keys
      auto keys = [&](auto width, auto& acc, uint32_t a_parts, uint32_t b_tile) {
        constexpr int C = decltype(width)::value;
        const int tr = (lane & 7) + ((lane >> 4) << 3), tc = 2 * warp + ((lane >> 3) & 1);
#pragma unroll
        for (int kk = 0; kk < kRows / 16; ++kk) {
          if (kk >= nb) break;
          uint32_t a[2][4];
          ptx::ldsm4t(a[0], sm + a_parts + chunk_at<kRows>(kk * 16 + tr, tc));
          ptx::ldsm4t(a[1], sm + a_parts + L::PART + chunk_at<kRows>(kk * 16 + tr, tc));
#pragma unroll
          for (int cc = 0; cc < C / 16; ++cc) {
            uint32_t r[4];
            ptx::ldsm4t(r, sm + b_tile + chunk_at<C>(kk * 16 + (lane & 15), 2 * cc + (lane >> 4)));
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              ptx::mma16816(acc[2 * cc], a[part], r[0], r[1]);
              ptx::mma16816(acc[2 * cc + 1], a[part], r[2], r[3]);
            }
          }
        }
      };
      keys(std::integral_constant<int, DV>{}, dv, L::P, L::DO);
      keys(std::integral_constant<int, D>{}, dk, L::DS, L::Q);
    }
    __syncthreads();  // the next head's tiles may come
  }
  if (cl > 1) {
    // the tiles' memory takes dV and dK, fp32 [key][DV + D], for the cluster; each
    // of its blocks sums the keys j with j % cl == rank
    constexpr int W = L::W;
    float* mine = reinterpret_cast<float*>(short_sm);
    auto leave = [&](auto width, const auto& acc, int col) {
#pragma unroll
      for (int c = 0; c < decltype(width)::value / 8; ++c)
#pragma unroll
        for (int w = 0; w < 2; ++w)
          *reinterpret_cast<float2*>(mine + (warp * 16 + g + 8 * w) * W + col + 8 * c + 2 * t4) =
              make_float2(acc[c][2 * w], acc[c][2 * w + 1]);
    };
    leave(std::integral_constant<int, DV>{}, dv, 0);
    leave(std::integral_constant<int, D>{}, dk, DV);
    ptx::cluster_barrier();
    constexpr int CP = (D + DV) / 2;
    for (int e = tid; e < (n - rank + cl - 1) / cl * CP; e += kShortThreads) {
      const int j = rank + cl * (e / CP), c = 2 * (e % CP);
      float2 x = make_float2(0.f, 0.f);
      for (int r = 0; r < cl; ++r) {
        x.x += ptx::ld_cluster(sm + (j * W + c) * 4, r);
        x.y += ptx::ld_cluster(sm + (j * W + c) * 4 + 4, r);
      }
      __nv_bfloat16* out = c < DV ? static_cast<__nv_bfloat16*>(p.dv) + (krow0 + j) * DV + c
                                  : static_cast<__nv_bfloat16*>(p.dk) + (krow0 + j) * D + c - DV;
      const float f = c < DV ? 1.0f : p.scale;
      *reinterpret_cast<uint32_t*>(out) = ptx::pack_bf16x2(x.x * f, x.y * f);
    }
    ptx::cluster_barrier();  // no block leaves while another reads its part
    return;
  }
  auto store = [&](auto width, const auto& acc, void* base, float f) {
    constexpr int C = decltype(width)::value;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(base) + krow0 * C;
#pragma unroll
    for (int c = 0; c < C / 8; ++c)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int j = warp * 16 + g + 8 * w;
        if (j < n)
          *reinterpret_cast<uint32_t*>(out + static_cast<int64_t>(j) * C + 8 * c + 2 * t4) =
              ptx::pack_bf16x2(acc[c][2 * w] * f, acc[c][2 * w + 1] * f);
      }
  };
  store(std::integral_constant<int, DV>{}, dv, p.dv, 1.0f);
  store(std::integral_constant<int, D>{}, dk, p.dk, p.scale);
}

template <int D, int DV, int SCORE>
cudaError_t launch_short_ds(const BwdParams& p, int sm_count, cudaStream_t s) {
  constexpr int smem = ShortLayout<D, DV>::BYTES;
  static OncePerDevice once;
  const cudaError_t attr = on_this_device(once, [] {
    return cudaFuncSetAttribute(attn_bwd_short_kernel<D, DV, SCORE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (attr != cudaSuccess) return attr;
  // a cluster per (batch, key/value head) while all of its blocks find a place,
  // two an SM: a power of two that divides the group, up to the portable 8
  const int64_t units = static_cast<int64_t>(p.B) * p.Hkv;
  const int group = p.Hq / p.Hkv;
  int cl = 1;
  while (cl < 8 && group % (2 * cl) == 0 && units * cl <= sm_count) cl *= 2;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  cfg.gridDim = dim3(static_cast<unsigned>(units * cl));
  cfg.blockDim = dim3(kShortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(cl);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  return cudaLaunchKernelEx(&cfg, attn_bwd_short_kernel<D, DV, SCORE>, p, cl);
}

template <int D, int DV>
cudaError_t launch_short_d(int score_mod, const BwdParams& p, int sm_count, cudaStream_t s) {
  return score_mod == 0 ? launch_short_ds<D, DV, 0>(p, sm_count, s)
         : score_mod == 1 ? launch_short_ds<D, DV, 1>(p, sm_count, s)
                          : launch_short_ds<D, DV, 2>(p, sm_count, s);
}

}  // namespace

cudaError_t launch_bwd_short(int d, int dv, int score_mod, const BwdParams& p, int sm_count, cudaStream_t s) {
  if (dv != d) return launch_short_d<64, 128>(score_mod, p, sm_count, s);
  switch (d) {
    case 32: return launch_short_d<32, 32>(score_mod, p, sm_count, s);
    case 64: return launch_short_d<64, 64>(score_mod, p, sm_count, s);
    default: return launch_short_d<128, 128>(score_mod, p, sm_count, s);
  }
}

}  // namespace fl
