// Rotation of new queries and keys and their append, with the values, to a
// paged cache in bf16 or in 4 bits.
//
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin            (fp32)
//   bf16: y rounded once
//   e2m1: u = y (1 / cache scale);  s = e4m3(max|u| over 16 channels (1/6));
//         code = e2m1(u / s)                    (each step rounded once)
//
// The kernel moves bytes: every row is read and written once and a channel
// costs a few operations.  One warp takes one token (its place in the cache
// and its rotation are then warp-uniform) and d / 8 lanes take one head's
// row, eight channels (16 bytes) each.  A lane keeps its channels' cos and
// sin in registers for all heads of the token, so the tables are read once a
// token; the partner channel of the half-split pairing sits in another lane of
// the row and comes by shuffle, and the two lanes of a 16-channel block share
// their maxima the same way.  With few tokens the rows of one are spread over
// several warps.
//
// Measured: one token 2.9 us, which is the launch; 9730 prompt tokens of 32 + 2 x 8
// heads of 128 channels into 4 bits, stored values back, 51 us (4.9 TB/s of what
// it must move); 16384 tokens of 3 x 16 heads of 64 in bf16, values back, 44 us
// (6.1 TB/s).  Bound by memory in bf16; in 4 bits by loads that wait (half of
// the warps' time) with the conversion's instructions in 57 % of the issue
// slots: 80 registers for six blocks an SM were 54 -> 51 us, eight or two row
// groups in flight instead of four slower.  With that cap the 4-bit kernels spill
// (half-split rotation 56 to 60 bytes, reloaded 164 to 176; in pairs 20 and 36; none
// 4), which the residency outweighs.
//
// A product and a sum are rounded separately (no fused multiply-add), so that
// a value next to a rounding border of the 4-bit code falls to the side that
// the definition says.  The code of u / s is decided on the correctly rounded
// quotient: with r = 1 / s correctly rounded, q = u r and one residual step q -
// r (q s - u) give it (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990), three operations where the general
// division takes a dozen.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cvt4.cuh"
#include "paged.h"
#include "paged_rows.cuh"
#include "ptx.cuh"

namespace fl {
namespace {

constexpr int kAppThreads = 128;
constexpr float kSixth = 1.0f / 6.0f;
// Above this a block saturates its scale: its values are clamped first, so that
// an infinite one goes through the quotient's residual.
constexpr float kBlockMax = 448.0f * 6.0f;

enum Rope : int { ROPE_NONE = 0, ROPE_HALF = 1, ROPE_PAIRS = 2 };

template <int FMT, int D, int ROPE>
__global__ void __launch_bounds__(kAppThreads, 6) kv_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPR = D / 8;        // lanes per row
  constexpr int RPS = 32 / LPR;     // rows a warp handles at once
  constexpr int NB = 4;             // row groups in flight per warp
  const int lane = threadIdx.x & 31;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kAppThreads + threadIdx.x) >> 5;
  const int t = static_cast<int>(w / p.splits);
  const int part = static_cast<int>(w % p.splits);
  if (t >= p.T) return;
  int b = t, i = 0, n = 1;
  if (p.seq_offsets) {
    b = sequence_of(p.seq_offsets, p.B, t, lane);
    if (b >= p.B) return;  // a row behind the last sequence
    const int first = __ldg(p.seq_offsets + b);
    i = t - first;
    n = __ldg(p.seq_offsets + b + 1) - first;
  }
  const int pos = __ldg(p.kv_len + b) - n + i;
  if (pos < 0 || i < 0) return;
  const int page_size = 1 << p.c.page_shift;
  const int col = pos >> p.c.page_shift;
  int page = -1;
  if (col < p.max_pages && (ROPE == ROPE_NONE || pos < p.rope_positions)) page = __ldg(p.table + b * p.table_stride + col);
  if (page < 0 || page >= p.c.num_pages) {
    if (lane == 0 && part == 0) atomicOr(p.status, 2u);
    return;
  }
  const int at = pos & (page_size - 1);
  const int sub = lane / LPR, c8 = lane % LPR;
  const int c0 = 8 * c8;
  // this lane's rotation: cs, sn of channels c0 .. c0 + 7 in pairs, the sign of
  // sin folded in (y = x cos + partner * sn; the partner of the first channel
  // of a pair enters with -sin)
  const bool turn = ROPE != ROPE_NONE && c0 < p.rope_dim;
  const int half = p.rope_dim >> 1;
  const bool second = ROPE == ROPE_HALF && c0 >= half;
  const int partner = turn && ROPE == ROPE_HALF ? sub * LPR + (second ? c0 - half : c0 + half) / 8 : lane;
  float2 cs[4], sn[4];
  if (turn) {
    const int64_t row = static_cast<int64_t>(pos) * half;
    if (ROPE == ROPE_PAIRS) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(p.cos + row + c0 / 2));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(p.sin + row + c0 / 2));
      const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs[e] = make_float2(cc[e], cc[e]);
        sn[e] = make_float2(-ss[e], ss[e]);
      }
    } else {
      const float4* cp = reinterpret_cast<const float4*>(p.cos + row + (second ? c0 - half : c0));
      const float4* sp = reinterpret_cast<const float4*>(p.sin + row + (second ? c0 - half : c0));
      const float4 ca = __ldg(cp), cb = __ldg(cp + 1), sa = __ldg(sp), sb = __ldg(sp + 1);
      const float f = second ? 1.f : -1.f;
      cs[0] = make_float2(ca.x, ca.y); cs[1] = make_float2(ca.z, ca.w);
      cs[2] = make_float2(cb.x, cb.y); cs[3] = make_float2(cb.z, cb.w);
      sn[0] = make_float2(f * sa.x, f * sa.y); sn[1] = make_float2(f * sa.z, f * sa.w);
      sn[2] = make_float2(f * sb.x, f * sb.y); sn[3] = make_float2(f * sb.z, f * sb.w);
    }
  }
  auto rotate = [&](const uint4& raw, float2 (&x)[4]) {
    float2 y[4];
    if (ROPE == ROPE_HALF) {
      const uint4 o = make_uint4(__shfl_sync(0xffffffffu, raw.x, partner), __shfl_sync(0xffffffffu, raw.y, partner),
                                 __shfl_sync(0xffffffffu, raw.z, partner), __shfl_sync(0xffffffffu, raw.w, partner));
      unpack8(o, y);
    } else if (ROPE == ROPE_PAIRS) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = make_float2(x[e].y, x[e].x);
    }
    if (ROPE != ROPE_NONE && turn) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // scalar: the packed product and sum came out fused
        x[e].x = __fadd_rn(__fmul_rn(x[e].x, cs[e].x), __fmul_rn(y[e].x, sn[e].x));
        x[e].y = __fadd_rn(__fmul_rn(x[e].y, cs[e].y), __fmul_rn(y[e].y, sn[e].y));
      }
    }
  };
  // Rows r = part-th, (part + splits)-th ... group of `heads` rows of a tensor,
  // NB groups in flight; `first`: groups before this tensor's.
  auto for_rows = [&](const void* base, int64_t st, int64_t sh, int heads, int first, auto&& row) {
    const int groups = (heads + RPS - 1) / RPS;
    int g = (part - first) % p.splits;
    if (g < 0) g += p.splits;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(base) + t * st + c0;
    for (; g < groups; g += NB * p.splits) {
      uint4 raw[NB];
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        const int r = (g + u * p.splits) * RPS + sub;
        raw[u] = r < heads ? *reinterpret_cast<const uint4*>(src + r * sh) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        if (g + u * p.splits >= groups) break;
        const int r = (g + u * p.splits) * RPS + sub;
        row(raw[u], r, r < heads);
      }
    }
  };
  const int Hkv = p.c.Hkv;
  const int q_groups = (p.Hq + RPS - 1) / RPS, k_groups = (Hkv + RPS - 1) / RPS;
  if (p.Hq) {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.q_out) + t * p.qo_t + c0;
    for_rows(p.q, p.q_t, p.q_h, p.Hq, 0, [&](const uint4& raw, int r, bool ok) {
      float2 x[4];
      unpack8(raw, x);
      rotate(raw, x);
      if (ok) *reinterpret_cast<uint4*>(dst + r * p.qo_h) = pack8(x);
    });
  }
  // stores row h of K or V: cache (and the values that it now holds)
  auto store = [&](float2 (&x)[4], int h, bool ok, bool is_v, void* pool, uint8_t* scales, float inv, float scale,
                   void* out, int64_t ot, int64_t oh) {
    const int64_t run = (static_cast<int64_t>(page) * Hkv + h) << p.c.page_shift;  // tokens before this head
    const int64_t slot = run + at;
    uint4 held;
    if constexpr (FMT == KV_BF16) {
      held = pack8(x);
      if (ok) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pool) + slot * D + c0) = held;
    } else {
      // x becomes -u: see the residual step
      const float2 inv2 = make_float2(-inv, -inv);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = ptx::mul2(x[e], inv2);
      float a = fmaxf(fabsf(x[0].x), fabsf(x[0].y));
#pragma unroll
      for (int e = 1; e < 4; ++e) a = ptx::max3(a, fabsf(x[e].x), fabsf(x[e].y));
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
      const uint32_t s8 = cvt4::to_e4m3(__fmul_rn(a, kSixth));
      const float s = cvt4::unpack_f16x2(cvt4::from_e4m3x2(s8)).x;
      if (a > kBlockMax) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = make_float2(fminf(fmaxf(x[e].x, -2.f * kBlockMax), 2.f * kBlockMax),
                             fminf(fmaxf(x[e].y, -2.f * kBlockMax), 2.f * kBlockMax));
      }
      const float rs = s > 0.f ? __frcp_rn(s) : 0.f;  // a zero scale: all codes zero
      // q - r (q s - u): with these signs a zero keeps its own, where q + r (u -
      // q s) would make -0 of u a +0
      const float2 nr2 = make_float2(-rs, -rs), s2 = make_float2(s, s);
      float z[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 q = ptx::mul2(x[e], nr2);
        const float2 f = ptx::fma2(ptx::fma2(q, s2, x[e]), nr2, q);
        z[2 * e] = s > 0.f ? f.x : 0.f;
        z[2 * e + 1] = s > 0.f ? f.y : 0.f;
      }
      const uint32_t code = cvt4::to_e2m1x8(z);
      if (ok) {
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(pool) + slot * (D / 2) + c0 / 2) = code;
        if ((c8 & 1) == 0)
          scales[is_v ? run * (D / kScaleBlock) + (static_cast<int64_t>(c8 >> 1) << p.c.page_shift) + at
                      : slot * (D / kScaleBlock) + (c8 >> 1)] = s8;
      }
      if (out) {
        uint32_t hv[4];
        cvt4::from_e2m1x8(code, hv);
        const float2 g2 = make_float2(scale, scale);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = ptx::mul2(ptx::mul2(cvt4::unpack_f16x2(hv[e]), s2), g2);
        held = pack8(x);
      }
    }
    if (out && ok) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + t * ot + h * oh + c0) = held;
  };
  for_rows(p.k, p.k_t, p.k_h, Hkv, q_groups, [&](const uint4& raw, int h, bool ok) {
    float2 x[4];
    unpack8(raw, x);
    rotate(raw, x);
    store(x, h, ok, false, p.c.k, p.c.ks, p.inv_k_scale, p.c.k_scale, p.k_out, p.ko_t, p.ko_h);
  });
  for_rows(p.v, p.v_t, p.v_h, Hkv, q_groups + k_groups, [&](const uint4& raw, int h, bool ok) {
    float2 x[4];
    unpack8(raw, x);
    store(x, h, ok, true, p.c.v, p.c.vs, p.inv_v_scale, p.c.v_scale, p.v_out, p.vo_t, p.vo_h);
  });
}

template <int FMT, int D, int ROPE>
cudaError_t launch_append(AppendParams& p, int sm_count, cudaStream_t s) {
  constexpr int RPS = 32 / (D / 8);
  const int groups = (p.Hq + RPS - 1) / RPS + 2 * ((p.c.Hkv + RPS - 1) / RPS);
  // spread a token's rows over more warps while that leaves fewer than 32
  // warps an SM
  const int64_t want = static_cast<int64_t>(sm_count) * 32;
  int64_t splits = (want + p.T - 1) / p.T;
  splits = splits < 1 ? 1 : splits > groups ? groups : splits;
  p.splits = static_cast<int>(splits);
  const int64_t warps = splits * p.T;
  const int64_t blocks = (warps + kAppThreads / 32 - 1) / (kAppThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  kv_append_kernel<FMT, D, ROPE><<<static_cast<unsigned>(blocks), kAppThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int FMT, int D>
cudaError_t launch_append_d(AppendParams& p, int sm_count, cudaStream_t s) {
  if (!p.rope_dim) return launch_append<FMT, D, ROPE_NONE>(p, sm_count, s);
  return p.interleaved ? launch_append<FMT, D, ROPE_PAIRS>(p, sm_count, s) : launch_append<FMT, D, ROPE_HALF>(p, sm_count, s);
}

}  // namespace

cudaError_t launch_kv_append(int format, int d, AppendParams& p, int sm_count, cudaStream_t s) {
  if (format == KV_BF16) return d == 64 ? launch_append_d<KV_BF16, 64>(p, sm_count, s) : launch_append_d<KV_BF16, 128>(p, sm_count, s);
  return d == 64 ? launch_append_d<KV_E2M1, 64>(p, sm_count, s) : launch_append_d<KV_E2M1, 128>(p, sm_count, s);
}

}  // namespace fl
