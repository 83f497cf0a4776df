// Rotation of new queries and keys and their append, with the values, to a
// paged cache in bf16 or in 4 bits.
//
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin            (fp32)
//   bf16: y rounded once
//   e2m1: u = y / cache scale;  s = e4m3(max|u| over 16 channels / 6);
//         code = e2m1(u / s)
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
// A product and a sum are rounded separately (no fused multiply-add), so that
// a value next to a rounding border of the 4-bit code falls to the side that
// the definition says.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cvt4.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace fl {
namespace {

constexpr int kAppThreads = 128;
constexpr float kSixth = 1.0f / 6.0f;

// Sequence of row t: the number of seq_offsets[1..] that are <= t, found by
// narrowing 32-fold (a warp-wide count a step); B when t is past the last.
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int B, int t, int lane) {
  int lo = 0, n = B;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + (lane + 1) * step;  // offsets[i] <= t: the answer is at least i
    const bool le = (lane + 1) * step <= n && __ldg(offsets + i) <= t;
    lo += __popc(__ballot_sync(0xffffffffu, le)) * step;
    const int rest = B - lo;
    n = step - 1 < rest ? step - 1 : rest;
  }
  return lo;
}

template <int FMT, int D>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
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
  if (col < p.max_pages && (p.rope_dim == 0 || pos < p.rope_positions)) page = __ldg(p.table + b * p.table_stride + col);
  if (page < 0 || page >= p.c.num_pages) {
    if (lane == 0 && part == 0) atomicOr(p.status, 2u);
    return;
  }
  const int at = pos & (page_size - 1);
  const int sub = lane / LPR, c8 = lane % LPR;
  const int c0 = 8 * c8;
  // this lane's rotation: cs[e], sn[e] of channel c0 + e, the sign of sin
  // folded in (y = x cos + partner * sn; the partner of the first channel of
  // a pair enters with -sin)
  const bool turn = c0 < p.rope_dim;
  const int half = p.rope_dim >> 1;
  const bool second = !p.interleaved && c0 >= half;
  const int partner = turn && !p.interleaved ? sub * LPR + (second ? c0 - half : c0 + half) / 8 : lane;
  float cs[8], sn[8];
  if (turn) {
    const int64_t row = static_cast<int64_t>(pos) * half;
    if (p.interleaved) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(p.cos + row + c0 / 2));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(p.sin + row + c0 / 2));
      cs[0] = cs[1] = c4.x; cs[2] = cs[3] = c4.y; cs[4] = cs[5] = c4.z; cs[6] = cs[7] = c4.w;
      sn[1] = s4.x; sn[3] = s4.y; sn[5] = s4.z; sn[7] = s4.w;
      sn[0] = -s4.x; sn[2] = -s4.y; sn[4] = -s4.z; sn[6] = -s4.w;
    } else {
      const float4* cp = reinterpret_cast<const float4*>(p.cos + row + (second ? c0 - half : c0));
      const float4* sp = reinterpret_cast<const float4*>(p.sin + row + (second ? c0 - half : c0));
      const float4 ca = __ldg(cp), cb = __ldg(cp + 1), sa = __ldg(sp), sb = __ldg(sp + 1);
      const float f = second ? 1.f : -1.f;
      cs[0] = ca.x; cs[1] = ca.y; cs[2] = ca.z; cs[3] = ca.w; cs[4] = cb.x; cs[5] = cb.y; cs[6] = cb.z; cs[7] = cb.w;
      sn[0] = f * sa.x; sn[1] = f * sa.y; sn[2] = f * sa.z; sn[3] = f * sa.w;
      sn[4] = f * sb.x; sn[5] = f * sb.y; sn[6] = f * sb.z; sn[7] = f * sb.w;
    }
  }
  const int Hkv = p.c.Hkv;
  const int rows = p.Hq + 2 * Hkv;  // q heads, then k heads, then v heads
  const int groups = (rows + RPS - 1) / RPS;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + t * p.q_t;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + t * p.k_t;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + t * p.v_t;
  for (int g0 = part; g0 < groups; g0 += NB * p.splits) {
    uint4 raw[NB];
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const int r = (g0 + u * p.splits) * RPS + sub;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) {
        const __nv_bfloat16* src = r < p.Hq ? q + r * p.q_h
                                   : r < p.Hq + Hkv ? k + (r - p.Hq) * p.k_h
                                                    : v + (r - p.Hq - Hkv) * p.v_h;
        raw[u] = *reinterpret_cast<const uint4*>(src + c0);
      }
    }
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      if (g0 + u * p.splits >= groups) break;
      const int r = (g0 + u * p.splits) * RPS + sub;
      const uint32_t own[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(own[e] << 16);
        x[2 * e + 1] = __uint_as_float(own[e] & 0xffff0000u);
      }
      const bool is_v = r >= p.Hq + Hkv;
      if (p.rope_dim) {
        float y[8];
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t o = __shfl_sync(0xffffffffu, own[e], partner);
            y[2 * e] = __uint_as_float(o << 16);
            y[2 * e + 1] = __uint_as_float(o & 0xffff0000u);
          }
        }
        if (turn && !is_v) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __fadd_rn(__fmul_rn(x[e], cs[e]), __fmul_rn(y[e], sn[e]));
        }
      }
      const uint4 rounded = make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]),
                                       ptx::pack_bf16x2(x[4], x[5]), ptx::pack_bf16x2(x[6], x[7]));
      const int h = is_v ? r - p.Hq - Hkv : r - p.Hq;  // key/value head
      if (FMT == KV_BF16) {
        if (r < p.Hq) {
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) + t * p.qo_t + r * p.qo_h + c0) = rounded;
        } else if (r < rows) {
          const int64_t slot = ((static_cast<int64_t>(page) * Hkv + h) << p.c.page_shift) + at;
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? p.c.v : p.c.k) + slot * D + c0) = rounded;
          if (p.k_out) {
            __nv_bfloat16* o = is_v ? static_cast<__nv_bfloat16*>(p.v_out) + t * p.vo_t + h * p.vo_h
                                    : static_cast<__nv_bfloat16*>(p.k_out) + t * p.ko_t + h * p.ko_h;
            *reinterpret_cast<uint4*>(o + c0) = rounded;
          }
        }
      } else {
        const float inv = is_v ? p.inv_v_scale : p.inv_k_scale;
        float a = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // q rows keep x (stored below); their u is not used
          a = fmaxf(a, fabsf(__fmul_rn(x[e], inv)));
        }
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
        if (r < p.Hq) {
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) + t * p.qo_t + r * p.qo_h + c0) = rounded;
        } else if (r < rows) {
          const uint32_t s8 = cvt4::to_e4m3(__fmul_rn(a, kSixth));
          const float s = cvt4::unpack_f16x2(cvt4::from_e4m3x2(s8)).x;
          float z[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = s > 0.f ? __fdiv_rn(__fmul_rn(x[e], inv), s) : 0.f;
          const uint32_t code = cvt4::to_e2m1x8(z);
          const int64_t run = (static_cast<int64_t>(page) * Hkv + h) << p.c.page_shift;  // tokens before this head
          const int64_t slot = run + at;
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(is_v ? p.c.v : p.c.k) + slot * (D / 2) + c0 / 2) = code;
          if ((c8 & 1) == 0) {
            if (is_v) p.c.vs[run * (D / kScaleBlock) + (static_cast<int64_t>(c8 >> 1) << p.c.page_shift) + at] = s8;
            else p.c.ks[slot * (D / kScaleBlock) + (c8 >> 1)] = s8;
          }
          if (p.k_out) {
            const float g = is_v ? p.c.v_scale : p.c.k_scale;
            uint32_t hv[4], o4[4];
            cvt4::from_e2m1x8(code, hv);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = cvt4::unpack_f16x2(hv[e]);
              o4[e] = ptx::pack_bf16x2(__fmul_rn(__fmul_rn(f.x, s), g), __fmul_rn(__fmul_rn(f.y, s), g));
            }
            __nv_bfloat16* o = is_v ? static_cast<__nv_bfloat16*>(p.v_out) + t * p.vo_t + h * p.vo_h
                                    : static_cast<__nv_bfloat16*>(p.k_out) + t * p.ko_t + h * p.ko_h;
            *reinterpret_cast<uint4*>(o + c0) = make_uint4(o4[0], o4[1], o4[2], o4[3]);
          }
        }
      }
    }
  }
}

template <int FMT, int D>
cudaError_t launch_append(AppendParams& p, int sm_count, cudaStream_t s) {
  constexpr int RPS = 32 / (D / 8);
  const int groups = (p.Hq + 2 * p.c.Hkv + RPS - 1) / RPS;
  // spread a token's rows over more warps while that leaves fewer than 32
  // warps an SM
  const int64_t want = static_cast<int64_t>(sm_count) * 32;
  int64_t splits = (want + p.T - 1) / p.T;
  splits = splits < 1 ? 1 : splits > groups ? groups : splits;
  p.splits = static_cast<int>(splits);
  const int64_t warps = splits * p.T;
  const int64_t blocks = (warps + kAppThreads / 32 - 1) / (kAppThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  kv_append_kernel<FMT, D><<<static_cast<unsigned>(blocks), kAppThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(int format, int d, AppendParams& p, int sm_count, cudaStream_t s) {
  if (format == KV_BF16) return d == 64 ? launch_append<KV_BF16, 64>(p, sm_count, s) : launch_append<KV_BF16, 128>(p, sm_count, s);
  return d == 64 ? launch_append<KV_E2M1, 64>(p, sm_count, s) : launch_append<KV_E2M1, 128>(p, sm_count, s);
}

}  // namespace fl
