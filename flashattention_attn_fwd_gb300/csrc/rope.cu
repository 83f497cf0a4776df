// Rotation of queries and keys by their positions, forward and backward, and the
// tables that it reads.
//
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin   (fp32, every product and sum
//   rounded once, then y to bf16), pairs (c, c + rope_dim / 2) or (2c, 2c + 1)
//
// The gradient is the turn the other way: the same with -sin.  Bound by memory:
// every row is read and written once.  One warp takes one token: its position
// and rotation are then warp-uniform, and a lane keeps the cos and sin of its
// eight channels in registers for all heads, d / 8 lanes a row; the partner
// channel of the half-split pairing comes by shuffle.  Strides are free, so that
// the projection's token-major output becomes the [B, H, L, d] that the backward
// pass of attention takes, in the same pass.
//
// Measured: 2 x 8192 tokens of 32 + 8 heads of 128, half of the channels in pairs, 57 us
// (5.9 TB/s, 88 % of the copy rate); 4 x 2048 tokens of 2 x 16 heads of 64, 15 us a
// direction (4.4 TB/s: two waves of blocks and the launch); 64 tokens 6 us, the launch
// and three loads one after another.  Two or eight row groups in flight instead of
// four, more warps a token, registers for more blocks an SM: 20 to 40 % slower in the
// second case, whose blocks then make a third, ragged wave.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged_rows.cuh"
#include "ptx.cuh"
#include "rope.h"

namespace fl {
namespace {

constexpr int kRopeThreads = 128;

template <int D, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LPR = D / 8;        // lanes per row
  constexpr int RPS = 32 / LPR;     // rows a warp handles at once
  constexpr int NB = 4;             // row groups in flight per warp
  const int lane = threadIdx.x & 31;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x) >> 5;
  const int64_t token = w / p.splits;
  const int part = static_cast<int>(w % p.splits);
  if (token >= static_cast<int64_t>(p.B) * p.L) return;
  const int b = static_cast<int>(token / p.L), l = static_cast<int>(token % p.L);
  const int pos = p.positions ? __ldg(p.positions + b * p.pos_b + l) : l;
  const int sub = lane / LPR, c8 = lane % LPR, c0 = 8 * c8;
  if (pos < 0 || pos >= p.table_rows) {
    if (lane == 0 && part == 0) atomicOr(p.status, 2u);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const RopeRows& t = p.t[k];
      if (!t.zero) continue;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(t.y) + b * t.y_b + l * t.y_l + c0;
      for (int r = part * RPS + sub; r < t.heads; r += p.splits * RPS)
        *reinterpret_cast<uint4*>(dst + r * t.y_h) = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  const bool turn = c0 < p.rope_dim;
  const int half = p.rope_dim >> 1;
  const bool second = !PAIRS && c0 >= half;
  const int partner = turn && !PAIRS ? sub * LPR + (second ? c0 - half : c0 + half) / 8 : lane;
  // y = x cos + partner * sn; the first channel of a pair takes its partner with -sin
  float2 cs[4], sn[4];
  if (turn) {
    const int64_t row = static_cast<int64_t>(pos) * half;
    if (PAIRS) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(p.cos + row + c0 / 2));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(p.sin + row + c0 / 2));
      const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs[e] = make_float2(cc[e], cc[e]);
        sn[e] = make_float2(-p.sign * ss[e], p.sign * ss[e]);
      }
    } else {
      const int at = second ? c0 - half : c0;
      const float4* cp = reinterpret_cast<const float4*>(p.cos + row + at);
      const float4* sp = reinterpret_cast<const float4*>(p.sin + row + at);
      const float4 ca = __ldg(cp), cb = __ldg(cp + 1), sa = __ldg(sp), sb = __ldg(sp + 1);
      const float f = second ? p.sign : -p.sign;
      cs[0] = make_float2(ca.x, ca.y); cs[1] = make_float2(ca.z, ca.w);
      cs[2] = make_float2(cb.x, cb.y); cs[3] = make_float2(cb.z, cb.w);
      sn[0] = make_float2(f * sa.x, f * sa.y); sn[1] = make_float2(f * sa.z, f * sa.w);
      sn[2] = make_float2(f * sb.x, f * sb.y); sn[3] = make_float2(f * sb.z, f * sb.w);
    }
  }
  int first = 0;  // row groups before this tensor's
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const RopeRows& t = p.t[k];
    const int groups = (t.heads + RPS - 1) / RPS;
    int g = (part - first) % p.splits;
    if (g < 0) g += p.splits;
    first += groups;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(t.x) + b * t.x_b + l * t.x_l + c0;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(t.y) + b * t.y_b + l * t.y_l + c0;
    for (; g < groups; g += NB * p.splits) {
      uint4 raw[NB];
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        const int r = (g + u * p.splits) * RPS + sub;
        raw[u] = r < t.heads ? *reinterpret_cast<const uint4*>(src + r * t.x_h) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        if (g + u * p.splits >= groups) break;
        const int r = (g + u * p.splits) * RPS + sub;
        float2 x[4], y[4];
        unpack8(raw[u], x);
        if (PAIRS) {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = make_float2(x[e].y, x[e].x);
        } else {
          unpack8(make_uint4(__shfl_sync(0xffffffffu, raw[u].x, partner), __shfl_sync(0xffffffffu, raw[u].y, partner),
                             __shfl_sync(0xffffffffu, raw[u].z, partner), __shfl_sync(0xffffffffu, raw[u].w, partner)),
                  y);
        }
        if (turn) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // products and sums rounded one by one, as the cache's append does
            x[e].x = __fadd_rn(__fmul_rn(x[e].x, cs[e].x), __fmul_rn(y[e].x, sn[e].x));
            x[e].y = __fadd_rn(__fmul_rn(x[e].y, cs[e].y), __fmul_rn(y[e].y, sn[e].y));
          }
        }
        if (r < t.heads) *reinterpret_cast<uint4*>(dst + r * t.y_h) = turn ? pack8(x) : raw[u];
      }
    }
  }
}

template <int D>
cudaError_t launch_rope_d(RopeParams& p, int sm_count, cudaStream_t s) {
  constexpr int RPS = 32 / (D / 8);
  const int64_t tokens = static_cast<int64_t>(p.B) * p.L;
  const int groups = (p.t[0].heads + RPS - 1) / RPS + (p.t[1].heads + RPS - 1) / RPS;
  // spread a token's rows over more warps while that leaves fewer than 32 warps an SM
  int64_t splits = (static_cast<int64_t>(sm_count) * 32 + tokens - 1) / tokens;
  splits = splits > groups ? groups : splits;
  p.splits = static_cast<int>(splits);
  const int64_t blocks = (tokens * splits + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (p.interleaved) rope_kernel<D, true><<<static_cast<unsigned>(blocks), kRopeThreads, 0, s>>>(p);
  else rope_kernel<D, false><<<static_cast<unsigned>(blocks), kRopeThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// Tables: cos and sin of position * angle step.  The angle is a 64-bit fraction
// of a turn, so that position times step wraps exactly where a turn ends, in
// integers (fp64's rate is low).  What the step itself is off by grows with the
// position: the host's fp64 gives it within about 2^-55 turns (352 units of 2^-64 at
// worst over bases 1e4 and 5e5, 64 and 128 channels), 1e-10 of a turn at 2^22 positions.  Its quarter turns pick the function and the sign;
// the rest x, in half turns at most 1/4 either way, goes through
//   sin(pi x) = x S(x^2),  cos(pi x) = C(x^2)
// (fit_poly.py turn: within 9e-8, two channels an instruction).  A thread takes
// four neighbouring pairs at several positions.  131072 positions of 64 pairs: 12 us
// (5.4 TB/s of writes; with sincospif 18), 4096 of 32 pairs 4.1 (the launch).
constexpr int kTabThreads = 256;
constexpr int kTabRowsMax = 8;  // positions of a thread

struct TableLaunch {
  RopeTableParams t;
  int rows;  // positions of a thread
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__global__ void __launch_bounds__(kTabThreads) rope_tables_kernel(const __grid_constant__ TableLaunch a) {
  constexpr float kTurnS[4] = {3.14159274f, -5.16770792f, 2.54976106f, -0.589013278f};
  constexpr float kTurnC[5] = {1.f, -4.93480206f, 4.05870676f, -1.33503592f, 0.231261194f};
  const RopeTableParams& p = a.t;
  const int lanes = p.half / 4;              // threads of a position
  const int wide = kTabThreads / lanes;      // positions at once
  const int c = threadIdx.x % lanes, r = threadIdx.x / lanes;
  if (r >= wide) return;
  int64_t pos = static_cast<int64_t>(blockIdx.x) * wide * a.rows + r;
  uint64_t turn[4], step[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t t = p.turn[4 * c + e];
    turn[e] = t * static_cast<uint64_t>(pos) + (uint64_t(1) << 61);  // an eighth of a turn further
    step[e] = t * static_cast<uint64_t>(wide);
  }
  for (int k = 0; k < a.rows; ++k, pos += wide) {
    if (pos >= p.positions) return;
    float2 co[2], si[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t h0 = static_cast<uint32_t>(turn[2 * e] >> 32), h1 = static_cast<uint32_t>(turn[2 * e + 1] >> 32);
      turn[2 * e] += step[2 * e];
      turn[2 * e + 1] += step[2 * e + 1];
      // what is left of the quarter turn, in half turns
      const float2 x = ptx::mul2(make_float2(static_cast<float>(static_cast<int>(h0 & 0x3fffffffu) - (1 << 29)),
                                             static_cast<float>(static_cast<int>(h1 & 0x3fffffffu) - (1 << 29))),
                                 both(0x1p-31f));
      const float2 z = ptx::mul2(x, x);
      float2 s = ptx::fma2(both(kTurnS[3]), z, both(kTurnS[2]));
      s = ptx::fma2(s, z, both(kTurnS[1]));
      s = ptx::fma2(s, z, both(kTurnS[0]));
      s = ptx::mul2(s, x);
      float2 q = ptx::fma2(both(kTurnC[4]), z, both(kTurnC[3]));
      q = ptx::fma2(q, z, both(kTurnC[2]));
      q = ptx::fma2(q, z, both(kTurnC[1]));
      q = ptx::fma2(q, z, both(kTurnC[0]));
      s = ptx::mul2(s, both(p.amplitude));
      q = ptx::mul2(q, both(p.amplitude));
      // quarter 0: (q, s), 1: (-s, q), 2: (-q, -s), 3: (s, -q)
      auto place = [](uint32_t h, float s1, float q1, float& cosine, float& sine) {
        const bool odd = h & 0x40000000u;
        const uint32_t cs = (h ^ (h << 1)) & 0x80000000u, ss = h & 0x80000000u;
        cosine = __uint_as_float(__float_as_uint(odd ? s1 : q1) ^ cs);
        sine = __uint_as_float(__float_as_uint(odd ? q1 : s1) ^ ss);
      };
      place(h0, s.x, q.x, co[e].x, si[e].x);
      place(h1, s.y, q.y, co[e].y, si[e].y);
    }
    const int64_t at = pos * p.half + 4 * c;
    *reinterpret_cast<float4*>(p.cos + at) = make_float4(co[0].x, co[0].y, co[1].x, co[1].y);
    *reinterpret_cast<float4*>(p.sin + at) = make_float4(si[0].x, si[0].y, si[1].x, si[1].y);
  }
}

}  // namespace

cudaError_t launch_rope(int d, RopeParams& p, int sm_count, cudaStream_t s) {
  switch (d) {
    case 32: return launch_rope_d<32>(p, sm_count, s);
    case 64: return launch_rope_d<64>(p, sm_count, s);
    case 128: return launch_rope_d<128>(p, sm_count, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_rope_tables(const RopeTableParams& p, int sm_count, cudaStream_t s) {
  // several positions a thread once every SM has eight blocks
  const int wide = kTabThreads / (p.half / 4);
  const int64_t rows = static_cast<int64_t>(p.positions) / (static_cast<int64_t>(sm_count) * 8 * wide);
  const TableLaunch a{p, static_cast<int>(rows < 1 ? 1 : rows > kTabRowsMax ? kTabRowsMax : rows)};
  const int64_t per = static_cast<int64_t>(wide) * a.rows;
  rope_tables_kernel<<<static_cast<unsigned>((p.positions + per - 1) / per), kTabThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace fl
