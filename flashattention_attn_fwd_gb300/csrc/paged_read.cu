// Reading a paged key/value cache back: rows of packed tokens in bf16.
//
//   bf16: the stored row;  e2m1: code * block scale * cache scale  (fp32, the code
//   times its scale exact, then rounded once to fp32 and once to bf16)
//
// Bound by memory: per row and head 2 d bytes out and 2 d (bf16) or d / 2 + d / 16
// (4 bits) in.  A warp takes four consecutive tokens, d / 8 lanes a row, and goes
// through the heads: one head's rows of neighbouring tokens lie side by side in
// a page, scales of the values too, so that every sector read is used (the rest by
// the neighbouring warps), and rows go out as whole lines.  With few tokens the
// heads are spread over several warps.
//
// Measured: 12 sequences of 5001 to 20000 tokens, 8 heads of 128 in 4 bits, 111 us for
// 667 MB (6.0 TB/s, 89 % of the copy rate; eight tokens a warp 115, sixteen 119);
// one of 701, 8 heads of 64, 5.4 us (eight tokens 6.1), four loads one after another.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cvt4.cuh"
#include "paged.h"
#include "paged_rows.cuh"
#include "ptx.cuh"

namespace fl {
namespace {

constexpr int kReadThreads = 128;
constexpr int kReadTokens = 4;  // of a warp

struct ReadLaunch {
  ReadParams r;
  int splits;  // warps that share four tokens' heads
};

template <int FMT, int D>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const __grid_constant__ ReadLaunch a) {
  constexpr int LPR = D / 8;                // lanes per row
  constexpr int RPS = 32 / LPR;             // rows a warp handles at once
  constexpr int N = kReadTokens / RPS;      // rows of a lane
  const ReadParams& p = a.r;
  const int lane = threadIdx.x & 31;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kReadThreads + threadIdx.x) >> 5;
  const int64_t t0 = w / a.splits * kReadTokens;
  const int part = static_cast<int>(w % a.splits);
  if (t0 >= p.T) return;
  int b = p.seq_offsets ? sequence_of(p.seq_offsets, p.B, static_cast<int>(t0), lane) : static_cast<int>(t0);
  const int sub = lane / LPR, c8 = lane % LPR, c0 = 8 * c8;
  const int shift = p.c.page_shift, page_mask = (1 << shift) - 1;
  int64_t run[N];  // tokens before this one's page's first head; < 0: no row
  int at[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    run[i] = -1;
    at[i] = 0;
    const int64_t t = t0 + i * RPS + sub;
    if (t >= p.T) continue;
    int pos;
    if (p.seq_offsets) {
      int end = 0;
      while (b < p.B && (end = __ldg(p.seq_offsets + b + 1)) <= t) ++b;
      if (b >= p.B) continue;  // a row behind the last sequence
      pos = __ldg(p.kv_len + b) - end + static_cast<int>(t);
    } else {
      b = static_cast<int>(t);
      pos = __ldg(p.kv_len + b) - 1;
    }
    if (pos < 0) continue;
    const int col = pos >> shift;
    const int page = col < p.max_pages ? __ldg(p.table + b * p.table_stride + col) : -1;
    if (page < 0 || page >= p.c.num_pages) {
      if (c8 == 0 && part == 0) atomicOr(p.status, 2u);
      continue;
    }
    run[i] = (static_cast<int64_t>(page) * p.c.Hkv) << shift;
    at[i] = pos & page_mask;
  }
  for (int h = part; h < p.c.Hkv; h += a.splits) {
    const int64_t head = static_cast<int64_t>(h) << shift;
    if constexpr (FMT == KV_BF16) {
      uint4 x[2][N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t row = (run[i] + head + at[i]) * D + c0;
        if (run[i] >= 0) {
          x[0][i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.c.k) + row));
          x[1][i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.c.v) + row));
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (run[i] < 0) continue;
        const int64_t t = t0 + i * RPS + sub;
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k_out) + t * p.ko_t + h * p.ko_h + c0) = x[0][i];
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.v_out) + t * p.vo_t + h * p.vo_h + c0) = x[1][i];
      }
    } else {
      uint32_t code[2][N];
      uint8_t s8[2][N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t first = run[i] + head, slot = first + at[i];
        if (run[i] >= 0) {
          code[0][i] = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.c.k) + slot * (D / 2)) + c8);
          code[1][i] = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.c.v) + slot * (D / 2)) + c8);
          s8[0][i] = __ldg(p.c.ks + slot * (D / kScaleBlock) + (c8 >> 1));
          s8[1][i] = __ldg(p.c.vs + first * (D / kScaleBlock) + (static_cast<int64_t>(c8 >> 1) << shift) + at[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (run[i] < 0) continue;
        const int64_t t = t0 + i * RPS + sub;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const float s = cvt4::unpack_f16x2(cvt4::from_e4m3x2(s8[v][i])).x;
          const float2 s2 = make_float2(s, s);
          const float g = v ? p.c.v_scale : p.c.k_scale;
          const float2 g2 = make_float2(g, g);
          uint32_t hv[4];
          cvt4::from_e2m1x8(code[v][i], hv);
          float2 x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = ptx::mul2(ptx::mul2(cvt4::unpack_f16x2(hv[e]), s2), g2);
          __nv_bfloat16* dst = v ? static_cast<__nv_bfloat16*>(p.v_out) + t * p.vo_t + h * p.vo_h
                                 : static_cast<__nv_bfloat16*>(p.k_out) + t * p.ko_t + h * p.ko_h;
          __stcs(reinterpret_cast<uint4*>(dst + c0), pack8(x));
        }
      }
    }
  }
}

template <int FMT, int D>
cudaError_t launch_read(const ReadParams& p, int sm_count, cudaStream_t s) {
  const int64_t groups = (static_cast<int64_t>(p.T) + kReadTokens - 1) / kReadTokens;
  // spread a group's heads over more warps while that leaves fewer than 32 warps an SM
  int64_t splits = (static_cast<int64_t>(sm_count) * 32 + groups - 1) / groups;
  splits = splits > p.c.Hkv ? p.c.Hkv : splits;
  const ReadLaunch a{p, static_cast<int>(splits)};
  const int64_t blocks = (groups * splits + kReadThreads / 32 - 1) / (kReadThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  kv_read_kernel<FMT, D><<<static_cast<unsigned>(blocks), kReadThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_read(int format, int d, const ReadParams& p, int sm_count, cudaStream_t s) {
  if (format == KV_BF16) return d == 64 ? launch_read<KV_BF16, 64>(p, sm_count, s) : launch_read<KV_BF16, 128>(p, sm_count, s);
  return d == 64 ? launch_read<KV_E2M1, 64>(p, sm_count, s) : launch_read<KV_E2M1, 128>(p, sm_count, s);
}

}  // namespace fl
