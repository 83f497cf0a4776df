// What the kernels that move rows of tokens share: the sequence of a packed row,
// and eight bf16 channels as fp32 pairs.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace fl {

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

__device__ __forceinline__ void unpack8(const uint4& w, float2 (&x)[4]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = make_float2(__uint_as_float(v[e] << 16), __uint_as_float(v[e] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
  return make_uint4(ptx::pack_bf16x2(x[0].x, x[0].y), ptx::pack_bf16x2(x[1].x, x[1].y), ptx::pack_bf16x2(x[2].x, x[2].y),
                    ptx::pack_bf16x2(x[3].x, x[3].y));
}

}  // namespace fl
