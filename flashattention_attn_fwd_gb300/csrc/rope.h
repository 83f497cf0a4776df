// Rotary positions: parameters shared by the host entry points and the kernels
// (internal header).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace fl {

constexpr int kRopeMaxDim = 128;

struct RopeRows {
  const void* x;
  void* y;
  int64_t x_b, x_h, x_l, y_b, y_h, y_l;  // strides, elements
  int heads;
  int zero;  // rows without a position in the tables become zeros
};

struct RopeParams {
  RopeRows t[2];             // queries, keys (heads 0: none)
  const float* cos;
  const float* sin;
  const int32_t* positions;  // null: row l takes position l
  int64_t pos_b;             // elements between the batches' positions
  int B, L, table_rows, rope_dim, interleaved;
  float sign;                // -1: the backward pass, a turn the other way
  int splits;                // warps that share one token's rows
  uint32_t* status;
};
cudaError_t launch_rope(int d, RopeParams& p, int sm_count, cudaStream_t s);

struct RopeTableParams {
  float* cos;
  float* sin;
  int positions, half;
  float amplitude;
  uint64_t turn[kRopeMaxDim / 2];  // of a position step: its fraction of a turn in units of 2^-64
};
cudaError_t launch_rope_tables(const RopeTableParams& p, int sm_count, cudaStream_t s);

}  // namespace fl
