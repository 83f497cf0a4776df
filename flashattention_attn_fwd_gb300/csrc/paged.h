// Paged key/value cache: parameters shared by the host entry points, the
// append kernel and the decode kernels (internal header).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace fl {

enum KvFormat : int { KV_BF16 = 0, KV_E2M1 = 1 };

constexpr int kScaleBlock = 16;  // channels that share one e4m3 scale

struct PagedCache {
  void* k;
  void* v;
  uint8_t* ks;  // e4m3 [page][head][token][d / 16]
  uint8_t* vs;  // e4m3 [page][head][d / 16][token]
  float k_scale, v_scale;
  int num_pages, page_shift, Hkv;
};

struct AppendParams {
  PagedCache c;
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_out;
  void* v_out;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h;  // (token, head) strides, elements
  int64_t qo_t, qo_h, ko_t, ko_h, vo_t, vo_h;
  const int32_t* seq_offsets;
  const int32_t* kv_len;
  const int32_t* table;
  int64_t table_stride;
  const float* cos;
  const float* sin;
  float inv_k_scale, inv_v_scale;
  int T, B, Hq, max_pages;
  int rope_positions, rope_dim, interleaved;
  int splits;       // warps that share one token's rows
  uint32_t* status;
};

cudaError_t launch_kv_append(int format, int d, AppendParams& p, int sm_count, cudaStream_t s);

// Query rows (heads of a group times Lq) one call serves per key/value head.
constexpr int kPagedMaxRows = 64;

struct PagedDecodeParams {
  PagedCache c;
  const void* q;
  void* out;
  float* lse;
  int64_t q_b, q_h, q_l, o_b, o_h, o_l;  // strides, elements
  const int32_t* kv_len;
  const int32_t* table;
  int64_t table_stride;
  const float* slopes;
  int B, Hq, Lq, G, M;       // M = G * Lq rows per key/value head
  int max_pages, cap;        // cap = max_pages * page_size
  float scale_log2;          // scale * log2(e) * k_scale
  float softcap;             // in log2 units (cap * log2(e))
  int score_mod, causal, window, sink;  // window 0: none
  // workspace: the plan (tiles per CTA, then for every sequence the tiles of
  // one head before it) and two partial results for every CTA
  int64_t* plan;
  float* opart;              // [grid][2][M][d], normalised
  float* lpart;              // [grid][2][M], log2
  int grid;
  uint32_t* status;
};

// CTAs of the decode kernel for M rows (every one resident at once), < 0 on a
// CUDA error.
int paged_decode_grid(int format, int d, int M, int sm_count);

cudaError_t launch_paged_decode(int format, int d, const PagedDecodeParams& p, cudaStream_t s);

}  // namespace fl
