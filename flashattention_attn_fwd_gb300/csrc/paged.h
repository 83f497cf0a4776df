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
  int cluster;               // CTAs of a cluster that share a unit; 0: the line is cut evenly
  uint32_t* status;
};

// CTAs of a cluster that takes one unit of at most `keys` keys, 0 for the line:
// a power of two up to the portable 8, no more than one 128-key round of a CTA's
// warps needs, and no more than fill half of the places for CTAs (128 units of
// 1092 keys: 12.0 us in pairs, 13.2 in fours and 13.0 alone).  Past kClusterKeys
// per CTA the line's even cut is worth its plan and merge (5 us).
constexpr int kClusterMax = 8;
constexpr int64_t kClusterKeys = 2048;
inline int paged_cluster(int64_t keys, int64_t units, int64_t resident) {
  int c = 1;
  while (c < kClusterMax && keys > 128 * static_cast<int64_t>(c) && units * 4 * c <= resident) c *= 2;
  return keys <= kClusterKeys * c ? c : 0;
}

// Per format and head dim: resident CTAs per SM of the cluster's or the line's
// kernel for M rows (< 1 on a CUDA error; call before a launch), and the launch.
#define FL_DECLARE_PAGED(NAME)                     \
  int paged_resident_##NAME(int M, bool cluster);  \
  cudaError_t launch_paged_##NAME(const PagedDecodeParams& p, cudaStream_t s);
FL_DECLARE_PAGED(bf16_d64)
FL_DECLARE_PAGED(bf16_d128)
FL_DECLARE_PAGED(e2m1_d64)
FL_DECLARE_PAGED(e2m1_d128)
#undef FL_DECLARE_PAGED

inline int paged_resident(int format, int d, int M, bool cluster) {
  if (format == KV_BF16) return d == 64 ? paged_resident_bf16_d64(M, cluster) : paged_resident_bf16_d128(M, cluster);
  return d == 64 ? paged_resident_e2m1_d64(M, cluster) : paged_resident_e2m1_d128(M, cluster);
}
inline cudaError_t launch_paged_decode(int format, int d, const PagedDecodeParams& p, cudaStream_t s) {
  if (format == KV_BF16) return d == 64 ? launch_paged_bf16_d64(p, s) : launch_paged_bf16_d128(p, s);
  return d == 64 ? launch_paged_e2m1_d64(p, s) : launch_paged_e2m1_d128(p, s);
}

}  // namespace fl
