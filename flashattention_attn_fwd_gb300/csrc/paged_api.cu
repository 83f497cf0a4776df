// C ABI of the paged key/value cache: argument checks, parameters and
// launches of the append and of the decode attention.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "flattn.h"
#include "host.h"
#include "paged.h"

namespace {

constexpr double kLog2e = 1.4426950408889634;
// Tokens a sequence's table can name: positions and window arithmetic stay
// within 32 bits.
constexpr int64_t kMaxTokens = int64_t(1) << 30;

// Rows (heads times tokens) of a page: its bytes stay below 2^31.
constexpr int64_t kMaxPageRows = int64_t(1) << 22;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool normal_scale(float x) { return x > 0.f && std::isnormal(x) && std::isnormal(1.0f / x); }

fl_status cache_check(const fl_kv_cache* c) {
  if (!c || !c->k || !c->v) return FL_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->Hkv < 1 || c->page_size < 1 || c->d < 1) return FL_ERR_INVALID_ARG;
  if (c->format != FL_KV_BF16 && c->format != FL_KV_E2M1) return FL_ERR_INVALID_ARG;
  if (!normal_scale(c->k_scale) || !normal_scale(c->v_scale)) return FL_ERR_INVALID_ARG;
  for (int i = 0; i < 5; ++i)
    if (c->reserved[i]) return FL_ERR_INVALID_ARG;
  if (c->format == FL_KV_E2M1) {
    if (!c->k_scales || !c->v_scales) return FL_ERR_INVALID_ARG;
  } else if (c->k_scales || c->v_scales || c->k_scale != 1.f || c->v_scale != 1.f) {
    return FL_ERR_INVALID_ARG;
  }
  if (c->d != 64 && c->d != 128) return FL_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->Hkv) * c->page_size > kMaxPageRows) return FL_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return FL_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return FL_ERR_ALIGNMENT;
  if (c->format == FL_KV_E2M1 && (!aligned(c->k_scales, 16) || !aligned(c->v_scales, 16))) return FL_ERR_ALIGNMENT;
  return FL_OK;
}

fl::PagedCache cache_params(const fl_kv_cache& c) {
  fl::PagedCache p{};
  p.k = c.k;
  p.v = c.v;
  p.ks = static_cast<uint8_t*>(c.k_scales);
  p.vs = static_cast<uint8_t*>(c.v_scales);
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.num_pages = c.num_pages;
  p.Hkv = c.Hkv;
  while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
  return p;
}

// (token, head) strides of a row tensor: multiples of eight elements, heads
// and tokens not overlapping within a row.
fl_status rows_check(const int64_t s[2], int d) {
  if (s[0] < d || s[1] < d) return FL_ERR_INVALID_ARG;
  return (s[0] % 8 || s[1] % 8) ? FL_ERR_ALIGNMENT : FL_OK;
}

fl_status append_check(const void* k, const void* v, const fl_kv_cache* cache, const fl_kv_append_desc* desc) {
  if (!k || !v || !desc) return FL_ERR_INVALID_ARG;
  const fl_status cs = cache_check(cache);
  if (cs != FL_OK) return cs;
  const fl_kv_append_desc& a = *desc;
  if (a.T < 1 || a.B < 1 || a.Hq < 0 || a.max_pages < 1 || a.reserved0) return FL_ERR_INVALID_ARG;
  if (!a.kv_len || !a.block_table || a.table_stride < a.max_pages) return FL_ERR_INVALID_ARG;
  if (!a.seq_offsets && a.T != a.B) return FL_ERR_INVALID_ARG;
  if (static_cast<int64_t>(a.max_pages) * cache->page_size > kMaxTokens) return FL_ERR_UNSUPPORTED;
  if (!a.rope_cos != !a.rope_sin) return FL_ERR_INVALID_ARG;
  if (a.rope_cos) {
    if (a.rope_positions < 1 || a.rope_dim < 1 || a.rope_dim > cache->d) return FL_ERR_INVALID_ARG;
    if (a.rope_dim % 16) return FL_ERR_UNSUPPORTED;
    if (a.rope_interleaved != 0 && a.rope_interleaved != 1) return FL_ERR_INVALID_ARG;
    if (!aligned(a.rope_cos, 16) || !aligned(a.rope_sin, 16)) return FL_ERR_ALIGNMENT;
  }
  const bool has_q = a.q != nullptr;
  if (has_q != (a.q_out != nullptr) || has_q != (a.Hq > 0)) return FL_ERR_INVALID_ARG;
  if (has_q && a.Hq % cache->Hkv) return FL_ERR_INVALID_ARG;
  if (!a.k_out != !a.v_out) return FL_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(a.q, 16) || !aligned(a.q_out, 16) || !aligned(a.k_out, 16) ||
      !aligned(a.v_out, 16) || !aligned(a.seq_offsets, 4) || !aligned(a.kv_len, 4) || !aligned(a.block_table, 4))
    return FL_ERR_ALIGNMENT;
  fl_status st = rows_check(a.k_strides, cache->d);
  if (st == FL_OK) st = rows_check(a.v_strides, cache->d);
  if (st == FL_OK && has_q) st = rows_check(a.q_strides, cache->d);
  if (st == FL_OK && has_q) st = rows_check(a.q_out_strides, cache->d);
  if (st == FL_OK && a.k_out) st = rows_check(a.k_out_strides, cache->d);
  if (st == FL_OK && a.k_out) st = rows_check(a.v_out_strides, cache->d);
  return st;
}

// (b, h, l, c) strides of q or out; all zero: contiguous [B, Hq, Lq, d].
fl_status row_strides(const int64_t s[4], int64_t H, int64_t L, int64_t d, int64_t* b, int64_t* h, int64_t* l) {
  if (s[0] == 0 && s[1] == 0 && s[2] == 0 && s[3] == 0) {
    *l = d;
    *h = L * d;
    *b = H * L * d;
    return FL_OK;
  }
  if (s[3] != 1 || s[0] <= 0 || s[1] <= 0 || s[2] <= 0) return FL_ERR_INVALID_ARG;
  *b = s[0];
  *h = s[1];
  *l = s[2];
  return (s[0] % 8 || s[1] % 8 || s[2] % 8) ? FL_ERR_ALIGNMENT : FL_OK;
}

fl_status decode_desc_check(const fl_kv_cache* cache, const fl_attn_desc* desc) {
  if (!desc) return FL_ERR_INVALID_ARG;
  const fl_status cs = cache_check(cache);
  if (cs != FL_OK) return cs;
  const fl_attn_desc& d = *desc;
  if (d.B < 1 || d.Hq < 1 || d.Hkv < 1 || d.Lq < 1 || d.Lk < 1 || d.Hq % d.Hkv != 0) return FL_ERR_INVALID_ARG;
  if (d.Hkv != cache->Hkv || d.d != cache->d || d.dv != cache->d || d.Lk % cache->page_size) return FL_ERR_INVALID_ARG;
  if (d.Lk > kMaxTokens) return FL_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(d.Hq / d.Hkv) * d.Lq > fl::kPagedMaxRows) return FL_ERR_UNSUPPORTED;
  if (!std::isfinite(d.scale)) return FL_ERR_INVALID_ARG;
  if (d.mask_kind < FL_MASK_NONE || d.mask_kind > FL_MASK_DOCUMENT) return FL_ERR_INVALID_ARG;
  if (d.mask_kind > FL_MASK_SLIDING_WINDOW) return FL_ERR_UNSUPPORTED;
  if (d.mask_kind == FL_MASK_SLIDING_WINDOW && d.window < 1) return FL_ERR_INVALID_ARG;
  if (d.sink < 0 || (d.sink && d.mask_kind != FL_MASK_SLIDING_WINDOW)) return FL_ERR_INVALID_ARG;
  if (d.score_mod < FL_SCORE_NONE || d.score_mod > FL_SCORE_SOFTCAP) return FL_ERR_INVALID_ARG;
  if (d.score_mod == FL_SCORE_ALIBI && !d.alibi_slopes) return FL_ERR_INVALID_ARG;
  if (d.score_mod == FL_SCORE_SOFTCAP && !(d.softcap > 0.f && std::isfinite(d.softcap))) return FL_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (d.k_strides[i] || d.v_strides[i]) return FL_ERR_UNSUPPORTED;
  // one merge block per row
  if (static_cast<int64_t>(d.B) * d.Hq * d.Lq > 0x7fffffff) return FL_ERR_UNSUPPORTED;
  return FL_OK;
}

// Workspace: the plan (2 + B int64), partial outputs and log-sum-exps of two
// pieces per CTA.
struct WorkspaceLayout {
  size_t opart, lpart, bytes;
};
WorkspaceLayout workspace_layout(const fl_attn_desc& d, int M, int grid) {
  WorkspaceLayout w;
  w.opart = ((2 + static_cast<size_t>(d.B)) * sizeof(int64_t) + 15) / 16 * 16;
  w.lpart = w.opart + static_cast<size_t>(grid) * 2 * M * d.d * sizeof(float);
  w.bytes = w.lpart + static_cast<size_t>(grid) * 2 * M * sizeof(float);
  return w;
}

}  // namespace

extern "C" {

int32_t fl_kv_cache_size(void) { return static_cast<int32_t>(sizeof(fl_kv_cache)); }

int32_t fl_kv_append_desc_size(void) { return static_cast<int32_t>(sizeof(fl_kv_append_desc)); }

fl_status fl_kv_append(const void* k, const void* v, const fl_kv_cache* cache, const fl_kv_append_desc* desc) {
  const fl_status chk = append_check(k, v, cache, desc);
  if (chk != FL_OK) return chk;
  const fl_kv_append_desc& a = *desc;
  fl::AppendParams p{};
  int sm_count = 0;
  const fl_status st = fl::device_info(&sm_count, &p.status);
  if (st != FL_OK) return st;
  p.c = cache_params(*cache);
  p.q = a.q; p.k = k; p.v = v;
  p.q_out = a.q_out; p.k_out = a.k_out; p.v_out = a.v_out;
  p.q_t = a.q_strides[0]; p.q_h = a.q_strides[1];
  p.k_t = a.k_strides[0]; p.k_h = a.k_strides[1];
  p.v_t = a.v_strides[0]; p.v_h = a.v_strides[1];
  p.qo_t = a.q_out_strides[0]; p.qo_h = a.q_out_strides[1];
  p.ko_t = a.k_out_strides[0]; p.ko_h = a.k_out_strides[1];
  p.vo_t = a.v_out_strides[0]; p.vo_h = a.v_out_strides[1];
  p.seq_offsets = a.seq_offsets; p.kv_len = a.kv_len;
  p.table = a.block_table; p.table_stride = a.table_stride;
  p.inv_k_scale = 1.0f / cache->k_scale;
  p.inv_v_scale = 1.0f / cache->v_scale;
  p.T = a.T; p.B = a.B; p.Hq = a.Hq; p.max_pages = a.max_pages;
  if (a.rope_cos) {
    p.cos = a.rope_cos; p.sin = a.rope_sin;
    p.rope_positions = a.rope_positions; p.rope_dim = a.rope_dim; p.interleaved = a.rope_interleaved;
  }
  return fl::launch_result("cache append launch",
                           fl::launch_kv_append(cache->format, cache->d, p, sm_count, static_cast<cudaStream_t>(a.stream)));
}

size_t fl_attn_paged_decode_workspace_size(const fl_attn_desc* desc, const fl_kv_cache* cache) {
  if (decode_desc_check(cache, desc) != FL_OK) return 0;
  int sm_count = 0;
  uint32_t* status = nullptr;
  if (fl::device_info(&sm_count, &status) != FL_OK) return 0;
  const int M = desc->Hq / desc->Hkv * desc->Lq;
  const int grid = fl::paged_resident(cache->format, cache->d, M, false) * sm_count;
  if (grid < 1) {
    fl::launch_result("paged decode occupancy", cudaErrorInvalidDeviceFunction);
    return 0;
  }
  return workspace_layout(*desc, M, grid).bytes;
}

fl_status fl_attn_paged_decode_fwd(const void* q, const fl_kv_cache* cache, const int32_t* kv_len,
                                   const int32_t* block_table, int64_t table_stride, void* out, float* lse,
                                   void* workspace, size_t workspace_bytes, const fl_attn_desc* desc) {
  if (!q || !out || !kv_len || !block_table) return FL_ERR_INVALID_ARG;
  const fl_status chk = decode_desc_check(cache, desc);
  if (chk != FL_OK) return chk;
  const fl_attn_desc& d = *desc;
  fl::PagedDecodeParams p{};
  p.max_pages = d.Lk / cache->page_size;
  if (table_stride < p.max_pages) return FL_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(kv_len, 4) || !aligned(block_table, 4) ||
      !aligned(d.alibi_slopes, 4))
    return FL_ERR_ALIGNMENT;
  fl_status st = row_strides(d.q_strides, d.Hq, d.Lq, d.d, &p.q_b, &p.q_h, &p.q_l);
  if (st == FL_OK) st = row_strides(d.o_strides, d.Hq, d.Lq, d.d, &p.o_b, &p.o_h, &p.o_l);
  if (st != FL_OK) return st;
  if (!workspace) return FL_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return FL_ERR_ALIGNMENT;
  int sm_count = 0;
  st = fl::device_info(&sm_count, &p.status);
  if (st != FL_OK) return st;
  p.G = d.Hq / d.Hkv;
  p.M = p.G * d.Lq;
  p.grid = fl::paged_resident(cache->format, cache->d, p.M, false) * sm_count;
  if (p.grid < 1) return fl::launch_result("paged decode occupancy", cudaErrorInvalidDeviceFunction);
  const WorkspaceLayout w = workspace_layout(d, p.M, p.grid);
  if (workspace_bytes < w.bytes) return FL_ERR_INVALID_ARG;
  p.c = cache_params(*cache);
  p.q = q; p.out = out; p.lse = lse;
  p.kv_len = kv_len; p.table = block_table; p.table_stride = table_stride;
  p.slopes = d.alibi_slopes;
  p.B = d.B; p.Hq = d.Hq; p.Lq = d.Lq;
  p.cap = d.Lk;
  const float scale = d.scale > 0.f ? d.scale : 1.0f / std::sqrt(static_cast<float>(d.d));
  p.scale_log2 = scale * static_cast<float>(kLog2e) * cache->k_scale;
  p.softcap = std::fmin(d.softcap, 1e38f) * static_cast<float>(kLog2e);  // finite in log2 units too
  p.score_mod = d.score_mod;
  p.causal = d.mask_kind != FL_MASK_NONE;
  if (d.mask_kind == FL_MASK_SLIDING_WINDOW) {
    p.window = d.window < kMaxTokens ? d.window : static_cast<int>(kMaxTokens);
    p.sink = d.sink < kMaxTokens ? d.sink : static_cast<int>(kMaxTokens);
  }
  // keys that one unit reads at most: the table's, or the window's and the sinks'
  int64_t keys = d.Lk;
  if (p.window) {
    const int64_t seen = static_cast<int64_t>(p.window) + d.Lq + p.sink + 64;  // whole tiles at three borders
    keys = seen < keys ? seen : keys;
  }
  const int resident = fl::paged_resident(cache->format, cache->d, p.M, true) * sm_count;
  if (resident < 1) return fl::launch_result("paged decode occupancy", cudaErrorInvalidDeviceFunction);
  p.cluster = fl::paged_cluster(keys, static_cast<int64_t>(d.B) * d.Hkv, resident);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.plan = reinterpret_cast<int64_t*>(ws);
  p.opart = reinterpret_cast<float*>(ws + w.opart);
  p.lpart = reinterpret_cast<float*>(ws + w.lpart);
  return fl::launch_result("paged decode launch", fl::launch_paged_decode(cache->format, cache->d, p,
                                                                         static_cast<cudaStream_t>(d.stream)));
}

}  // extern "C"
