// C ABI of the paged key/value cache: argument checks, parameters and
// launches of the append, the read, the decode attention and the attention of
// chunks of new tokens.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

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

// ---- chunks of new tokens

// tanh(y) ~= y (p0 + p1 y^2 + p2 y^4 + p3 y^6) for |y| <= kTanhRange: the
// forward's polynomial (csrc/fit_poly.py)
constexpr double kTanhRange = 0.5;
constexpr float kTanhP[4] = {0.999999464f, -0.333263218f, 0.13190335f, -0.0444031134f};
constexpr uint64_t kDefaultWaitNs = 2000ull * 1000ull * 1000ull;
constexpr int64_t kMaxRows = int64_t(1) << 30;  // tokens of a call: positions stay within 32 bits

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// 4-D bf16 map with boxes of 64 channels, box[1] x box[2] x box[3], 128-byte swizzle
// (strides of dimensions 1 to 3 in elements); reads outside are zeros.
bool encode_rows(CUtensorMap* m, const void* base, const uint64_t (&dims)[4], const int64_t (&strides)[3],
                 const uint32_t (&rows)[3]) {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(ptr);
  });
  if (!fn) return false;
  const cuuint64_t d[4] = {dims[0], dims[1], dims[2], dims[3]};
  const cuuint64_t s[3] = {static_cast<cuuint64_t>(strides[0]) * 2, static_cast<cuuint64_t>(strides[1]) * 2,
                           static_cast<cuuint64_t>(strides[2]) * 2};
  const cuuint32_t b[4] = {64u, rows[0], rows[1], rows[2]}, e[4] = {1u, 1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

fl_status prefill_desc_check(const fl_kv_cache* cache, const fl_attn_desc* desc) {
  if (!desc) return FL_ERR_INVALID_ARG;
  const fl_status cs = cache_check(cache);
  if (cs != FL_OK) return cs;
  const fl_attn_desc& d = *desc;
  if (d.B < 1 || d.Hq < 1 || d.Hkv < 1 || d.Lq < 1 || d.Lk < 1 || d.Hq % d.Hkv != 0) return FL_ERR_INVALID_ARG;
  if (d.Hkv != cache->Hkv || d.d != cache->d || d.dv != cache->d || d.Lk % cache->page_size) return FL_ERR_INVALID_ARG;
  if (d.Lk > kMaxTokens || d.Lq > kMaxRows || d.B > kMaxRows) return FL_ERR_UNSUPPORTED;
  if (d.Hq / d.Hkv > fl::kPrefillMaxGroup) return FL_ERR_UNSUPPORTED;
  // a bf16 pool's groups of 8 rows, one page more for what is outside, are counted in 31
  // bits (two terabytes of keys at d 64)
  if (cache->format == FL_KV_BF16 &&
      (static_cast<int64_t>(cache->num_pages) + 1) * (static_cast<int64_t>(cache->Hkv) * cache->page_size / 8) > 0x7fffffff)
    return FL_ERR_UNSUPPORTED;
  if (!std::isfinite(d.scale)) return FL_ERR_INVALID_ARG;
  if (d.mask_kind < FL_MASK_NONE || d.mask_kind > FL_MASK_DOCUMENT) return FL_ERR_INVALID_ARG;
  if (d.mask_kind > FL_MASK_SLIDING_WINDOW) return FL_ERR_UNSUPPORTED;
  if (d.mask_kind == FL_MASK_SLIDING_WINDOW && d.window < 1) return FL_ERR_INVALID_ARG;
  if (d.sink < 0 || (d.sink && d.mask_kind != FL_MASK_SLIDING_WINDOW)) return FL_ERR_INVALID_ARG;
  if (d.score_mod < FL_SCORE_NONE || d.score_mod > FL_SCORE_SOFTCAP) return FL_ERR_INVALID_ARG;
  if (d.score_mod == FL_SCORE_ALIBI && !d.alibi_slopes) return FL_ERR_INVALID_ARG;
  if (d.score_mod == FL_SCORE_SOFTCAP && !(d.softcap > 0.f && std::isfinite(d.softcap))) return FL_ERR_INVALID_ARG;
  if (d.fill & ~(FL_FILL_OUT | FL_FILL_LSE)) return FL_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (d.k_strides[i] || d.v_strides[i]) return FL_ERR_UNSUPPORTED;
  return FL_OK;
}

// (token, head) strides of the packed q or out; all zero: contiguous [T, Hq, d]
fl_status packed_strides(const int64_t s[4], int64_t H, int64_t d, int64_t* t, int64_t* h) {
  if (s[0] == 0 && s[1] == 0 && s[2] == 0 && s[3] == 0) {
    *h = d;
    *t = H * d;
    return FL_OK;
  }
  if (s[0] != 0 || s[3] != 1 || s[1] < d || s[2] < d) return FL_ERR_INVALID_ARG;
  *h = s[1];
  *t = s[2];
  return (s[1] % 8 || s[2] % 8) ? FL_ERR_ALIGNMENT : FL_OK;
}

// Workspace: a record for every block, two partial results of 256 rows and
// their log-sum-exps.
struct PrefillWorkspace {
  size_t opart, lpart, bytes;
};
PrefillWorkspace prefill_workspace(int d, int grid) {
  PrefillWorkspace w;
  const size_t rows = static_cast<size_t>(grid) * 4 * fl::kPrefillTile;
  w.opart = static_cast<size_t>(grid) * 8 * sizeof(int32_t);
  w.lpart = w.opart + rows * d * sizeof(float);
  w.bytes = w.lpart + rows * sizeof(float);
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

int32_t fl_kv_read_desc_size(void) { return static_cast<int32_t>(sizeof(fl_kv_read_desc)); }

fl_status fl_kv_read(const fl_kv_cache* cache, void* k_out, void* v_out, const fl_kv_read_desc* desc) {
  if (!k_out || !v_out || !desc) return FL_ERR_INVALID_ARG;
  const fl_status cs = cache_check(cache);
  if (cs != FL_OK) return cs;
  const fl_kv_read_desc& a = *desc;
  if (a.T < 1 || a.B < 1 || a.max_pages < 1 || a.reserved0) return FL_ERR_INVALID_ARG;
  if (!a.kv_len || !a.block_table || a.table_stride < a.max_pages) return FL_ERR_INVALID_ARG;
  if (!a.seq_offsets && a.T != a.B) return FL_ERR_INVALID_ARG;
  if (static_cast<int64_t>(a.max_pages) * cache->page_size > kMaxTokens) return FL_ERR_UNSUPPORTED;
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(a.seq_offsets, 4) || !aligned(a.kv_len, 4) ||
      !aligned(a.block_table, 4))
    return FL_ERR_ALIGNMENT;
  fl_status st = rows_check(a.k_out_strides, cache->d);
  if (st == FL_OK) st = rows_check(a.v_out_strides, cache->d);
  if (st != FL_OK) return st;
  fl::ReadParams p{};
  int sm_count = 0;
  st = fl::device_info(&sm_count, &p.status);
  if (st != FL_OK) return st;
  p.c = cache_params(*cache);
  p.k_out = k_out; p.v_out = v_out;
  p.ko_t = a.k_out_strides[0]; p.ko_h = a.k_out_strides[1];
  p.vo_t = a.v_out_strides[0]; p.vo_h = a.v_out_strides[1];
  p.seq_offsets = a.seq_offsets; p.kv_len = a.kv_len;
  p.table = a.block_table; p.table_stride = a.table_stride;
  p.T = a.T; p.B = a.B; p.max_pages = a.max_pages;
  return fl::launch_result("cache read launch",
                           fl::launch_kv_read(cache->format, cache->d, p, sm_count, static_cast<cudaStream_t>(a.stream)));
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

size_t fl_attn_paged_prefill_workspace_size(const fl_attn_desc* desc, const fl_kv_cache* cache) {
  if (prefill_desc_check(cache, desc) != FL_OK) return 0;
  int sm_count = 0;
  uint32_t* status = nullptr;
  if (fl::device_info(&sm_count, &status) != FL_OK) return 0;
  return prefill_workspace(desc->d, sm_count).bytes;
}

fl_status fl_attn_paged_prefill_fwd(const void* q, const fl_kv_cache* cache, const int32_t* seq_offsets,
                                    const int32_t* kv_len, const int32_t* block_table, int64_t table_stride, void* out,
                                    float* lse, void* workspace, size_t workspace_bytes, const fl_attn_desc* desc) {
  if (!q || !out || !kv_len || !block_table) return FL_ERR_INVALID_ARG;
  const fl_status chk = prefill_desc_check(cache, desc);
  if (chk != FL_OK) return chk;
  const fl_attn_desc& d = *desc;
  if (!seq_offsets && d.Lq != d.B) return FL_ERR_INVALID_ARG;
  fl::PrefillParams p{};
  p.max_pages = d.Lk / cache->page_size;
  if (table_stride < p.max_pages) return FL_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(seq_offsets, 4) || !aligned(kv_len, 4) ||
      !aligned(block_table, 4) || !aligned(d.alibi_slopes, 4))
    return FL_ERR_ALIGNMENT;
  fl_status st = packed_strides(d.q_strides, d.Hq, d.d, &p.q_t, &p.q_h);
  if (st == FL_OK) st = packed_strides(d.o_strides, d.Hq, d.d, &p.o_t, &p.o_h);
  if (st != FL_OK) return st;
  if (!workspace) return FL_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return FL_ERR_ALIGNMENT;
  int sm_count = 0;
  st = fl::device_info(&sm_count, &p.status);
  if (st != FL_OK) return st;
  p.grid = sm_count;
  const PrefillWorkspace w = prefill_workspace(d.d, p.grid);
  if (workspace_bytes < w.bytes) return FL_ERR_INVALID_ARG;
  p.c = cache_params(*cache);
  p.q = q; p.out = out; p.lse = lse;
  p.seq_offsets = seq_offsets; p.kv_len = kv_len;
  p.table = block_table; p.table_stride = table_stride;
  p.slopes = d.alibi_slopes;
  p.B = d.B; p.T = d.Lq; p.Hq = d.Hq; p.G = d.Hq / d.Hkv;
  p.RT = fl::kPrefillTile / p.G;
  while ((2 << p.div_s) < 2 * p.RT) ++p.div_s;
  p.div_m = static_cast<uint32_t>((uint64_t(1) << (32 + p.div_s)) / (2 * p.RT)) + 1u;
  p.cap = d.Lk;
  const float scale = (d.scale > 0.f ? d.scale : 1.0f / std::sqrt(static_cast<float>(d.d))) * cache->k_scale;
  p.scale_log2 = scale * static_cast<float>(kLog2e);
  if (d.score_mod == FL_SCORE_SOFTCAP) {
    const double cap = std::fmin(d.softcap, 1e38f);  // finite in log2 units too
    const double y = static_cast<double>(scale) / cap;
    double power = y * cap * kLog2e;
    for (int i = 0; i < 4; ++i, power *= y * y) p.sc_q[i] = static_cast<float>(kTanhP[i] * power);
    p.sc_smax = static_cast<float>(kTanhRange / y);
    p.softcap = static_cast<float>(cap * kLog2e);
    p.cap_arg = static_cast<float>(2.0 * kLog2e * y);
  }
  p.causal = d.mask_kind != FL_MASK_NONE;
  if (d.mask_kind == FL_MASK_SLIDING_WINDOW) {
    p.window = d.window < kMaxTokens ? d.window : static_cast<int>(kMaxTokens);
    p.sink = d.sink < kMaxTokens ? d.sink : static_cast<int>(kMaxTokens);
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.rec = reinterpret_cast<int32_t*>(ws);
  p.opart = reinterpret_cast<float*>(ws + w.opart);
  p.lpart = reinterpret_cast<float*>(ws + w.lpart);
  p.timeout_ns = d.wait_limit_ms ? static_cast<uint64_t>(d.wait_limit_ms) * 1000ull * 1000ull : kDefaultWaitNs;
  p.dbg_skip_tile = (d.debug_flags & FL_DEBUG_SKIP_KV_LOAD) ? d.debug_arg : -1;
  p.fill = seq_offsets ? d.fill & (FL_FILL_OUT | (lse ? FL_FILL_LSE : 0u)) : 0u;
  CUtensorMap maps[3] = {};
  if (cache->format == FL_KV_BF16) {
    const uint64_t D = d.d, G = p.G, Hkv = d.Hkv, page = cache->page_size;
    const uint64_t qd[4] = {D, G, Hkv, static_cast<uint64_t>(p.T)};
    const int64_t qs[3] = {p.q_h, p.q_h * p.G, p.q_t};
    const uint32_t qb[3] = {static_cast<uint32_t>(G), 1u, static_cast<uint32_t>(p.RT)};
    // the pool as groups of 8 rows: 64 channels, rows, halves of a row, groups
    const uint64_t groups = static_cast<uint64_t>(cache->num_pages) * Hkv * (page / 8);
    const uint64_t kd[4] = {64u, 8u, D / 64, groups};
    const int64_t ks[3] = {cache->d, 64, 8 * static_cast<int64_t>(cache->d)};
    const uint32_t kb[3] = {8u, static_cast<uint32_t>(D / 64),
                            static_cast<uint32_t>(page < fl::kPrefillBox ? page : fl::kPrefillBox) / 8u};
    if (!encode_rows(&maps[0], q, qd, qs, qb) || !encode_rows(&maps[1], cache->k, kd, ks, kb) ||
        !encode_rows(&maps[2], cache->v, kd, ks, kb))
      return fl::launch_result("paged prefill tensor map", cudaErrorInvalidValue);
  }
  const cudaStream_t s = static_cast<cudaStream_t>(d.stream);
  const bool bf16 = cache->format == FL_KV_BF16;
  const cudaError_t e = d.d == 64 ? (bf16 ? fl::launch_prefill_bf16_d64(d.score_mod, maps, p, s)
                                          : fl::launch_prefill_e2m1_d64(d.score_mod, maps, p, s))
                                  : (bf16 ? fl::launch_prefill_bf16_d128(d.score_mod, maps, p, s)
                                          : fl::launch_prefill_e2m1_d128(d.score_mod, maps, p, s));
  return fl::launch_result("paged prefill launch", e);
}

}  // extern "C"
