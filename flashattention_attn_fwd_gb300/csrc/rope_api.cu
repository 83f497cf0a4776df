// C ABI of the rotary positions: argument checks, parameters and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "flattn.h"
#include "host.h"
#include "rope.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// (b, h, l) strides; all zero: contiguous [B, H, L, d]
fl_status strides(const int64_t s[3], int64_t H, int64_t L, int64_t d, int64_t* b, int64_t* h, int64_t* l) {
  if (s[0] == 0 && s[1] == 0 && s[2] == 0) {
    *l = d;
    *h = L * d;
    *b = H * L * d;
    return FL_OK;
  }
  if (s[0] <= 0 || s[1] <= 0 || s[2] <= 0) return FL_ERR_INVALID_ARG;
  *b = s[0];
  *h = s[1];
  *l = s[2];
  return (s[0] % 8 || s[1] % 8 || s[2] % 8) ? FL_ERR_ALIGNMENT : FL_OK;
}

fl_status rope_call(const char* what, const void* q, const void* k, void* q_out, void* k_out, const fl_rope_desc* desc,
                    float sign) {
  if (!q || !q_out || !desc || !k != !k_out) return FL_ERR_INVALID_ARG;
  const fl_rope_desc& d = *desc;
  if (d.B < 1 || d.L < 1 || d.Hq < 1 || d.Hk < 0 || (d.Hk > 0) != (k != nullptr)) return FL_ERR_INVALID_ARG;
  if (!d.rope_cos || !d.rope_sin || d.rope_positions < 1 || d.rope_dim < 1 || d.rope_dim > d.d) return FL_ERR_INVALID_ARG;
  const int32_t interleaved = d.rope_interleaved & ~(FL_ROPE_ZERO_Q | FL_ROPE_ZERO_K);
  if (interleaved != 0 && interleaved != 1) return FL_ERR_INVALID_ARG;
  if (d.positions ? d.positions_stride < 0 : d.L > d.rope_positions) return FL_ERR_INVALID_ARG;
  if (d.d != 32 && d.d != 64 && d.d != 128) return FL_ERR_UNSUPPORTED;
  if (d.rope_dim % 16) return FL_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(d.rope_cos, 16) ||
      !aligned(d.rope_sin, 16) || !aligned(d.positions, 4))
    return FL_ERR_ALIGNMENT;
  fl::RopeParams p{};
  auto rows = [&](fl::RopeRows& r, const void* x, void* y, int heads, const int64_t xs[3], const int64_t ys[3]) {
    r.x = x;
    r.y = y;
    r.heads = heads;
    const fl_status st = strides(xs, heads, d.L, d.d, &r.x_b, &r.x_h, &r.x_l);
    return st != FL_OK ? st : strides(ys, heads, d.L, d.d, &r.y_b, &r.y_h, &r.y_l);
  };
  fl_status st = rows(p.t[0], q, q_out, d.Hq, d.q_strides, d.q_out_strides);
  if (st == FL_OK && k) st = rows(p.t[1], k, k_out, d.Hk, d.k_strides, d.k_out_strides);
  if (st != FL_OK) return st;
  p.t[0].zero = (d.rope_interleaved & FL_ROPE_ZERO_Q) != 0;
  p.t[1].zero = (d.rope_interleaved & FL_ROPE_ZERO_K) != 0;
  int sm_count = 0;
  st = fl::device_info(&sm_count, &p.status);
  if (st != FL_OK) return st;
  p.cos = d.rope_cos;
  p.sin = d.rope_sin;
  p.positions = d.positions;
  p.pos_b = d.positions_stride;
  p.B = d.B;
  p.L = d.L;
  p.table_rows = d.rope_positions;
  p.rope_dim = d.rope_dim;
  p.interleaved = interleaved;
  p.sign = sign;
  return fl::launch_result(what, fl::launch_rope(d.d, p, sm_count, static_cast<cudaStream_t>(d.stream)));
}

}  // namespace

extern "C" {

int32_t fl_rope_desc_size(void) { return static_cast<int32_t>(sizeof(fl_rope_desc)); }

int32_t fl_rope_scaling_size(void) { return static_cast<int32_t>(sizeof(fl_rope_scaling)); }

fl_status fl_rope_fwd(const void* q, const void* k, void* q_out, void* k_out, const fl_rope_desc* desc) {
  return rope_call("rope launch", q, k, q_out, k_out, desc, 1.f);
}

fl_status fl_rope_bwd(const void* dq_out, const void* dk_out, void* dq, void* dk, const fl_rope_desc* desc) {
  return rope_call("rope backward launch", dq_out, dk_out, dq, dk, desc, -1.f);
}

fl_status fl_rope_tables(float* rope_cos, float* rope_sin, int32_t positions, int32_t rope_dim,
                         const fl_rope_scaling* scaling, void* stream) {
  if (!rope_cos || !rope_sin || !scaling || positions < 1 || rope_dim < 1) return FL_ERR_INVALID_ARG;
  const fl_rope_scaling& c = *scaling;
  if (!(c.base > 1.0) || !std::isfinite(c.base)) return FL_ERR_INVALID_ARG;
  if (c.kind < FL_ROPE_PLAIN || c.kind > FL_ROPE_BY_PARTS || c.reserved) return FL_ERR_INVALID_ARG;
  if (!(c.amplitude > 0.f) || !std::isfinite(c.amplitude)) return FL_ERR_INVALID_ARG;
  if (c.kind != FL_ROPE_PLAIN && !(c.factor >= 1.0 && std::isfinite(c.factor))) return FL_ERR_INVALID_ARG;
  if (c.kind == FL_ROPE_BY_PARTS &&
      (c.original < 1 || !(c.low_turns >= 0.0) || !(c.high_turns > c.low_turns) || !std::isfinite(c.high_turns)))
    return FL_ERR_INVALID_ARG;
  if (rope_dim % 16 || rope_dim > fl::kRopeMaxDim) return FL_ERR_UNSUPPORTED;
  if (!aligned(rope_cos, 16) || !aligned(rope_sin, 16)) return FL_ERR_ALIGNMENT;
  fl::RopeTableParams p{};
  p.cos = rope_cos;
  p.sin = rope_sin;
  p.positions = positions;
  p.half = rope_dim / 2;
  p.amplitude = c.amplitude;
  const double two_pi = 6.283185307179586476925;
  const double r = rope_dim;
  const double base = c.kind == FL_ROPE_NTK ? c.base * std::pow(c.factor, r / (r - 2.0)) : c.base;
  for (int i = 0; i < p.half; ++i) {
    double inv = std::pow(base, -2.0 * i / r);  // radians a position
    if (c.kind == FL_ROPE_LINEAR) {
      inv /= c.factor;
    } else if (c.kind == FL_ROPE_BY_PARTS) {
      double keep = (c.original * inv / two_pi - c.low_turns) / (c.high_turns - c.low_turns);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      inv *= keep + (1.0 - keep) / c.factor;
    }
    p.turn[i] = static_cast<uint64_t>(std::ldexp(inv / two_pi, 64));  // inv <= 1
  }
  int sm_count = 0;
  uint32_t* status = nullptr;
  const fl_status st = fl::device_info(&sm_count, &status);
  if (st != FL_OK) return st;
  return fl::launch_result("rope tables launch", fl::launch_rope_tables(p, sm_count, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
