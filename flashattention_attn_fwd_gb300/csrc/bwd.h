// Backward pass of the fused attention: parameters shared by the host
// launcher and the kernels (internal header).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace fl {

struct BwdParams {
  const void* q;          // bf16 [B, Hq, Lq, D]
  const void* k;          // bf16 [B, Hkv, Lk, D]
  const void* v;          // bf16 [B, Hkv, Lk, DV]
  const void* out;        // bf16 [B, Hq, Lq, DV] forward output
  const void* dout;       // bf16 [B, Hq, Lq, DV] gradient of the output
  const float* lse;       // fp32 [B, Hq, Lq] forward log-sum-exp (natural log)
  void* dq;               // bf16 [B, Hq, Lq, D]
  void* dk;               // bf16 [B, Hkv, Lk, D]
  void* dv;               // bf16 [B, Hkv, Lk, DV]
  float* dq_acc;          // fp32 [B, Hq, Lq, D] workspace
  float* dvec;            // fp32 [B, Hq, Lq_pad] workspace: rowsum(dO * O)
  float* l2;              // fp32 [B, Hq, Lq_pad] workspace: LSE * log2(e)
  float* part;            // sinks: fp32 partial dV, dK (below)
  const float* slopes;    // ALiBi slopes [Hq]
  const int32_t* doc_offsets;
  uint32_t* status;
  uint64_t timeout_ns;
  int B, Hq, Hkv, Lq, Lk;
  int Lq_pad;             // Lq rounded up to 4 (16-byte rows of dvec and l2)
  int n_ktiles;           // ceil(Lk / 128)
  int64_t rows;           // B * Hq * Lq
  float scale, softcap;
  // softcap on the FMA pipe, as in the forward: cap*log2(e)*tanh(s*scale/cap)
  // = s * (q0 + q1 s^2 + q2 s^4 + q3 s^6) while |s| <= sc_smax
  float sc_q[4];
  float sc_smax;
  int mask_kind, doc_causal, window, prefix, num_docs;
  // the gradients are those of dout_scale * dout (1 for the plain backward;
  // -lambda for the second branch of differential attention), and with
  // dv_accumulate the kernel adds its dV to the bf16 values already in dv
  float dout_scale;
  int dv_accumulate;
  // Window with sinks: key tiles [0, sink_tiles) are seen by every later query,
  // far more tiles than a window's.  The query tiles from far0(tile) on are
  // cut into far_chunks runs of far_len tiles, one CTA each; those CTAs and
  // the tile's own leave fp32 partial dV and dK, [B * Hkv * sink_tiles][1 +
  // far_chunks][128][DV + D], summed in order by a last kernel.  0: no split.
  int sink, sink_tiles, far_chunks, far_len;
};

// The split of the sink tiles' walks (see BwdParams), from sizes alone.
struct SinkSplit {
  int tiles, chunks, len;
};
// First query tile past key tile jt's window.
#ifdef __CUDACC__
__host__ __device__
#endif
inline int far_begin(int jt, int window) { return (jt * 128 + 127 + (window < (1 << 30) ? window : 1 << 30) - 1) / 128 + 1; }
inline SinkSplit sink_split(int B, int Hkv, int Lq, int Lk, int window, int sink) {
  SinkSplit s{0, 0, 0};
  if (sink < 1) return s;
  const int nq = (Lq + 127) / 128;
  s.tiles = ((sink < Lk ? sink : Lk) + 127) / 128;
  const int far = nq - far_begin(0, window);
  if (far <= 0) return SinkSplit{0, 0, 0};  // every query is within the first tile's window
  // walks about as long as a window tile's, on no more CTAs than a few waves
  const int near = far_begin(0, window);
  int64_t want = (far + near - 1) / near;
  const int64_t most = (608 + static_cast<int64_t>(B) * Hkv * s.tiles - 1) / (static_cast<int64_t>(B) * Hkv * s.tiles);
  want = want < most ? want : most;
  s.len = static_cast<int>((far + want - 1) / want);
  s.chunks = (far + s.len - 1) / s.len;
  return s;
}

// D, L2 and a zeroed dQ accumulator with sinks (sum P dP from the scores; the
// plain backward's pre-kernel takes dO . O); (d, dv) as below.
cudaError_t launch_bwd_dot(int d, int dv, int score_mod, const BwdParams& p, cudaStream_t s);

// (d, dv): (32, 32), (64, 64), (128, 128) or (64, 128)
cudaError_t launch_bwd(int d, int dv, int score_mod, const CUtensorMap* maps, const BwdParams& p, cudaStream_t s);

}  // namespace fl
