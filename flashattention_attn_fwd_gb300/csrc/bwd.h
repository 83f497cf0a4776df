// Backward pass of the fused attention: parameters shared by the host
// launcher and the kernels (internal header).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#ifdef __CUDACC__
#include "ptx.cuh"
#endif

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
  // far more tiles than a window's.  The query tiles from far_begin(tile) on are
  // cut into far_chunks runs of far_len tiles, one CTA each; those CTAs and
  // the tile's own leave fp32 partial dV and dK, [B * Hkv * sink_tiles][1 +
  // far_chunks][(DV + D) / 4][128][4], summed in order by a last kernel.  0: no split.
  int sink, sink_tiles, far_chunks, far_len;
  int dot_rows;           // sinks: rows of every head whose D comes from the scores
};

// The split of the sink tiles' walks (see BwdParams), from sizes alone.
struct SinkSplit {
  int tiles, chunks, len;
};
// SMs that the split balances for: a tuning value, not a limit (the split is right
// for any device), and fixed because the workspace's size, which depends on it, can
// be asked for without a device.
constexpr int kTunedSms = 152;
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
  // A walk costs its tiles and, at its two ends, about one more (three where
  // blocks take one walk), and its partial sums, so runs are as long as balance
  // allows: half of an SM's share of all tiles (they start
  // first), and no shorter than a window tile's walk.
  const int near = far_begin(0, window);
  const int64_t steps = static_cast<int64_t>(B) * Hkv * ((Lk + 127) / 128 * static_cast<int64_t>(near) + static_cast<int64_t>(far) * s.tiles);
  const int64_t share = steps / (2 * kTunedSms);
  const int64_t most = share > near ? share : near;
  const int64_t want = (far + most - 1) / most;
  s.len = static_cast<int>((far + want - 1) / want);
  s.chunks = (far + s.len - 1) / s.len;
  return s;
}

// With sinks: the first rows of every head whose D comes from the scores
// (launch_bwd_dot); dO . O does for the others.  Where rows see few keys the
// rounding of O shows: relative error of dQ against 64 bits 2.4e-3 from the scores
// at any size; from O 4.6e-3 at 4 tokens, 3.0e-3 at 16, 2.7e-3 at windows of 8,
// 2.5e-3 at windows of 64 and 2.4e-3 at 256.  So rows that see at most 64 keys:
// all of them under a narrow window, else the first 64 of every sequence (a block
// of that kernel).  The scores of all rows cost 40 us beside 108 at B 4 H 16 L
// 2048 window 256, those of 64 rows a head 2 us there and 2.4 beside 14.4 at B 1 H 2
// L 600; up to 512 tokens all rows' cost no more.
constexpr int kDotRows = 64;
inline int score_rows(int window, int sink, int Lq) {
  return static_cast<int64_t>(window) + sink <= 64 || Lq <= 512 ? Lq : kDotRows;
}

#ifdef __CUDACC__
// Byte offset of 16-byte chunk c of row r in a shared tile of C bf16 channels (the
// kernels with warp-level products): chunks permuted so that eight rows of one
// chunk column meet all banks.
template <int C>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  const int x = C >= 64 ? r & 7 : (r >> 1) & 3;
  return static_cast<uint32_t>(r * C * 2 + ((c ^ x) << 4));
}

// Softcap's t = cap log2(e) tanh(s scale / cap) of N by 4 raw scores of every lane,
// in place, and 1 - tanh^2: the forward's polynomial where all of the warp's scores are
// in its range, else 1 - 2 d with d = 1 / (1 + e^(2 s scale / cap)), whose error is
// one of cap and not of t (with a cap far above the scores it would be all of t).
template <int N, bool SECH>
__device__ __forceinline__ void softcap_log2(const BwdParams& p, float (&s)[N][4], float (&sech2)[SECH ? N : 1][4]) {
  const float kcap = p.softcap * 1.4426950408889634f;
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) top = fmaxf(top, fabsf(s[i / 4][i % 4]));
  if (__all_sync(0xffffffffu, top <= p.sc_smax)) {
    const float ikcap = 1.0f / kcap;
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) {
      float& x = s[i / 4][i % 4];
      const float z = x * x;
      x *= fmaf(fmaf(fmaf(p.sc_q[3], z, p.sc_q[2]), z, p.sc_q[1]), z, p.sc_q[0]);
      if (SECH) {
        const float th = x * ikcap;
        sech2[SECH ? i / 4 : 0][i % 4] = fmaf(-th, th, 1.0f);
      }
    }
  } else {
    const float zmul = 2.0f * p.scale * 1.4426950408889634f / p.softcap;
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) {
      float& x = s[i / 4][i % 4];
      const float d = ptx::rcp(1.0f + ptx::ex2(x * zmul));
      x = fmaf(-2.0f * kcap, d, kcap);
      if (SECH) sech2[SECH ? i / 4 : 0][i % 4] = 4.0f * d * (1.0f - d);
    }
  }
}
#endif

// D, L2 and a zeroed dQ accumulator of the first p.dot_rows rows of every head, from
// the scores (sum P dP); (d, dv) as below.
cudaError_t launch_bwd_dot(int d, int dv, int score_mod, const BwdParams& p, cudaStream_t s);

// With sinks, sequences of at most this many tokens: dQ, dK and dV in one launch.
constexpr int kShortRows = 64;
cudaError_t launch_bwd_short(int d, int dv, int score_mod, const BwdParams& p, int sm_count, cudaStream_t s);

// (d, dv): (32, 32), (64, 64), (128, 128) or (64, 128)
cudaError_t launch_bwd(int d, int dv, int score_mod, const CUtensorMap* maps, const BwdParams& p, cudaStream_t s);

}  // namespace fl
