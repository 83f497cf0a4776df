// Decode-phase attention over a paged key/value cache in bf16 or 4 bits.
//
//   S = scale q K^T (+ score_mod, mask),  out = softmax(S) V
//
// for the few new rows of every sequence (G = Hq / Hkv heads of a group times
// Lq tokens share a key/value head: M = G * Lq rows), online softmax in 32
// bits.  Bound by reading the cache: per key and head 2 (d / 2 + d / 16)
// bytes in 4 bits, 4 d in bf16, against 4 d M operations.
//
// Work split.  With at most a few thousand keys to read per key/value head (a
// narrow table, or a window), a cluster of CTAs takes each (sequence, head) unit,
// cuts its tiles evenly and joins the results through distributed shared memory:
// one launch and no workspace traffic.  The choice is the host's, which knows the
// table's width and not the lengths; a table wider than its sequences costs 0.8 us
// at one sequence of 701 tokens (6.1 against 6.9), 2 at 16 (8.1, 9.8) and 4 at 64
// (12.6, 16.7), 8 heads of 64 in 4 bits.
// Beyond that lengths matter more: the tiles that some row sees, over all
// (sequence, key/value head) units, form one line that is cut into equal pieces,
// one per resident CTA: lengths may differ as they like and every CTA reads the
// same amount.  A unit inside one piece is finished by its CTA; a
// unit that pieces share leaves one normalised partial result and log-sum-exp
// per piece in the workspace, and paged_merge_kernel joins them with weights
// 2^(LSE_piece - LSE).  The cut depends on the lengths alone, so the result of
// a call is the same every time.
//
// Inner loop.  The CTA's four warps take the tiles of its piece in turn; with
// more than 16 rows, groups of two or four warps share a tile, each for its own
// rows.  A group copies its tiles with 16-byte cp.async into a ring of stages of
// its own (one barrier per tile), so that a few stages per group, well above
// the SM's share of bandwidth times latency, are always on the way.  Both
// products are warp-level m16n8k16 tiles with the keys' side as the 16-row
// operand, so that 8 query rows fill a tile:
//   S^T (16 keys x 8 rows)      = K (16 keys x 16 channels) Q^T
//   O^T (16 channels x 8 rows) += V^T (16 channels x 16 keys) P^T
// (tcgen05 could take the same turn, 128 keys or the channels on its M side, 8 to
// 64 rows on N, O in TMEM.  That is not built: up to 8 rows these tiles read a bf16
// cache at 0.76 to 1.0 of the copy rate; 16 to 64 rows pay for O in registers, up to
// 255 a thread and two CTAs an SM.)  The order of the
// channels inside S's contraction, of the channels among O's rows and of the
// keys inside a tile is free, and is chosen so that a lane's fragments are
// contiguous bytes of the cache: lane (g, t) = (lane / 4, lane % 4) takes a
// quarter of the channels of two keys of K and an eighth of the channels of four
// consecutive keys of V, with wide loads and no shuffles.  The two 4-bit codes
// of a byte are neighbouring channels of one key, which is a K fragment's pair
// as it stands; V's pairs are two keys of one channel, so the nibbles of two
// keys are interleaved first.
// 4-bit values times their block scale have at most six significant bits and
// are exact in fp16; the products run in fp16 with fp32 sums.  The query row
// is scaled to fp16's range by a power of two (undone in the score), P carries a
// factor 2^7 so that weights down to 2^-31 of the largest survive in fp16.  Over a
// bf16 cache P is rounded to bf16, because a product's operands have one type and
// V's exponents need bf16's: at most 2^-8 of a weight, as in the forward (2.3e-3
// of the output in all; 1.7e-3, its own rounding, over a 4-bit cache).
//
// Measured (4 bits unless said; a copy reads and writes 6.8 TB/s): one sequence
// of 701 tokens 6.1 us; 16 of 2048 to 8192, 8 heads of 64: 21 us; 12 of 9001 to
// 32768, 8 heads of 128: 57 us, 4.7 TB/s; 8 of 1500 to 16001 with four new
// tokens, 4 heads of 128 in bf16: 31 us, 3.1 TB/s; a window of 1024 with 4 sinks,
// 32 sequences: 11 us.  One new token over bf16, 8 heads: 16 of 2048 to 8192 31 us
// at d 64 and 53 at d 128 (5.1 and 6.0 TB/s), 12 of 9001 to 32768 at d 128 141 us,
// which is the copy rate.  Fixed: 1.3 us for the plan, 2 to the first tile, 4 for the
// merge and its launch.  In between the longest case runs at the issue rate of
// three CTAs an SM (0.56 of the slots; waits on fixed latencies and the ALU pipe
// lead), the short ones at the latency of a few tiles per warp.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <cstdint>
#include <type_traits>

#include "cvt4.cuh"
#include "host.h"
#include "paged.h"
#include "ptx.cuh"

namespace fl {
namespace {

constexpr int kPdWarps = 4;
constexpr int kPdThreads = 32 * kPdWarps;
constexpr float kPLog2e = 1.4426950408889634f;
constexpr float kPLn2 = 0.6931471805599453f;

// A tile is kSteps steps of 16 keys, which share its bookkeeping (four of a 4-bit
// head of 64 channels: 7.2 us against 6.1 at one sequence of 701 tokens, and no
// gain over long ones).
template <int FMT, int D>
constexpr int kSteps = FMT == KV_BF16 && D == 128 ? 1 : 2;

// Starting a unit (queries, pages, the first copies, the join at its end) costs
// a CTA about as long as this many tiles; the line counts them before each
// unit's own, so that a CTA that starts a second unit gets fewer tiles.  A balance
// found by measuring 0, 8, 16, 28 and 48: in 4 bits 23.0, 21.6, 21.0, 22.2, 23.5 us
// (16 sequences, d 64), 58.9, 58.1, 56.4, 57.7, 59.2 (12 long ones, d 128) and 37.4,
// 34.5, 33.8, 36.6, 40.9 (64 of 500 to 4096, d 64); 64 rows of d 128 44.5, 45.1, 45.3,
// 44.9, 50.0.  Over bf16, whose tiles take as long as their bytes, anything from 8
// to 28 is within 1 % (d 64 and 128, one token and four), and 0 is 1 to 9 % worse.
template <int FMT, int D>
constexpr int kLead = FMT == KV_BF16 ? 28 : 16;


__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// d += a b, m16n8k16, fp32 accumulators; fp16 or bf16 operands
template <int FMT>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (FMT == KV_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit values across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

// floats between the rows of O that the warps leave for their join
template <int D>
constexpr int kORow = D + 2;


// a / b of non-negative values, in 32 bits where both fit (0.1 us less)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// Tiles of KT keys of one head of sequence b: `count` of them (at least one),
// tile i at key KT * (i < sink ? i : i + skip).
struct SeqTiles {
  int n;        // keys in the cache
  int count, sink, skip;
};
template <int KT>
__device__ __forceinline__ SeqTiles seq_tiles(const PagedDecodeParams& p, int b) {
  SeqTiles s;
  s.n = min(max(__ldg(p.kv_len + b), 0), p.cap);
  int first = 0;
  s.sink = 0;
  if (p.window) {
    first = max(s.n - p.Lq - p.window + 1, 0) / KT;  // of the first row's window
    s.sink = min((p.sink + KT - 1) / KT, first);
  }
  s.skip = first - s.sink;
  s.count = max((s.n + KT - 1) / KT - s.skip, 1);
  return s;
}

// Ring of one warp group.  A stage holds the tile's K rows, its V rows and
// (4 bits) its scales: K's [key][d / 16], V's [d / 16][16 keys] per step.  The
// 16-byte chunks of a row are permuted within their 128-byte line (swz_k,
// swz_v of the key) so that the fragment loads meet no bank twice.
template <int FMT, int D, int RW>
struct Ring {
  static constexpr int HV = kSteps<FMT, D>;
  static constexpr int KB = FMT == KV_E2M1 ? D / 2 : 2 * D;      // bytes of one key's row
  static constexpr int ROWS = 16 * HV * KB;                      // bytes of K (or V) per stage
  static constexpr int SC = FMT == KV_E2M1 ? D : 0;              // bytes of K (or V) scales per step
  static constexpr int STAGE = 2 * ROWS + 2 * HV * SC;
  static constexpr int STAGES = RW * (FMT == KV_BF16 ? 2 : 3);
  static constexpr int BYTES = kPdWarps / RW * STAGES * STAGE;   // of the CTA's groups
};
template <int FMT, int D>
__device__ __forceinline__ int swz_k(int j) {
  return FMT == KV_BF16 ? 4 * (j & 1) : D == 128 ? 2 * ((j >> 2) & 3) : 4 * ((j >> 2) & 1);
}
__device__ __forceinline__ int swz_v(int j) { return 2 * ((j >> 2) & 3); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// CL: a cluster of p.cluster CTAs per unit; else pieces of the line.
template <int FMT, int D, int NT, int RW, bool CL>
__global__ void __launch_bounds__(kPdThreads) paged_decode_kernel(const __grid_constant__ PagedDecodeParams p) {
  constexpr int KS = D / 16;        // k-steps of S, and 16-channel row tiles of O
  constexpr int HV = kSteps<FMT, D>;
  constexpr int KT = 16 * HV;       // keys per tile
  constexpr int WR = 8 * NT;        // query rows per warp
  // weights carry 2^kLift in fp16 (see above)
  constexpr float kLift = FMT == KV_E2M1 ? 7.f : 0.f;
  using L = Ring<FMT, D, RW>;
  constexpr int S = L::STAGES;
  constexpr int GT = 32 * RW;       // threads of a group
  // rings of the groups; after a unit's tiles O [warp][WR][D], then m, l
  // [warp][WR][2] for the merge
  extern __shared__ __align__(128) float psm[];
  __shared__ int64_t scan_sm[kPdWarps];
  __shared__ int found_sm;
  __shared__ int64_t base_sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int64_t H = p.c.Hkv;        // units (key/value heads) per sequence
  constexpr int LEAD = kLead<FMT, D>;

  int b;                // current sequence
  int64_t base;         // line position of its first unit
  int64_t begin, end;   // this CTA's piece of the line
  SeqTiles sq;
  if constexpr (CL) {
    const int unit = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
    b = unit / p.c.Hkv;
    sq = seq_tiles<KT>(p, b);
    base = 0;
    begin = static_cast<int64_t>(sq.count) * rank / p.cluster;
    end = static_cast<int64_t>(sq.count) * (rank + 1) / p.cluster;
  } else {
    // ---- the plan: tiles per CTA, and this CTA's first sequence
    auto warp_incl = [&](int64_t v) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      return v;
    };
    // tiles and lead of sequence b0 + tid, and of the chunk's up to it
    int64_t c = 0, s = 0, chunk = 0;
    auto scan = [&](int b0) {
      c = b0 + tid < p.B ? LEAD + seq_tiles<KT>(p, b0 + tid).count : 0;
      s = warp_incl(c);
      if (lane == 31) scan_sm[warp] = s;
      __syncthreads();
      chunk = 0;
#pragma unroll
      for (int i = 0; i < kPdWarps; ++i) {
        if (i < warp) s += scan_sm[i];
        chunk += scan_sm[i];
      }
      __syncthreads();
    };
    int64_t total = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPdThreads) {
      scan(b0);
      total += chunk;
    }
    const int64_t all = total * H;
    const int64_t per = (quotient(all + gridDim.x - 1, gridDim.x) + kPdWarps - 1) / kPdWarps * kPdWarps;
    begin = blockIdx.x * per;
    end = begin + per < all ? begin + per : all;
    int64_t carry = 0;  // tiles of one head before the chunk's sequences
    for (int b0 = 0; b0 < p.B; b0 += kPdThreads) {
      if (p.B > kPdThreads) scan(b0);  // else the one chunk's is at hand
      const int64_t before = carry + s - c;
      if (blockIdx.x == 0 && b0 + tid < p.B) p.plan[2 + b0 + tid] = before;
      if (c > 0 && before * H <= begin && begin < (before + c) * H) {
        found_sm = b0 + tid;
        base_sm = before * H;
      }
      carry += chunk;
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
      p.plan[0] = per;
      p.plan[1] = all;
    }
    if (begin >= end) return;
    b = found_sm;
    base = base_sm;
    sq = seq_tiles<KT>(p, b);
  }

  const int shift = p.c.page_shift;
  const int page_mask = (1 << shift) - 1;
  const uint32_t page_bytes = static_cast<uint32_t>(p.c.Hkv << shift) * L::KB;  // of K, of V
  // warps by row group and by key group
  const int rw = warp % RW, kw = warp / RW;
  constexpr int n_kw = kPdWarps / RW;
  const int row0 = rw * WR;         // this warp's first row
  const int gt = rw * 32 + lane;    // thread of the group
  const uint32_t ring = ptx::smem_u32(psm) + kw * (S * L::STAGE);
  auto group_sync = [&]() {
    if (RW == 1) __syncwarp();
    else ptx::named_bar_sync(1 + kw, GT);
  };
  // fragments: K keys 4 (g / 2) + g % 2 and two further, V keys 4 t4 ..; byte
  // offsets within a stage's K and V, whose swizzle depends on the lane alone
  // (kx: 4 bits the two keys, bf16 even and odd 64-byte chunks of a row)
  constexpr int KB = L::KB;
  const int kkey = 4 * (g >> 1) + (g & 1);
  uint32_t kx[2], vx[4];
#pragma unroll
  for (int q = 0; q < 2; ++q)
    kx[q] = (FMT == KV_E2M1 ? (kkey + 2 * q) * KB + t4 * (D / 8) : kkey * KB + 16 * t4 + 64 * q) ^ (16 * swz_k<FMT, D>(kkey));
#pragma unroll
  for (int i = 0; i < 4; ++i) vx[i] = ((4 * t4 + i) * KB + g * (FMT == KV_E2M1 ? D / 16 : 16)) ^ (16 * swz_v(4 * t4));
  const uint32_t ksx = kkey * (D / 16) + t4 * (D / 64), vsx = D + 16 * (D == 128 ? g : g >> 1) + 4 * t4;

  // a rank without tiles still leaves its (empty) part for the cluster
  for (int64_t cur = begin; cur < end || (CL && cur == begin);) {
    // ---- the unit at `cur`
    int hkv, t0, t1;
    int64_t next;
    if constexpr (CL) {
      hkv = blockIdx.x / p.cluster % p.c.Hkv;
      t0 = static_cast<int>(begin);
      t1 = static_cast<int>(end);
      next = end;
    } else {
      while (cur >= base + (LEAD + sq.count) * H) {
        base += (LEAD + sq.count) * H;
        sq = seq_tiles<KT>(p, ++b);
      }
      const int64_t local = cur - base;
      const int len = LEAD + sq.count;
      hkv = static_cast<int>(quotient(local, len));
      const int at = static_cast<int>(local - static_cast<int64_t>(hkv) * len);
      const int64_t room = at + (end - cur);
      const int to = room < len ? static_cast<int>(room) : len;
      t0 = max(at - LEAD, 0);
      t1 = to - LEAD;
      next = cur + (to - at);
      if (t1 <= t0) {  // the piece ends within a unit's lead
        cur = next;
        continue;
      }
    }
    const bool whole = CL ? p.cluster == 1 : t0 == 0 && t1 == sq.count;
    const int slot = cur == begin ? 0 : 1;

    // ---- the ring: tile i of this group is t0 + kw + i * n_kw
    const int32_t* trow = p.table + b * p.table_stride;
    auto key_of = [&](int t) { return KT * (t < sq.sink ? t : t + sq.skip); };
    // page of a tile's step; -1: none (past the piece, the cache or the pool)
    auto page_of = [&](int t, int hf) {
      const int j = key_of(t) + 16 * hf;
      const int pg = t < t1 && j < sq.n ? __ldg(trow + (j >> shift)) : -1;
      return static_cast<unsigned>(pg) < static_cast<unsigned>(p.c.num_pages) ? pg : -1;
    };
    // does a tile's step hf > 0 start a page of its own?
    auto fresh = [&](int hf) { return ((16 * hf) & page_mask) == 0; };
    // A page is page_bytes (of K, of V); a head's run in it starts at kh, vh; the
    // scales' counts are those over KB / (D / 16).
    const uint8_t* kh = static_cast<const uint8_t*>(p.c.k) + (static_cast<int64_t>(hkv) << shift) * KB + 16 * gt;
    const uint8_t* vh = static_cast<const uint8_t*>(p.c.v) + (static_cast<int64_t>(hkv) << shift) * KB + 16 * gt;
    constexpr int SH = D / 8;          // scale chunks per step: K's, then V's
    const int sx = gt % SH;
    const bool sv = sx >= SH / 2;
    const uint8_t* sh = nullptr;
    if (FMT == KV_E2M1)
      sh = (sv ? p.c.vs + ((sx - SH / 2) << shift) : p.c.ks + 16 * sx) + (static_cast<int64_t>(hkv) << shift) * (D / 16);
    // Copies tile t (pages pg) into a stage; page 0 stands in for a missing
    // one, whose keys are masked.
    auto copy = [&](int t, const int (&pg)[HV], uint32_t st) {
      uint32_t pn[HV], off[HV];
      int64_t at[HV];
      pn[0] = max(pg[0], 0);
      off[0] = key_of(t) & page_mask;
      at[0] = static_cast<int64_t>(static_cast<uint64_t>(pn[0]) * page_bytes + off[0] * KB);
#pragma unroll
      for (int hf = 1; hf < HV; ++hf) {
        pn[hf] = pn[hf - 1];
        off[hf] = off[hf - 1] + 16;
        at[hf] = at[hf - 1] + 16 * KB;
        if (fresh(hf)) {
          pn[hf] = max(pg[hf], 0);
          off[hf] = 0;
          at[hf] = static_cast<int64_t>(static_cast<uint64_t>(pn[hf]) * page_bytes);
        }
      }
      constexpr int CH = KB;           // chunks of one step's K
      constexpr int N = HV * CH;
#pragma unroll
      for (int i = 0; i < (N + GT - 1) / GT; ++i) {
        const int c = gt + GT * i;
        if (N % GT == 0 || c < N) {
          int64_t a;
          if constexpr (CH % GT == 0) {
            a = at[GT * i / CH] + 16 * (GT * i % CH);
          } else {  // a group's round covers several steps
            a = at[0] + 16 * GT * i;
#pragma unroll
            for (int hf = 1; hf < HV; ++hf)
              if (c >= hf * CH) a = at[hf] + 16 * (GT * i - hf * CH);
          }
          const int j = c / (KB / 16);
          cp_async16(st + 16 * (c ^ swz_k<FMT, D>(j)), kh + a);
          cp_async16(st + L::ROWS + 16 * (c ^ swz_v(j)), vh + a);
        }
      }
      if constexpr (FMT == KV_E2M1) {
        static_assert(HV * SH <= 32, "a scale chunk per lane");
        if (gt < HV * SH) {
          uint32_t pp = pn[0], oo = off[0];
#pragma unroll
          for (int hf = 1; hf < HV; ++hf)
            if (gt >= hf * SH) pp = pn[hf], oo = off[hf];
          cp_async16(st + 2 * L::ROWS + 16 * gt,
                     sh + static_cast<int64_t>(static_cast<uint64_t>(pp) * (page_bytes / (KB / (D / 16))) + oo * (sv ? 1 : D / 16)));
        }
      }
    };
    const int n_tiles = (t1 - t0 - kw + n_kw - 1) / n_kw;  // of this group (0 or less: none)
    // pages of the next tile to copy, and which pages of the tiles under way
    // exist: HV bits a tile, the current tile's lowest
    int pg[HV];
    using Bits = std::conditional_t<(HV * S > 32), uint64_t, uint32_t>;
    static_assert(HV * S <= 64, "a bit per step under way");
    Bits have = 0;
    auto fetch = [&](int i) {
      pg[0] = page_of(t0 + kw + i * n_kw, 0);
#pragma unroll
      for (int hf = 1; hf < HV; ++hf) pg[hf] = fresh(hf) ? page_of(t0 + kw + i * n_kw, hf) : pg[hf - 1];
    };
    auto issue = [&](int i, int ahead, uint32_t st, const int (&page)[HV]) {  // tile i into stage st
      if (i < n_tiles) {
        copy(t0 + kw + i * n_kw, page, st);
#pragma unroll
        for (int hf = 0; hf < HV; ++hf) have |= static_cast<Bits>(page[hf] >= 0) << (HV * ahead + hf);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // ---- queries: row g of every 8-row tile, channels in the order of K's
    // fragments; fp16 rows scaled to magnitude [1, 2) by a power of two
    uint32_t qf[NT][KS][2];
    float sc[NT][2];   // factor of S (log2 units) of rows 2 t4, 2 t4 + 1
    int pos[NT][2];    // their positions
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rr = row0 + 8 * nt + g;
      const bool rv = rr < p.M;
      const int hq = hkv * p.G + (rv ? rr : 0) / p.Lq, i = (rv ? rr : 0) % p.Lq;
      const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(p.q) + b * p.q_b + hq * p.q_h + i * p.q_l;
      // channels: bf16 32 j + 8 t4 .., 4-bit t4 d / 4 + 8 j ..
#pragma unroll
      for (int j = 0; j < KS / 2; ++j) {
        const uint4 w = rv ? __ldg(reinterpret_cast<const uint4*>(qr + (FMT == KV_E2M1 ? t4 * (D / 4) + 8 * j : 32 * j + 8 * t4)))
                           : make_uint4(0u, 0u, 0u, 0u);
        qf[nt][2 * j][0] = w.x; qf[nt][2 * j][1] = w.y;
        qf[nt][2 * j + 1][0] = w.z; qf[nt][2 * j + 1][1] = w.w;
      }
    }
    // the first tiles' pages all at once, then their copies (a page after the
    // copy before it costs a table read's latency each: 0.7 us)
    int first[S - 1][HV];
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      fetch(i);
#pragma unroll
      for (int hf = 0; hf < HV; ++hf) first[i][hf] = pg[hf];
    }
    fetch(S - 1);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(i, i, ring + i * L::STAGE, first[i]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float undo = 1.f;
      if (FMT == KV_E2M1) {
        float a = 0.f;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            a = fmaxf(a, fmaxf(fabsf(__uint_as_float(qf[nt][kk][e] << 16)), fabsf(__uint_as_float(qf[nt][kk][e] & 0xffff0000u))));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const uint32_t ex = min(max(__float_as_uint(a) >> 23, 1u), 253u);
        const float f = __uint_as_float((254u - ex) << 23);  // 2^(127 - ex)
        undo = __uint_as_float(ex << 23);
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qf[nt][kk][e] = pack_f16(__uint_as_float(qf[nt][kk][e] << 16) * f, __uint_as_float(qf[nt][kk][e] & 0xffff0000u) * f);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sc[nt][e] = p.scale_log2 * __shfl_sync(0xffffffffu, undo, 4 * (2 * t4 + e));
        const int rc = row0 + 8 * nt + 2 * t4 + e;
        pos[nt][e] = sq.n - p.Lq + (rc < p.M ? rc % p.Lq : 0);
      }
    }
    const int pos_lo = sq.n - p.Lq, pos_hi = sq.n - 1;
    // first keys of tiles that every row sees whole: at most full_hi, and from
    // full_lo on or within the sinks
    const int full_hi = (p.causal ? pos_lo + 1 : sq.n) - KT;
    const int full_lo = p.window ? pos_hi - p.window + 1 : 0;
    const int full_sink = p.window ? p.sink - KT : -1;

    // online softmax: reference maximum m, the offset of the exponent
    // (2^kLift in fp16) and the bound beyond which m moves
    float o[NT][KS][4], m[NT][2], l[NT][2], off[NT][2], bound[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = bound[nt][e] = -CUDART_INF_F;
        l[nt][e] = off[nt][e] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
    }

    const bool plain = p.score_mod == 0;
    // The reference maximum moves only when a score exceeds it by more than 2^8
    // (O rescaled then); m0, m1: the lane's largest scores of its two rows.
    auto raise = [&](int nt, float m0, float m1) {
      float mx[2] = {m0, m1};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], d));
        const float mn = fmaxf(m[nt][e], mx[e]);
        if (mn != -CUDART_INF_F) {
          const float alpha = ptx::ex2(m[nt][e] - mn);
          m[nt][e] = mn;
          off[nt][e] = kLift - mn;
          bound[nt][e] = mn + 8.f;
          l[nt][e] *= alpha;
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            o[nt][mt][e] *= alpha;
            o[nt][mt][2 + e] *= alpha;
          }
        }
      }
    };
    uint32_t stage = 0, ahead = S - 1;  // ring positions of tile i and tile i + S - 1
    for (int i = 0; i < n_tiles; ++i) {
      cp_async_wait<S - 2>();
      group_sync();  // tile i is here, and its predecessor's stage is free
      issue(i + S - 1, S - 1, ring + ahead * L::STAGE, pg);
      fetch(i + S);
      const uint32_t st = ring + stage * L::STAGE;
      const int key0 = key_of(t0 + kw + i * n_kw);
      const uint32_t got = static_cast<uint32_t>(have) & ((1u << HV) - 1);
      have >>= HV;
      const bool full = got == (1u << HV) - 1 && key0 <= full_hi && (key0 >= full_lo || key0 <= full_sink);
      // ---- S^T = K Q^T
      float s[HV][NT][4];
#pragma unroll
      for (int hf = 0; hf < HV; ++hf)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[hf][nt][0] = s[hf][nt][1] = s[hf][nt][2] = s[hf][nt][3] = 0.f;
#pragma unroll
      for (int hf = 0; hf < HV; ++hf) {
        const uint32_t kt = st + hf * 16 * KB;
        if constexpr (FMT == KV_E2M1) {
          uint32_t ksc[2][2];  // [key][block of the lane's channels] fp16 pairs
          uint32_t kw4[2][D / 32];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t sa = st + 2 * L::ROWS + hf * 2 * D + ksx + 2 * q * (D / 16);
            const uint32_t h2 = cvt4::from_e4m3x2(D == 128 ? lds16(sa) : lds8(sa));
            ksc[q][0] = __byte_perm(h2, 0u, 0x1010);
            ksc[q][1] = D == 128 ? __byte_perm(h2, 0u, 0x3232) : ksc[q][0];
            if constexpr (D == 128) {
              const uint4 w = lds128(kt + kx[q]);
              kw4[q][0] = w.x; kw4[q][1] = w.y; kw4[q][2] = w.z; kw4[q][3] = w.w;
            } else {
              const uint2 w = lds64(kt + kx[q]);
              kw4[q][0] = w.x; kw4[q][1] = w.y;
            }
          }
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            uint32_t ha[4], hb[4];
            cvt4::from_e2m1x8(kw4[0][w], ha);
            cvt4::from_e2m1x8(kw4[1][w], hb);
            const int bl = D == 128 ? w >> 1 : 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              ha[e] = cvt4::hmul2(ha[e], ksc[0][bl]);
              hb[e] = cvt4::hmul2(hb[e], ksc[1][bl]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a[4] = {ha[2 * h], hb[2 * h], ha[2 * h + 1], hb[2 * h + 1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<FMT>(s[hf][nt], a, qf[nt][2 * w + h][0], qf[nt][2 * w + h][1]);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint4 ka = lds128(kt + kx[j & 1] + 128 * (j >> 1));
            const uint4 kb = lds128(kt + kx[j & 1] + 128 * (j >> 1) + 2 * KB);
            const uint32_t a0[4] = {ka.x, kb.x, ka.y, kb.y};
            const uint32_t a1[4] = {ka.z, kb.z, ka.w, kb.w};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816<FMT>(s[hf][nt], a0, qf[nt][2 * j][0], qf[nt][2 * j][1]);
              mma16816<FMT>(s[hf][nt], a1, qf[nt][2 * j + 1][0], qf[nt][2 * j + 1][1]);
            }
          }
        }
      }
      // ---- scores (log2 units) of key kkey (e < 2) and kkey + 2, rows 2 t4, +1
      uint32_t pb[HV][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[HV][4];
        if (NT == 1 && plain && full) {
          // the maximum of the raw scores against the bound in their units, then
          // scale and offset in one packed step
          float mx[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
            for (int hf = 1; hf < HV; ++hf) mx[e] = ptx::max3(mx[e], s[hf][nt][e], s[hf][nt][2 + e]);
          }
          if (__any_sync(0xffffffffu, mx[0] * sc[nt][0] > bound[nt][0] || mx[1] * sc[nt][1] > bound[nt][1]))
            raise(nt, mx[0] * sc[nt][0], mx[1] * sc[nt][1]);
          const float2 sc2 = make_float2(sc[nt][0], sc[nt][1]), off2 = make_float2(off[nt][0], off[nt][1]);
#pragma unroll
          for (int hf = 0; hf < HV; ++hf)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const float2 v = ptx::fma2(make_float2(s[hf][nt][e], s[hf][nt][e + 1]), sc2, off2);
              x[hf][e] = v.x;
              x[hf][e + 1] = v.y;
            }
        } else {
#pragma unroll
          for (int hf = 0; hf < HV; ++hf)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[hf][e] = s[hf][nt][e] * sc[nt][e & 1];
          if (p.score_mod != 0) {
            const int rc = row0 + 8 * nt + 2 * t4;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float slope = p.score_mod == 1 && rc + (e & 1) < p.M
                                      ? __ldg(p.slopes + hkv * p.G + (rc + (e & 1)) / p.Lq) * kPLog2e : 0.f;
#pragma unroll
              for (int hf = 0; hf < HV; ++hf) {
                if (p.score_mod == 2) x[hf][e] = p.softcap * tanhf(x[hf][e] / p.softcap);
                else x[hf][e] = fmaf(slope, static_cast<float>(key0 + 16 * hf + kkey + (e & 2) - pos[nt][e & 1]), x[hf][e]);
              }
            }
          }
          if (!full) {
#pragma unroll
            for (int hf = 0; hf < HV; ++hf) {
              const bool pok = (got >> hf) & 1u;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int j = key0 + 16 * hf + kkey + (e & 2), ps = pos[nt][e & 1];
                const bool vis = pok && j < sq.n && (!p.causal || j <= ps) && (!p.window || j > ps - p.window || j < p.sink);
                x[hf][e] = vis ? x[hf][e] : -CUDART_INF_F;
              }
            }
          }
          float mx[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(x[0][e], x[0][2 + e]);
#pragma unroll
            for (int hf = 1; hf < HV; ++hf) mx[e] = ptx::max3(mx[e], x[hf][e], x[hf][2 + e]);
          }
          if (__any_sync(0xffffffffu, mx[0] > bound[nt][0] || mx[1] > bound[nt][1])) raise(nt, mx[0], mx[1]);
#pragma unroll
          for (int hf = 0; hf < HV; ++hf)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[hf][e] += off[nt][e & 1];
        }
#pragma unroll
        for (int hf = 0; hf < HV; ++hf) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[hf][e] = ptx::ex2(x[hf][e]);
            l[nt][e & 1] += x[hf][e];
          }
          if (FMT == KV_E2M1) {
            pb[hf][nt][0] = transpose8(pack_f16(x[hf][0], x[hf][1]));
            pb[hf][nt][1] = transpose8(pack_f16(x[hf][2], x[hf][3]));
          } else {
            pb[hf][nt][0] = transpose8(ptx::pack_bf16x2(x[hf][0], x[hf][1]));
            pb[hf][nt][1] = transpose8(ptx::pack_bf16x2(x[hf][2], x[hf][3]));
          }
        }
      }
      // keys that no row sees may hold anything: their V must not reach the
      // product (0 * NaN)
      uint32_t drop = 0;  // of V keys 4 t4 .. of each half, one bit each
      if (!full) {
#pragma unroll
        for (int hf = 0; hf < HV; ++hf) {
          const bool pok = (got >> hf) & 1u;
          const int h0 = key0 + 16 * hf;
          const bool seen = h0 < sq.n && (!p.window || h0 + 15 > pos_lo - p.window || h0 < p.sink);
          if (!pok && seen && lane == 0) atomicOr(p.status, 2u);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = h0 + 4 * t4 + i;
            if (!pok || j >= sq.n || (p.window && j <= pos_lo - p.window && j >= p.sink)) drop |= 1u << (4 * hf + i);
          }
        }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int hf = 0; hf < HV; ++hf) {
        const uint32_t vt = st + L::ROWS + hf * 16 * KB;
        if constexpr (FMT == KV_E2M1) {
          uint32_t vs = lds32(st + 2 * L::ROWS + hf * 2 * D + vsx);
          if (drop) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((drop >> (4 * hf + i)) & 1u) vs &= ~(0xffu << (8 * i));
          }
          const uint32_t s01 = cvt4::from_e4m3x2(vs & 0xffffu), s23 = cvt4::from_e4m3x2(vs >> 16);
          uint32_t vw[4][D / 64];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (D == 128) {
              const uint2 w = lds64(vt + vx[i]);
              vw[i][0] = w.x; vw[i][1] = w.y;
            } else {
              vw[i][0] = lds32(vt + vx[i]);
            }
          }
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            // nibble pairs (key 0, key 1) of even and of odd channels
            const uint32_t v0 = vw[0][w], v1 = vw[1][w], v2 = vw[2][w], v3 = vw[3][w];
            uint32_t e01[4], o01[4], e23[4], o23[4];
            cvt4::from_e2m1x8((v0 & 0x0f0f0f0fu) | ((v1 << 4) & 0xf0f0f0f0u), e01);
            cvt4::from_e2m1x8(((v0 >> 4) & 0x0f0f0f0fu) | (v1 & 0xf0f0f0f0u), o01);
            cvt4::from_e2m1x8((v2 & 0x0f0f0f0fu) | ((v3 << 4) & 0xf0f0f0f0u), e23);
            cvt4::from_e2m1x8(((v2 >> 4) & 0x0f0f0f0fu) | (v3 & 0xf0f0f0f0u), o23);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a[4] = {cvt4::hmul2(e01[i], s01), cvt4::hmul2(o01[i], s01), cvt4::hmul2(e23[i], s23),
                                     cvt4::hmul2(o23[i], s23)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<FMT>(o[nt][4 * w + i], a, pb[hf][nt][0], pb[hf][nt][1]);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            uint4 vv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              vv[i] = lds128(vt + vx[i] + 128 * j);
              if ((drop >> (4 * hf + i)) & 1u) vv[i] = make_uint4(0u, 0u, 0u, 0u);
            }
            const uint32_t v0[4] = {vv[0].x, vv[0].y, vv[0].z, vv[0].w}, v1[4] = {vv[1].x, vv[1].y, vv[1].z, vv[1].w};
            const uint32_t v2[4] = {vv[2].x, vv[2].y, vv[2].z, vv[2].w}, v3[4] = {vv[3].x, vv[3].y, vv[3].z, vv[3].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a[4] = {__byte_perm(v0[i], v1[i], 0x5410), __byte_perm(v0[i], v1[i], 0x7632),
                                     __byte_perm(v2[i], v3[i], 0x5410), __byte_perm(v2[i], v3[i], 0x7632)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<FMT>(o[nt][4 * j + i], a, pb[hf][nt][0], pb[hf][nt][1]);
            }
          }
        }
      }
      stage = stage + 1 == S ? 0 : stage + 1;
      ahead = ahead + 1 == S ? 0 : ahead + 1;
    }

    if (!CL && next >= end) ptx::launch_dependents();  // the merge may be set up
    // ---- the warps' states meet: weights 2^(m_w - m), found once a row.  Rows of
    // O lie kORow apart, which spreads a warp's stores over the banks.
    constexpr int OW = kORow<D>;
    float* msm = psm + kPdWarps * WR * OW;
    cp_async_wait<0>();
    __syncthreads();  // the rings are idle: their memory takes the states
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[nt][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (g == 0) {
          msm[(warp * WR + 8 * nt + 2 * t4 + e) * 2] = m[nt][e];
          msm[(warp * WR + 8 * nt + 2 * t4 + e) * 2 + 1] = v;
        }
        // O's channel of row tile mt, half hf, lane group g
        float* od = psm + (warp * WR + 8 * nt + 2 * t4 + e) * OW;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          const int c = FMT == KV_E2M1 ? g * (D / 8) + 2 * mt : 64 * (mt >> 2) + 8 * g + 2 * (mt & 3);
          *reinterpret_cast<float2*>(od + c) = make_float2(o[nt][mt][e], o[nt][mt][2 + e]);
        }
      }
    }
    __syncthreads();
    constexpr int CP = D / 2;
    float* part = msm + kPdWarps * WR * 2;  // CL: O [M][D], then log-sum-exp [M]
    const int64_t piece = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * p.M;
    static_assert(kPagedMaxRows <= kPdThreads, "a thread per row");
    if (tid < p.M) {
      // row rr belongs to row warp rr / WR of every group
      const int rr = tid, w0 = rr / WR, rl = rr % WR;
      float mr = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < n_kw; ++i) mr = fmaxf(mr, msm[((w0 + i * RW) * WR + rl) * 2]);
      const float ms = mr == -CUDART_INF_F ? 0.f : mr;
      float ls = 0.f;
#pragma unroll
      for (int i = 0; i < n_kw; ++i) {
        float* st = msm + ((w0 + i * RW) * WR + rl) * 2;
        const float wt = st[0] == -CUDART_INF_F ? 0.f : ptx::ex2(st[0] - ms);
        ls = fmaf(wt, st[1], ls);
        st[0] = wt;
      }
      msm[(w0 * WR + rl) * 2 + 1] = ls == 0.f ? 0.f : p.c.v_scale / ls;
      const float lse2 = ls == 0.f ? -CUDART_INF_F : ms - kLift + __log2f(ls);
      if (whole) {
        if (p.lse) p.lse[(static_cast<int64_t>(b) * p.Hq + hkv * p.G + rr / p.Lq) * p.Lq + rr % p.Lq] = lse2 * kPLn2;
      } else if (CL) {
        part[p.M * D + rr] = lse2;
      } else {
        p.lpart[piece + rr] = lse2;
      }
    }
    __syncthreads();
    for (int e = tid; e < p.M * CP; e += kPdThreads) {
      const int rr = e / CP, c2 = e % CP;
      const int w0 = rr / WR, rl = rr % WR;
      float2 ov = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < n_kw; ++i) {
        const int at = (w0 + i * RW) * WR + rl;
        const float wt = msm[at * 2];
        const float2 ow = *reinterpret_cast<const float2*>(psm + at * OW + 2 * c2);
        ov = make_float2(fmaf(wt, ow.x, ov.x), fmaf(wt, ow.y, ov.y));
      }
      const float inv = msm[(w0 * WR + rl) * 2 + 1];
      ov = make_float2(ov.x * inv, ov.y * inv);
      if (whole) {
        const int hq = hkv * p.G + rr / p.Lq, i = rr % p.Lq;
        __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) + b * p.o_b + hq * p.o_h + i * p.o_l;
        reinterpret_cast<__nv_bfloat162*>(orow)[c2] = __floats2bfloat162_rn(ov.x, ov.y);
      } else if (CL) {
        *reinterpret_cast<float2*>(part + rr * D + 2 * c2) = ov;
      } else {
        reinterpret_cast<float2*>(p.opart)[(piece + rr) * CP + c2] = ov;
      }
    }
    if (CL && p.cluster > 1) {
      // ---- the cluster's parts meet: every CTA joins a share of the outputs
      ptx::cluster_barrier();
      const uint32_t pa = ptx::smem_u32(part);
      const int rank = blockIdx.x % p.cluster;
      for (int e = rank + p.cluster * tid; e < p.M * CP; e += p.cluster * kPdThreads) {
        const int rr = e / CP, c2 = e % CP;
        float lse[kClusterMax], Lm = -CUDART_INF_F;
        float2 ow[kClusterMax];
#pragma unroll
        for (int c = 0; c < kClusterMax; ++c) {
          if (c < p.cluster) {
            lse[c] = ptx::ld_cluster(pa + (p.M * D + rr) * 4, c);
            ow[c] = make_float2(ptx::ld_cluster(pa + (rr * D + 2 * c2) * 4, c), ptx::ld_cluster(pa + (rr * D + 2 * c2) * 4 + 4, c));
          }
        }
#pragma unroll
        for (int c = 0; c < kClusterMax; ++c)
          if (c < p.cluster) Lm = fmaxf(Lm, lse[c]);
        const float Ls = Lm == -CUDART_INF_F ? 0.f : Lm;
        float tot = 0.f;
        float2 ov = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kClusterMax; ++c) {
          if (c < p.cluster) {
            const float w = ptx::ex2(lse[c] - Ls);
            tot += w;
            ov = make_float2(fmaf(w, ow[c].x, ov.x), fmaf(w, ow[c].y, ov.y));
          }
        }
        const float inv = tot == 0.f ? 0.f : 1.f / tot;
        const int hq = hkv * p.G + rr / p.Lq, i = rr % p.Lq;
        __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) + b * p.o_b + hq * p.o_h + i * p.o_l;
        reinterpret_cast<__nv_bfloat162*>(orow)[c2] = __floats2bfloat162_rn(ov.x * inv, ov.y * inv);
        if (c2 == 0 && p.lse)
          p.lse[(static_cast<int64_t>(b) * p.Hq + hq) * p.Lq + i] = tot == 0.f ? -CUDART_INF_F : (Ls + __log2f(tot)) * kPLn2;
      }
      ptx::cluster_barrier();  // no CTA leaves while another reads its part
    }
    if (CL) return;
    cur = next;
    if (cur < end) __syncthreads();  // the results have been read: the rings may fill again
  }
}

// Joins the partial results of the units that several CTAs share: one block
// per query row, its warps taking the pieces in turn.
constexpr int kMergeWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) paged_merge_kernel(const __grid_constant__ PagedDecodeParams p, int lead) {
  __shared__ float osm[kMergeWarps][D];
  __shared__ float wsm[kMergeWarps];
  const int64_t H = p.c.Hkv;
  // (sequence, key/value head, row of the group)
  const uint32_t row = blockIdx.x, unit = row / static_cast<uint32_t>(p.M);
  const int m = static_cast<int>(row - unit * p.M);
  const int b = static_cast<int>(unit / static_cast<uint32_t>(p.c.Hkv));
  const int hkv = static_cast<int>(unit - static_cast<uint32_t>(b) * p.c.Hkv);
  ptx::wait_prerequisites();
  const int64_t per = p.plan[0];
  const int64_t before = p.plan[2 + b];
  const int64_t count = (b + 1 < p.B ? p.plan[3 + b] : quotient(p.plan[1], H)) - before;
  const int64_t first = before * H + hkv * count;  // count: the unit's lead, then its tiles
  const int64_t c0 = quotient(first + lead, per), c1 = quotient(first + count - 1, per);
  if (c0 == c1) return;  // finished by its CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // piece i: CTA c0 + i; the first CTA's piece is its second one unless it starts there
  const int n = static_cast<int>(c1 - c0) + 1;
  const int64_t head = (c0 * 2 + (first <= c0 * per ? 0 : 1)) * p.M + m;
  auto part = [&](int i) { return i == 0 ? head : (c0 + i) * 2 * p.M + m; };
  constexpr int PER = D / 32;
  // the warp's first two pieces set out before the weights are known
  constexpr int AHEAD = 2;
  float first_o[AHEAD][PER], first_l[AHEAD];
#pragma unroll
  for (int a = 0; a < AHEAD; ++a) {
    const int i = warp + a * kMergeWarps;
    const int64_t at = part(i < n ? i : 0);
    const float* op = p.opart + at * D + lane * PER;
    first_l[a] = i < n ? p.lpart[at] : -CUDART_INF_F;
#pragma unroll
    for (int c = 0; c < PER; ++c) first_o[a][c] = op[c];
  }
  float L = -CUDART_INF_F;
  for (int i = lane; i < n; i += 32) L = fmaxf(L, p.lpart[part(i)]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) L = fmaxf(L, __shfl_xor_sync(0xffffffffu, L, d));
  const float Ls = L == -CUDART_INF_F ? 0.f : L;
  float o[PER], ws = 0.f;
#pragma unroll
  for (int c = 0; c < PER; ++c) o[c] = 0.f;
#pragma unroll
  for (int a = 0; a < AHEAD; ++a) {
    const float w = ptx::ex2(first_l[a] - Ls);  // 0 where there is no piece
    ws += w;
#pragma unroll
    for (int c = 0; c < PER; ++c) o[c] = fmaf(w, first_o[a][c], o[c]);
  }
#pragma unroll 4
  for (int i = warp + AHEAD * kMergeWarps; i < n; i += kMergeWarps) {
    const float w = ptx::ex2(p.lpart[part(i)] - Ls);
    const float* op = p.opart + part(i) * D + lane * PER;
    ws += w;
#pragma unroll
    for (int c = 0; c < PER; ++c) o[c] = fmaf(w, op[c], o[c]);
  }
#pragma unroll
  for (int c = 0; c < PER; ++c) osm[warp][lane * PER + c] = o[c];
  if (lane == 0) wsm[warp] = ws;
  __syncthreads();
  float tot = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) tot += wsm[w];
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  const int hq = hkv * p.G + m / p.Lq, i = m % p.Lq;
  __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) + b * p.o_b + hq * p.o_h + i * p.o_l;
  const int c2 = threadIdx.x;
  if (c2 < D / 2) {
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      v.x += osm[w][2 * c2];
      v.y += osm[w][2 * c2 + 1];
    }
    reinterpret_cast<__nv_bfloat162*>(orow)[c2] = __floats2bfloat162_rn(v.x * inv, v.y * inv);
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[(static_cast<int64_t>(b) * p.Hq + hq) * p.Lq + i] = tot == 0.f ? -CUDART_INF_F : (Ls + __log2f(tot)) * kPLn2;
}

template <int FMT, int D, int NT, int RW, bool CL>
constexpr int decode_smem() {
  // the warps' states, and the CTA's part of a cluster's result
  constexpr int merge = kPdWarps * 8 * NT * (kORow<D> + 2) * 4 + (CL ? 8 * NT * RW * (D + 1) * 4 : 0);
  constexpr int ring = Ring<FMT, D, RW>::BYTES;
  return merge > ring ? merge : ring;
}

// Resident CTAs per SM of the current device; sets the kernel's shared-memory
// limit there (< 1 on a CUDA error).
template <int FMT, int D, int NT, int RW, bool CL>
int resident() {
  static OncePerDevice once;
  static int found[kMaxDevices];
  const int dev = t_device;
  const cudaError_t e = on_this_device(once, [dev] {
    constexpr int smem = decode_smem<FMT, D, NT, RW, CL>();
    auto* kernel = paged_decode_kernel<FMT, D, NT, RW, CL>;
    const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return r != cudaSuccess ? r : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&found[dev], kernel, kPdThreads, smem);
  });
  return e == cudaSuccess ? found[dev] : -1;
}

template <int FMT, int D, int NT, int RW>
cudaError_t launch_rows(const PagedDecodeParams& p, cudaStream_t s) {
  if (p.cluster) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.B * p.c.Hkv * p.cluster));
    cfg.blockDim = dim3(kPdThreads);
    cfg.dynamicSmemBytes = decode_smem<FMT, D, NT, RW, true>();
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(p.cluster);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    return cudaLaunchKernelEx(&cfg, paged_decode_kernel<FMT, D, NT, RW, true>, p);
  }
  paged_decode_kernel<FMT, D, NT, RW, false><<<p.grid, kPdThreads, decode_smem<FMT, D, NT, RW, false>(), s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // chained: 26.3 -> 22.9 us at B 16 in a stream (0.2 us less in a graph)
  return launch_chained(paged_merge_kernel<D>, static_cast<unsigned>(p.B * p.c.Hkv * p.M), 32 * kMergeWarps, 0, s, p,
                        kLead<FMT, D>);
}

// 8-row tiles per warp and warps per tile: (1, 1) to 8 rows, (2, 1) to 16, then
// (2, 2) and (2, 4), or with 64 channels, whose O leaves room, (4, 1) and (4, 2)
// (8 sequences to 16001, 4 heads, 64 rows in 4 bits: 30 us against 62; 32 rows
// the same; with 128 channels (4, 2) spills: 50 us against 51 in bf16, 49 against
// 47 in 4 bits)
template <int D>
constexpr int kWide = D == 64 ? 4 : 2;
template <int FMT, int D, bool CL>
int resident_ctas(int M) {
  return M <= 8    ? resident<FMT, D, 1, 1, CL>()
         : M <= 16 ? resident<FMT, D, 2, 1, CL>()
         : M <= 32 ? resident<FMT, D, kWide<D>, 4 / kWide<D>, CL>()
                   : resident<FMT, D, kWide<D>, 8 / kWide<D>, CL>();
}
template <int FMT, int D>
cudaError_t launch_paged(const PagedDecodeParams& p, cudaStream_t s) {
  return p.M <= 8    ? launch_rows<FMT, D, 1, 1>(p, s)
         : p.M <= 16 ? launch_rows<FMT, D, 2, 1>(p, s)
         : p.M <= 32 ? launch_rows<FMT, D, kWide<D>, 4 / kWide<D>>(p, s)
                     : launch_rows<FMT, D, kWide<D>, 8 / kWide<D>>(p, s);
}

}  // namespace

// The launch functions of one format and head width (a translation unit each).
#define FL_DEFINE_PAGED(NAME, FMT, D)                                                                             \
  int paged_resident_##NAME(int M, bool cluster) {                                                                \
    return cluster ? resident_ctas<FMT, D, true>(M) : resident_ctas<FMT, D, false>(M);                            \
  }                                                                                                               \
  cudaError_t launch_paged_##NAME(const PagedDecodeParams& p, cudaStream_t s) { return launch_paged<FMT, D>(p, s); }

}  // namespace fl
