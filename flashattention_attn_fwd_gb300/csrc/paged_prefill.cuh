// Attention of chunks of new tokens over a paged key/value cache in bf16 or in
// 4 bits, for packed sequences that bring anything from no to many tokens.
//
//   t = mod(scale q K^T),  out = softmax(t) V,  lse = log sum exp t
//
// with an online softmax in 32 bits.  4 d operations per visible (query, key)
// and head; the cache's rows are read once per head and unit of 256 query rows.
//
// Rows.  The G query heads of a group times 128 / G consecutive tokens make the
// 128 rows of a slot (row r: token r / G, head r % G), so that a few new tokens of
// grouped heads already fill a tile and a diagonal tile is one of few tokens.  A
// unit is two slots, next to each other in one sequence, and one key/value head:
// both slots use each key tile that is brought in.
//
// Work split.  The host knows neither lengths nor offsets.  The key tiles of all
// (unit, head) pairs form one line that is cut into equal pieces, a block each
// (one per SM), so that any mix of long and short sequences keeps all SMs busy
// to the end.  Every block finds its piece by itself: unit u of the batch takes
// the place floor(seq_offsets[b] / R) + b + (its number in sequence b), R tokens
// a unit, which needs no sum over the sequences before it; a scan of the units'
// tile counts gives the line.  A unit that pieces share leaves one normalised
// partial result and log-sum-exp per piece in the workspace, joined by
// paged_prefill_merge_kernel in piece order, so that a call's result is the same
// every time.  Where whole units are spread evenly enough none is cut.
//
// Roles of a block (bf16 384 threads, 4 bits 512):
//   warp 0      bf16: Q, K and V by TMA, a box per page (of up to 64 rows)
//   warps 1, 2  issue tcgen05.mma: d 64 one warp a slot, d 128 warp 1 for both
//   warp 3      bf16: zeroes V's rows that no row of the unit sees
//   warps 4-11  softmax, a warpgroup per slot and a thread per row; 4 bits: its
//               row of Q, scaled, in fp16
//   warps 12-15 4 bits: load codes and scales into registers a tile ahead, write
//               K and V as fp16 into the swizzled tiles
// K and V tiles alternate in one ring, so that at d 128 five 32 KB places hold
// two and a half tiles beside Q.
//
// 4 bits: code times block scale has at most six significant bits and is exact
// in fp16; the row of Q is scaled by a power of two into fp16's range (undone in
// the score), and P carries 2^7 so that weights down to 2^-31 of the largest
// survive in fp16.  bf16: P is rounded to bf16, V's type.
//
// Measured: 2048 tokens over 32768, 32 heads over 8: bf16 d 128 672 us (1.59 PFLOP/s; 745
// to 790 in a long run, once the power cap has brought the clock down), d 64 503 (1.06), 4 bits
// d 128 764 (1.40), d 64 566 (0.94).  bf16 d 128 is bound by the feeding of the tensor core: a P V and
// S pair takes 1034 cycles, one after another 1245, the waits for P between them.  The
// others are bound by the softmax warps, two a scheduler: 2400 cycles a tile in which each
// waits for S, loads it (300), looks for the maximum (450), writes P (1100).  A change of
// units costs a slot 4000 cycles beside its tiles (output 1800 to 2700, next unit 1200).
//
// TMEM (512 columns): S of slot s at 128 s; d 64: P at 256 + 64 s, O at 384 + 64 s,
// and the next tile's S is issued as soon as this one is in registers; d 128: P
// over the first half of S, O at 256 + 128 s.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <cstdint>

#include "cvt4.cuh"
#include "fused_attn.cuh"
#include "host.h"
#include "paged.h"
#include "ptx.cuh"

namespace fl {
namespace {

// Tiles that starting and ending a unit costs a block, found by measuring 1, 2, 3, 4 and 6
// on packed prompts of 901 to 2999 tokens, 32 heads over 8: bf16 d 128 166, 155, 159, 166
// and 176 us, d 64 144, 127, 125, 129 and 138; 4 bits d 128 258, 209, 197, 198 and 207,
// d 64 200, 161, 150, 153 and 166.
template <int FMT, int D>
constexpr int kPfLead = FMT == KV_BF16 && D == 128 ? 2 : 3;
// Tiles that leaving partial results and joining them costs.
constexpr int kPfJoin = 4;
constexpr uint64_t kPfTurnNs = 4000;
// Softcap: caps up to this take the form for large scores for a whole warp (its error, 2^-20
// cap or 6e-5 of a score, is far below the rounding of P); above, score by score.  Scores past
// the cap, 2048 over 8192 tokens, 32 heads over 8: bf16 d 64 434 us against 593, d 128 413
// against 660; 4 bits 441 against 683 and 468 against 660.
constexpr float kPfCapAll = 64.f;
constexpr uint32_t kPfLift = 7;  // 4 bits: P carries 2^kPfLift

template <int FMT, int D>
struct PfLayout {
  static constexpr bool Q4 = FMT == KV_E2M1;
  static constexpr int THREADS = Q4 ? 512 : 384;
  // registers per thread: at launch, then of the control, softmax and loading warpgroups
  static constexpr int LAUNCH_REGS = Q4 ? 128 : 168;
  static constexpr int CTL_REGS = Q4 ? 64 : D == 128 ? 104 : 72;
  static constexpr int SOFT_REGS = Q4 ? 184 : D == 128 ? 200 : 216;
  static constexpr int LOAD_REGS = Q4 ? 80 : 0;
  static_assert(CTL_REGS + 2 * SOFT_REGS + LOAD_REGS <= (THREADS / 128) * LAUNCH_REGS, "register split");
  static constexpr int HALVES = D / 64;                // 64-channel halves of a row (128 bytes each)
  static constexpr int HALF = 128 * 128;               // bytes of one half of a tile
  static constexpr int TILE = HALVES * HALF;           // bytes of a K, V or Q tile
  // Q: one half after the other.  K and V: groups of 8 rows, in a group 8 rows of one half
  // before 8 of the other, so that one box of a page holds both halves (with a box for each,
  // pages of 16 at d 128 took 869 us for 2048 over 32768 tokens, 32 boxes of 2 KB a tile; 695).
  static constexpr int GROUP = HALVES * 1024;
  static constexpr int FIXED = 2048;                   // barriers and small arrays
  static constexpr int BUDGET = 227 * 1024 - 1024 - FIXED;
  static constexpr int SLOTS_FIT = (BUDGET - 2 * TILE) / TILE;
  static constexpr int NS = SLOTS_FIT > 8 ? 8 : SLOTS_FIT;  // ring places
  static_assert(NS >= 4, "ring too small");
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_FIXED = OFF_RING + NS * TILE;
  // at least 117 KB, so that one block (which owns TMEM) is resident per SM
  static constexpr int END = OFF_FIXED + FIXED + 1024;
  static constexpr int SMEM = END > 120 * 1024 ? END : 120 * 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// One (unit, head): tokens, keys, tiles.
struct PfUnit {
  int b, qt, h;
  int tok0, ntok;     // first token (row of q) and tokens of the unit
  int p0, n;          // position of the first token; keys of the sequence
  int vis_lo, vis_end;  // some row sees keys [vis_lo, vis_end) and, below vis_end, [0, sink)
  int sinkt, skip, count;  // tile i is that of key 128 (i < sinkt ? i : i + skip)
  int64_t base;       // line position of tile 0 (whole units: the unit's)
};

// Barriers and small arrays in the fixed area.
template <int NS>
struct PfShared {
  uint64_t kv_full[NS], kv_empty[NS];
  uint64_t q_full[2], q_empty[2], s_full[2], s_free[2], p_lo[2], p_hi[2], pv_done[2], o_empty[2], drain[2];
  uint64_t v_land[8];       // V tiles with rows to be zeroed: landed
  int64_t scan[16];
  int scan_units[16], largest[16];
  PfUnit found;             // the piece's first unit; b < 0: none
  uint32_t tmem, abort;
  uint32_t bad[16];         // by tile: bits of 16-key groups whose page is not in the pool
  uint32_t issued[NS];      // last load of each place: (barrier << 1 | parity) + 1, 0: none
  uint32_t turn[2];         // tiles of which a slot's products have been issued
  int64_t begin, end;       // this block's piece of the line
  int whole;                // the line counts units: none is cut
  PfUnit unit[16];          // of every warp: where it is (in registers they would be spilled)
};

// As wait_bar, its slow path out of the way.
__device__ __forceinline__ bool pf_wait(uint64_t* bar, uint32_t parity, const Ctl& c, int where) {
  if (__builtin_expect(ptx::mbar_try_wait(bar, parity), 1)) return true;
  return wait_slow(bar, parity, c, where);
}

template <int LEAD>
struct PfSeqs {
  const PrefillParams& p;
  int R;  // tokens per unit
  __device__ __forceinline__ int offset(int b) const {
    if (!p.seq_offsets) return b;
    return min(max(__ldg(p.seq_offsets + b), 0), p.T);
  }
  // units in t tokens, rounded down
  __device__ __forceinline__ int units(int t) const {
    return static_cast<int>(__umulhi(static_cast<uint32_t>(t), p.div_m) >> p.div_s);
  }
  // tiles of unit qt of sequence b (offsets o to e), with its fields
  __device__ __forceinline__ void fill(PfUnit& u, int b, int qt, int o, int e) const {
    u.b = b;
    u.qt = qt;
    u.tok0 = o + qt * R;
    u.ntok = min(R, e - u.tok0);
    u.n = min(max(__ldg(p.kv_len + b), 0), p.cap);
    u.p0 = u.n - (e - o) + qt * R;
    tiles(u);
  }
  __device__ __forceinline__ void tiles(PfUnit& u) const {
    u.vis_end = p.causal ? max(u.p0 + u.ntok, 0) : u.n;
    u.vis_lo = p.window ? max(u.p0 - p.window + 1, 0) : 0;
    const int first = u.vis_lo >> 7;
    u.sinkt = p.window ? min((p.sink + 127) >> 7, first) : 0;
    u.skip = first - u.sinkt;
    u.count = max(((u.vis_end + 127) >> 7) - u.skip, 1);
  }
  // the next (unit, head) of the line; false behind the last
  __device__ __forceinline__ bool next(PfUnit& u, bool whole) const {
    u.base += whole ? 1 : LEAD + u.count;
    if (++u.h < p.c.Hkv) return true;
    u.h = 0;
    int o = offset(u.b), e = max(offset(u.b + 1), o);
    if (u.tok0 + R < e) {
      fill(u, u.b, u.qt + 1, o, e);
      return true;
    }
    for (int b = u.b + 1; b < p.B; ++b) {
      o = offset(b);
      e = max(offset(b + 1), o);
      if (e > o) {
        fill(u, b, 0, o, e);
        return true;
      }
    }
    return false;
  }
};
__device__ __forceinline__ int pf_key(const PfUnit& u, int i) { return 128 * (i < u.sinkt ? i : i + u.skip); }
__device__ __forceinline__ bool pf_seen(const PrefillParams& p, const PfUnit& u, int j) {
  return j < u.vis_end && (j >= u.vis_lo || j < p.sink);
}
// does every key of [j, j + len) meet some row of the unit, does any
__device__ __forceinline__ bool pf_all_seen(const PrefillParams& p, const PfUnit& u, int j, int len) {
  return j + len <= u.vis_end && (j >= u.vis_lo || j + len <= p.sink);
}
__device__ __forceinline__ bool pf_any_seen(const PrefillParams& p, const PfUnit& u, int j, int len) {
  return j < u.vis_end && (j + len > u.vis_lo || j < p.sink);
}

// a / b of non-negative values, in 32 bits where both fit
__device__ __forceinline__ int64_t pf_quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// the lowest n bits (n <= 0: none, n >= 32: all)
__device__ __forceinline__ uint32_t pf_low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

__device__ __forceinline__ uint32_t pf_pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void st_shared128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// One lane of the converged warp.  The warps that issue tcgen05.mma stay converged
// and wait with all lanes: a lane that went its own way had 200 cycles between a
// wait and its next product, time in which the tensor core runs dry (it is fed a
// product or two ahead).
__device__ __forceinline__ bool pf_elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0u;
}

template <int FMT, int D, int SCORE>
__global__ void __launch_bounds__(PfLayout<FMT, D>::THREADS, 1)
    paged_prefill_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PrefillParams p) {
  using L = PfLayout<FMT, D>;
  constexpr bool Q4 = L::Q4;
  constexpr int NS = L::NS;
  constexpr bool kSepP = D == 64;
  constexpr uint32_t kColP = kSepP ? 256u : 0u, kStrP = kSepP ? 64u : 128u;
  constexpr uint32_t kColO = kSepP ? 384u : 256u;
  extern __shared__ uint8_t pf_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pf_raw) + 1023) & ~uintptr_t(1023));
  using Shared = PfShared<NS>;
  static_assert(sizeof(Shared) <= L::FIXED, "fixed area");
  Shared& sh = *reinterpret_cast<Shared*>(smem + L::OFF_FIXED);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int LEAD = kPfLead<FMT, D>;
  const PfSeqs<LEAD> seqs{p, 2 * p.RT};
  const int64_t H = p.c.Hkv;

  // the plan's first reads, on their way during the set-up
  if (32 * tid <= p.B) {
    if (p.seq_offsets) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.seq_offsets + 32 * tid));
    if (32 * tid < p.B) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.kv_len + 32 * tid));
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      ptx::mbar_init(&sh.kv_full[i], Q4 ? 4 : 1);
      ptx::mbar_init(&sh.kv_empty[i], 2);
      sh.issued[i] = 0u;
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sh.q_full[i], Q4 ? 4 : 1);
      ptx::mbar_init(&sh.q_empty[i], 1);
      ptx::mbar_init(&sh.s_full[i], 1);
      ptx::mbar_init(&sh.s_free[i], 4);
      ptx::mbar_init(&sh.p_lo[i], 4);
      ptx::mbar_init(&sh.p_hi[i], 4);
      ptx::mbar_init(&sh.pv_done[i], 1);
      ptx::mbar_init(&sh.o_empty[i], 4);
      ptx::mbar_init(&sh.drain[i], 1);
    }
    for (int i = 0; i < 8; ++i) ptx::mbar_init(&sh.v_land[i], 1);
    sh.abort = 0u;
    sh.found.b = -1;
    sh.turn[0] = sh.turn[1] = 0u;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (tid < 16) sh.bad[tid] = 0u;
  if (warp == 1) {
    ptx::tmem_alloc(&sh.tmem, 512);
    ptx::tmem_relinquish();
  }
  if (warp == 0 && lane == 0 && !Q4) {
    ptx::prefetch_tensormap(&tmQ);
    ptx::prefetch_tensormap(&tmK);
    ptx::prefetch_tensormap(&tmV);
  }
  if (!Q4 && p.RT * p.G < 128) {
    // rows behind the last token's heads are never loaded: zeros
    uint4* q = reinterpret_cast<uint4*>(smem + L::OFF_Q);
    for (int i = tid; i < 2 * L::TILE / 16; i += L::THREADS) q[i] = make_uint4(0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
  }

  // ---- this block's piece of the line
  const int R = seqs.R;
  const int places = seqs.units(p.T) + p.B;
  int64_t per, begin, end;
  bool whole;
  {
    const int chunk = (places + L::THREADS - 1) / L::THREADS;
    const int u0 = tid * chunk, u1 = min(u0 + chunk, places);
    // the last sequence whose units start at or before place u0
    auto start = [&](int b) { return seqs.units(seqs.offset(b)) + b; };
    int b0 = 0;
    if (u0 < u1) {
      int hi = p.B - 1;
      while (b0 < hi) {
        const int mid = (b0 + hi + 1) >> 1;
        if (start(mid) <= u0) b0 = mid; else hi = mid - 1;
      }
    }
    auto walk = [&](auto&& f) {
      int b = b0;
      int o = 0, e = 0, s = 0, s1 = 0;
      if (u0 < u1) {
        o = seqs.offset(b);
        e = max(seqs.offset(b + 1), o);
        s = seqs.units(o) + b;
        s1 = b + 1 < p.B ? start(b + 1) : places;
      }
      for (int u = u0; u < u1; ++u) {
        while (u >= s1 && b + 1 < p.B) {
          ++b;
          o = seqs.offset(b);
          e = max(seqs.offset(b + 1), o);
          s = seqs.units(o) + b;
          s1 = b + 1 < p.B ? start(b + 1) : places;
        }
        if (u < s || static_cast<int64_t>(u - s) * R >= e - o) continue;
        PfUnit un;
        seqs.fill(un, b, u - s, o, e);
        f(un);
      }
    };
    int64_t mine = 0;
    int units = 0, largest = 0;
    walk([&](const PfUnit& un) {
      mine += LEAD + un.count;
      ++units;
      largest = max(largest, LEAD + un.count);
    });
    int64_t incl = mine;
    int incl_units = units;  // places fit 32 bits
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      const int w = __shfl_up_sync(0xffffffffu, incl_units, o);
      if (lane >= o) {
        incl += v;
        incl_units += w;
      }
    }
    largest = __reduce_max_sync(0xffffffffu, largest);
    if (lane == 31) {
      sh.scan[warp] = incl;
      sh.scan_units[warp] = incl_units;
      sh.largest[warp] = largest;
    }
    __syncthreads();
    int64_t before = incl - mine, total = 0;
    int before_units = incl_units - units, total_units = 0;
    for (int w = 0; w < L::THREADS / 32; ++w) {
      if (w < warp) {
        before += sh.scan[w];
        before_units += sh.scan_units[w];
      }
      total += sh.scan[w];
      total_units += sh.scan_units[w];
      largest = max(largest, sh.largest[w]);
    }
    per = pf_quotient(total * H + gridDim.x - 1, gridDim.x);
    // as many whole units a block where the longest such piece costs no more than a cut
    // one with a unit's start and the joining of partial results more
    const int64_t each = pf_quotient(total_units * H + gridDim.x - 1, gridDim.x);
    whole = each * largest <= per + LEAD + kPfJoin;
    if (whole) {
      per = each;
      total = total_units;
      mine = units;
      before = before_units;
    }
    total *= H;
    begin = per * blockIdx.x;
    end = min(begin + per, total);
    if (tid == 0) {
      sh.begin = begin;
      sh.end = end;
      sh.whole = whole;
    }
    if (begin < end && before * H <= begin && begin < (before + mine) * H) {
      int64_t at = before * H;
      walk([&](const PfUnit& un) {
        const int64_t c = whole ? 1 : LEAD + un.count;
        if (at <= begin && begin < at + c * H) {
          const int h = static_cast<int>(pf_quotient(begin - at, c));
          PfUnit f = un;
          f.h = h;
          f.base = at + h * c;
          sh.found = f;
        }
        at += c * H;
      });
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const Ctl ctl{reinterpret_cast<volatile uint32_t*>(&sh.abort), p.status, p.timeout_ns};
  const uint64_t drain_ns = 50ull * 1000ull * 1000ull;
  ptx::launch_dependents();

  if (blockIdx.x > 0 && tid == 0) {
    // is this block's border inside of a unit, and which pieces share that one
    const PfUnit f = sh.found;
    int32_t* r = p.rec + static_cast<int64_t>(blockIdx.x) * 8;
    const int64_t t = f.b >= 0 ? begin - f.base : 0;
    const bool cut = !whole && t > 0 && t < f.count;
    r[0] = cut ? 1 : 0;
    if (cut) {
      r[1] = f.tok0;
      r[2] = f.ntok;
      r[3] = f.h;
      r[4] = static_cast<int>(pf_quotient(f.base, per));
      r[5] = static_cast<int>(pf_quotient(f.base + f.count - 1, per));
    }
  }
  // The warp's next unit that has tiles in this piece, into sh.unit[warp], and its
  // tiles [a, z) there; not to be asked again once there is none.
  bool begun = false;
  auto next_unit = [&](int& a, int& z) -> bool {
    PfUnit& at = sh.unit[warp];
    while (true) {
      PfUnit u = begun ? at : sh.found;
      __syncwarp();
      if (begun ? !seqs.next(u, sh.whole) : u.b < 0) return false;
      begun = true;
      at = u;
      __syncwarp();
      const int64_t t0 = sh.begin - u.base, t1 = sh.end - u.base;
      if (t1 <= 0) return false;
      if (sh.whole) {
        a = 0;
        z = u.count;
        return true;
      }
      a = t0 > 0 ? static_cast<int>(min(t0, static_cast<int64_t>(u.count))) : 0;
      z = t1 < u.count ? static_cast<int>(t1) : u.count;
      if (a < z) return true;
    }
  };
  // f(unit, a, z) for each of them, until f fails
  auto each_unit = [&](auto&& f) {
    int a, z;
    while (next_unit(a, z))
      if (!f(static_cast<const PfUnit&>(sh.unit[warp]), a, z)) return;
  };
  const int shift = p.c.page_shift;
  const int page_mask = (1 << shift) - 1;

  if (warp < 4) {
    ptx::setmaxnreg_dec<L::CTL_REGS>();
    if (warp == 0 && !Q4) {
      // ---------------------------------------------------------------- loads
      const uint64_t pol_q = ptx::policy_evict_first(), pol_kv = ptx::policy_evict_last();
      const int sub_len = min(1 << shift, kPrefillBox), nsub = 128 / sub_len;  // boxes of a tile
      const int sub = lane & 15;                       // lanes 0-15 K, 16-31 V
      const bool mine = sub < nsub;
      const int groups = 1 << (shift - 3);             // of 8 rows, in a page and head
      uint32_t e = 0, tile = 0, part = 0, qc[2] = {0u, 0u};
      int q_phase[2] = {-1, -1};
      each_unit([&](const PfUnit& u, int a, int z) {
        // page of this lane's keys of tile i: num_pages (read as zeros) when no
        // row sees them, or (reported) when it is not in the pool
        auto lookup = [&](int i) -> int {
          const int j = pf_key(u, i) + sub * sub_len;
          if (i >= z || !mine || !pf_any_seen(p, u, j, sub_len)) return p.c.num_pages;
          return __ldg(p.table + u.b * p.table_stride + (j >> shift));
        };
        int next = lookup(a);
        for (int i = a; i < z; ++i, ++tile, e += 2) {
          const int j0 = pf_key(u, i);
          int page = next;
          next = lookup(i + 1);
          const bool out_of_pool = page != p.c.num_pages && (page < 0 || page > p.c.num_pages);
          const bool at_end = page == p.c.num_pages && mine && pf_any_seen(p, u, j0 + sub * sub_len, sub_len);
          const bool bad = out_of_pool || at_end;
          if (bad) page = p.c.num_pages;
          const uint32_t badl = __ballot_sync(0xffffffffu, bad && mine && lane < 16);
          if (lane == 0) {
            uint32_t w = 0u;
            if (badl) {
              atomicOr(p.status, 2u);
              for (int g = 0; g < 8; ++g)
                if (badl >> (g * 16 / sub_len) & 1u) w |= 1u << (8 * (g >> 1) + (g & 1));
            }
            sh.bad[tile & 15u] = w;
          }
          const int group = (page * p.c.Hkv + u.h) * groups + (((j0 + sub * sub_len) & page_mask) >> 3);
          const bool whole = pf_all_seen(p, u, j0, 128);
          for (int v = 0; v < 2; ++v) {
            const uint32_t ev = e + v;
            const int st = static_cast<int>(ev % NS);
            if (!__all_sync(0xffffffffu, pf_wait(&sh.kv_empty[st], ((ev / NS) & 1u) ^ 1u, ctl, 2))) return false;
            const bool land = v == 1 && !whole;
            uint64_t* bar = land ? &sh.v_land[part & 7u] : &sh.kv_full[st];
            const bool skip = v == 0 && p.dbg_skip_tile >= 0 && blockIdx.x == 0 &&
                              static_cast<int>(tile) == p.dbg_skip_tile;
            if (lane == 0) {
              const uint32_t ph = land ? (part >> 3) & 1u : (ev / NS) & 1u;
              const uint32_t which = land ? NS + (part & 7u) : st;
              sh.issued[st] = skip ? 0u : (which << 1 | ph) + 1u;
              ptx::mbar_arrive_expect_tx(bar, L::TILE);
            }
            __syncwarp();
            if (mine && (lane >= 16) == (v == 1) && !skip)
              ptx::tma_load_4d(smem + L::OFF_RING + st * L::TILE + sub * (sub_len / 8) * L::GROUP, v ? &tmV : &tmK, bar, 0, 0,
                               0, group, pol_kv);
            if (land) ++part;
            if (i > a || v) continue;
            // Q behind the first K, which need not wait for the last unit's end
            for (int s = 0; s < 2; ++s) {
              if (u.ntok <= s * p.RT) continue;
              if (!__all_sync(0xffffffffu, pf_wait(&sh.q_empty[s], (qc[s] & 1u) ^ 1u, ctl, 1))) return false;
              if (lane == 0) {
                ptx::mbar_arrive_expect_tx(&sh.q_full[s], p.RT * p.G * D * 2);
                for (int x = 0; x < L::HALVES; ++x)
                  ptx::tma_load_4d(smem + L::OFF_Q + s * L::TILE + x * L::HALF, &tmQ, &sh.q_full[s], 64 * x, 0, u.h,
                                   u.tok0 + s * p.RT, pol_q);
              }
              q_phase[s] = static_cast<int>(qc[s] & 1u);
              ++qc[s];
            }
          }
        }
        return true;
      });
      if (lane == 0 && *ctl.abort) {
        // let every copy land before the block exits
        for (int st = 0; st < NS; ++st) {
          const uint32_t w = sh.issued[st];
          if (!w) continue;
          const uint32_t which = (w - 1u) >> 1;
          wait_drain(which < NS ? &sh.kv_full[which] : &sh.v_land[which - NS], (w - 1u) & 1u, drain_ns);
        }
        for (int s = 0; s < 2; ++s)
          if (q_phase[s] >= 0) wait_drain(&sh.q_full[s], static_cast<uint32_t>(q_phase[s]), drain_ns);
      }
      __syncwarp();
    } else if (warp == 3 && !Q4) {
      // ------------------------- V's rows that no row of the unit sees: zeros
      // (P is 0 there, and 0 times whatever the pool holds has to be 0)
      uint32_t e = 0, part = 0;
      Ctl later = ctl;  // the limit once per tile that is passed
      each_unit([&](const PfUnit& u, int a, int z) {
        for (int i = a; i < z; ++i, e += 2) {
          const int j0 = pf_key(u, i);
          later.timeout_ns += ctl.timeout_ns;
          if (pf_all_seen(p, u, j0, 128)) continue;
          const int st = static_cast<int>((e + 1) % NS);
          if (!__all_sync(0xffffffffu, pf_wait(&sh.v_land[part & 7u], (part >> 3) & 1u, later, 3))) return false;
          later.timeout_ns = ctl.timeout_ns;
          ++part;
          const uint32_t base = ptx::smem_u32(smem + L::OFF_RING + st * L::TILE);
          const int end = u.vis_end - j0, from = u.vis_lo - j0, sinks = p.sink - j0;
#pragma unroll 4
          for (int r = lane >> 3; r < 128; r += 4)
            if (r >= end || (r < from && r >= sinks))
#pragma unroll
              for (int h = 0; h < L::HALVES; ++h)
                st_shared128(base + (r >> 3) * L::GROUP + h * 1024 + (r & 7) * 128 + (lane & 7) * 16, 0u, 0u, 0u, 0u);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.kv_full[st]);
        }
        return true;
      });
    } else if (warp == 1 || (kSepP && warp == 2)) {
      // ------------------------------------------------------------ MMA issue
      // A commit, too, costs the tensor core its lead (60 cycles where two follow
      // one another), so that there is one for S and one where P V has to be known
      // as done; the places of K and V are given back by the softmax warps, which
      // wait for those anyway.
      constexpr uint32_t kTypes = Q4 ? ~((1u << 7) | (1u << 10)) : ~0u;  // fp16 operands
      constexpr uint32_t IDESC_S = ptx::idesc_bf16_f32(128, 128, false) & kTypes;
      constexpr uint32_t IDESC_O = ptx::idesc_bf16_f32(128, D, true) & kTypes;
      const uint32_t ring = ptx::smem_u32(smem + L::OFF_RING);
      const uint32_t qa = ptx::smem_u32(smem + L::OFF_Q);
      // One answer for the warp: lanes that part where a wait gives up would not meet again
      // at the next elect.sync.
      auto wait = [&](uint64_t* bar, uint32_t parity, int where) {
        return __all_sync(0xffffffffu, pf_wait(bar, parity & 1u, ctl, where)) != 0;
      };
      auto full = [&](uint32_t ev, int where) { return wait(&sh.kv_full[ev % NS], ev / NS, where); };
      auto free_place = [&](uint32_t ev) {
        if (lane == 0) ptx::mbar_arrive(&sh.kv_empty[ev % NS]);
      };
      // by the elected lane
      auto issue_s = [&](int s, uint32_t ev) {
        const uint64_t qd = ptx::smem_desc(qa + s * L::TILE, 16, 1024, 2u);
        const uint64_t kd = ptx::smem_desc(ring + (ev % NS) * L::TILE, 16, L::GROUP, 2u);
#pragma unroll
        for (int kb = 0; kb < D / 16; ++kb) {
          const uint32_t c = (kb % 4) * 32;
          ptx::mma_ss(tmem + s * 128, qd + (((kb / 4) * L::HALF + c) >> 4), kd + (((kb / 4) * 1024 + c) >> 4), IDESC_S,
                      kb > 0 ? 1u : 0u);
        }
        ptx::mma_commit(&sh.s_full[s]);
      };
      auto issue_pv = [&](int s, uint32_t ev, bool acc, int kb0) {
        const uint64_t vd = ptx::smem_desc(ring + (ev % NS) * L::TILE, 1024, L::GROUP, 2u);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int kb = kb0 + k;
          ptx::mma_ts(tmem + kColO + s * D, tmem + kColP + s * kStrP + kb * 8, vd + ((kb * 2 * L::GROUP) >> 4), IDESC_O,
                      (acc || kb > 0) ? 1u : 0u);
        }
      };
      uint32_t e = 0;
      if constexpr (!kSepP) {
        // d 128, P over S: P V and then the next S of one slot, then of the other,
        // so that one slot's softmax runs under the other's products.  A unit's last P V
        // is followed by the next unit's first S (4 bits: once both slots are through,
        // since their queries come late).
        constexpr bool kAhead = !Q4;
        uint32_t qc = 0u, oc = 0u, pc = 0u;  // bit s: slot s's phases of Q, O and P
        auto next_piece = [&](int& n, int& slots) {
          int a, z;
          if (!next_unit(a, z)) return false;
          n = z - a;
          slots = sh.unit[warp].ntok > p.RT ? 2 : 1;  // with rows
          return true;
        };
        // a unit's first S of slot s, its K at ev
        auto first_s = [&](int s, uint32_t ev) {
          if (!full(ev, 11) || !wait(&sh.q_full[s], qc >> s, 10)) return false;
          ptx::tc_fence_after();
          if (pf_elect()) issue_s(s, ev);
          qc ^= 1u << s;
          return true;
        };
        int n = 0, slots = 0;
        bool go = next_piece(n, slots);
        bool ahead = false;  // the unit's first S is issued
        while (go) {
          if (!ahead) {
            if (!first_s(0, e) || (slots > 1 && !first_s(1, e))) break;
            if (slots < 2) free_place(e);
          }
          int n1 = 0, slots1 = 0;
          const bool go1 = next_piece(n1, slots1);
          for (int i = 0; i < n && go; ++i, e += 2) {
            const bool more = i + 1 < n;
#pragma unroll 1
            for (int s = 0; s < slots; ++s) {
              // all at once first: one wait's latency, not four
              uint64_t* v_bar = &sh.kv_full[(e + 1) % NS];
              uint64_t* k_bar = &sh.kv_full[(e + 2) % NS];
              const uint32_t v_ph = ((e + 1) / NS) & 1u, k_ph = ((e + 2) / NS) & 1u;
              const bool v_ok = ptx::mbar_test_wait(v_bar, v_ph), k_ok = ptx::mbar_test_wait(k_bar, k_ph);
              const bool o_ok = ptx::mbar_test_wait(&sh.o_empty[s], ((oc >> s) + 1u) & 1u);
              const bool p_ok = ptx::mbar_test_wait(&sh.p_lo[s], (pc >> s) & 1u);
              if (!__all_sync(0xffffffffu, v_ok & (k_ok | !more) & (o_ok | (i > 0)) & p_ok)) {
                go = wait(v_bar, v_ph, 16) && (!more || wait(k_bar, k_ph, 11)) &&
                     (i > 0 || wait(&sh.o_empty[s], (oc >> s) + 1u, 13)) && wait(&sh.p_lo[s], pc >> s, 14);
                if (!go) break;
              }
              ptx::tc_fence_after();
              if (pf_elect()) issue_pv(s, e + 1, i > 0, 0);
              go = wait(&sh.p_hi[s], pc >> s, 15);
              if (!go) break;
              ptx::tc_fence_after();
              if (pf_elect()) {
                issue_pv(s, e + 1, true, 4);
                if (more) issue_s(s, e + 2);
                else ptx::mma_commit(&sh.pv_done[s]);
              }
              pc ^= 1u << s;
              if (kAhead && !more && s < slots1) {
                go = first_s(s, e + 2);
                if (!go) break;
              }
            }
            if (slots < 2) {
              free_place(e + 1);
              if (more) free_place(e + 2);
            }
          }
          if (!go) break;
          oc ^= slots < 2 ? 1u : 3u;
          ahead = kAhead && go1;
          if (ahead) {
            if (slots1 < 2) free_place(e);
            else if (slots < 2 && !first_s(1, e)) break;
          }
          n = n1;
          slots = slots1;
          go = go1;
        }
      } else {
        // d 64, P beside S: a warp a slot; the next S as soon as this one is in
        // registers.  The slots' P V take turns: slot 1's of a tile follows slot 0's,
        // and slot 0's of the next tile that one; left alone, the slots fall into step.
        // Only an order: giving up is fine.
        const int s = warp - 1;
        uint32_t qc = 0, sc = 0, pc = 0;
        auto await_turn = [&](uint32_t tiles) {  // of the other slot
          volatile uint32_t* t = &sh.turn[s ^ 1];
          if (static_cast<int32_t>(*t - tiles) >= 0) return;
          const uint64_t t0 = ptx::globaltimer_ns();
          while (static_cast<int32_t>(*t - tiles) < 0)
            if (ptx::globaltimer_ns() - t0 > kPfTurnNs) return;
        };
        auto my_turn_over = [&](uint32_t tiles) {
          if (lane == 0) *const_cast<volatile uint32_t*>(&sh.turn[s]) = tiles;
        };
        auto next_s = [&](uint32_t ev) {
          if (!full(ev, 11) || !wait(&sh.s_free[s], sc + 1u, 12)) return false;
          ptx::tc_fence_after();
          if (pf_elect()) issue_s(s, ev);
          ++sc;
          return true;
        };
        each_unit([&](const PfUnit& u, int a, int z) {
          const int n = z - a;
          if (u.ntok <= s * p.RT) {
            // no rows in this slot: pass the unit's tiles
            for (int i = 0; i < 2 * n; ++i, ++e) {
              if (!full(e, 17)) return false;
              free_place(e);
              my_turn_over((e >> 1) + 1);
            }
            return true;
          }
          if (!wait(&sh.q_full[s], qc, 10) || !next_s(e)) return false;
          for (int i = 0; i < n; ++i, e += 2) {
            if (i + 1 < n && !next_s(e + 2)) return false;
            if (i == 0 && !wait(&sh.o_empty[s], qc + 1u, 13)) return false;
            if (!full(e + 1, 16)) return false;
            await_turn((e >> 1) + s);
            if (!wait(&sh.p_lo[s], pc, 14)) return false;
            ptx::tc_fence_after();
            if (pf_elect()) issue_pv(s, e + 1, i > 0, 0);
            if (!wait(&sh.p_hi[s], pc, 15)) return false;
            ptx::tc_fence_after();
            if (pf_elect()) {
              issue_pv(s, e + 1, true, 4);
              ptx::mma_commit(&sh.pv_done[s]);
            }
            ++pc;
            my_turn_over((e >> 1) + 1);
          }
          ++qc;
          return true;
        });
      }
      // every MMA that was issued must finish before TMEM is released
      __syncwarp();
      if (lane == 0) {
        ptx::mma_commit(&sh.drain[warp - 1]);
        wait_drain(&sh.drain[warp - 1], 0u, drain_ns);
      }
    }
    __syncwarp();
  } else if (warp < 12) {
    // -------------------------------------------------------------- softmax
    ptx::setmaxnreg_inc<L::SOFT_REGS>();
    const int sw = warp - 4, s = sw >> 2, quad = sw & 3;
    const int r = quad * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t tS = tl + s * 128, tP = tl + kColP + s * kStrP, tO = tl + kColO + s * D;
    const int rtok = r / p.G, rg = r - rtok * p.G;
    const bool row_used = rtok < p.RT;
    uint32_t sc = 0, tile = 0;
    int idle = 1;  // tiles of the other slot that were passed, in limits of a wait
    // What is left to do for a unit when its tiles are done: that runs once the
    // next unit's queries are on their way.
    struct Rest {
      float m, l;
      int64_t row;   // of out and lse, or of the partial results
      uint32_t tile; // the last one
      int h;
      bool live, whole;
    } rest{};
    bool have_rest = false;
    // the place of the ring that entry ev (2 tile: K, 2 tile + 1: V) had, for this slot
    auto free_place = [&](uint32_t ev) {
      if (lane == 0 && quad == 0) ptx::mbar_arrive(&sh.kv_empty[ev % NS]);
    };
    uint32_t units = 0;  // of this slot
    auto finish = [&]() -> bool {
      have_rest = false;
      const uint32_t done = kSepP ? sc - 1 : units - 1;  // phases: a tile each, or (d 128) a unit each
      if (!__all_sync(0xffffffffu, pf_wait(&sh.pv_done[s], done & 1u, ctl, 30 + s))) return false;
      free_place(2 * rest.tile + 1);
      ptx::tc_fence_after();
      const float l = rest.l, lift = Q4 ? static_cast<float>(kPfLift) : 0.f;
      const float lse2 = l > 0.f ? rest.m + __log2f(l) - lift : (l == l ? -CUDART_INF_F : l);
      const float inv = l > 0.f || l != l ? (Q4 ? p.c.v_scale : 1.f) / l : 0.f;
      if (rest.whole) {
        // Four lanes exchange 16-byte pieces so that each stores its piece of four
        // rows and the four together 64 bytes of a row: a thread's own row in
        // 16-byte stores took five times as long (32 lines an instruction).
        const int64_t at = rest.live ? rest.row * p.o_t + rest.h * p.o_h : -1;
        if (rest.live && p.lse) p.lse[rest.row * p.Hq + rest.h] = lse2 * kLn2;
        int64_t row[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) row[k] = __shfl_sync(0xffffffffu, at, (lane & ~3) + k);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + 8 * (lane & 3);
        // not unrolled: code that runs once a unit comes through the instruction cache anew (packed
        // prompts, bf16 d 128 163 -> 156 us, d 64 137 -> 130)
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          uint32_t w[4][4];
          ptx::tmem_ld32(tO + c, o);
          ptx::tmem_ld_wait();
          ptx::reg_fence32(o);
#pragma unroll
          for (int q = 0; q < 16; ++q)
            w[q >> 2][q & 3] = ptx::pack_bf16x2(__uint_as_float(o[2 * q]) * inv, __uint_as_float(o[2 * q + 1]) * inv);
#pragma unroll
          for (int st = 1; st < 4; st *= 2) {
            const bool up = lane & st;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (q & st) continue;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t t = __shfl_xor_sync(0xffffffffu, up ? w[q][k] : w[q + st][k], st);
                if (up) w[q][k] = t;
                else w[q + st][k] = t;
              }
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (row[k] >= 0) *reinterpret_cast<uint4*>(out + row[k] + c) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
        }
      } else {
        float4* op = reinterpret_cast<float4*>(p.opart) + rest.row * (D / 4) * 128 + r;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          ptx::tmem_ld32(tO + c, o);
          ptx::tmem_ld_wait();
          ptx::reg_fence32(o);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            op[(c / 4 + q) * 128] =
                make_float4(__uint_as_float(o[4 * q]) * inv, __uint_as_float(o[4 * q + 1]) * inv,
                            __uint_as_float(o[4 * q + 2]) * inv, __uint_as_float(o[4 * q + 3]) * inv);
        }
        p.lpart[rest.row * 128 + r] = lse2;
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.o_empty[s]);
      return true;
    };
    // one copy of each part in the code: the tile loop shares the instruction cache
    // with the other roles
    while (true) {
      int a = 0, z = 0;
      bool more;
      const PfUnit& u = sh.unit[warp];
      while ((more = next_unit(a, z)) && u.ntok <= s * p.RT) {
        tile += z - a;
        idle += z - a;
      }
      if (!more) {
        if (have_rest) finish();
        break;
      }
      // rows without a token take the last one's bounds (their results are dropped)
      const int tok = s * p.RT + rtok;
      const int pos = u.p0 + min(tok, u.ntok - 1);
      const int hi = p.causal ? min(pos, u.n - 1) : u.n - 1;
      const int lo = p.window ? max(pos - p.window + 1, 0) : 0;
      const int hq = u.h * p.G + rg;
      const bool live = row_used && tok < u.ntok;
      float rf = 1.f;
      if constexpr (Q4) {
        // Q to fp16, each row scaled by a power of two that takes its largest channel to
        // 2^14.  The last unit's Q is free: its last S is done (this warp has it).  Four
        // lanes read 64 bytes of a row together, four rows in turn (a thread's own row in
        // 16-byte loads took three times as long: 32 lines an instruction).
        const int64_t at = live ? static_cast<int64_t>(u.tok0 + tok) * p.q_t + hq * p.q_h : -1;
        const int r4 = lane & ~3, j4 = lane & 3;
        uint4 w[4][D / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t row = __shfl_sync(0xffffffffu, at, r4 + k);
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + row) + j4;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) w[k][c] = row >= 0 ? __ldg(src + 4 * c) : make_uint4(0u, 0u, 0u, 0u);
        }
        const uint32_t base = ptx::smem_u32(smem + L::OFF_Q) + s * L::TILE + (quad * 32 + r4) * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t mx = 0u;  // bf16 magnitudes order as integers
#pragma unroll
          for (int c = 0; c < D / 32; ++c)
            mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(w[k][c].x & 0x7fff7fffu, w[k][c].y & 0x7fff7fffu),
                                       __vmaxu2(w[k][c].z & 0x7fff7fffu, w[k][c].w & 0x7fff7fffu)));
          mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const int ex = static_cast<int>((max(mx & 0xffffu, mx >> 16) >> 7) & 0xffu);  // biased exponent
          // zeros, and rows whose largest is not finite, as they are; tiny ones by 2^110 at most
          const int up = ex == 0 || ex == 255 ? 0 : min(14 - (ex - 127), 110);
          const float f = __int_as_float((up + 127) << 23);
          if (k == j4) rf = __int_as_float((127 - up) << 23);
          const int rx = (r4 + k) & 7;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const int piece = 4 * c + j4;
            const uint32_t x[4] = {w[k][c].x, w[k][c].y, w[k][c].z, w[k][c].w};
            uint32_t y[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              y[q] = pf_pack_f16(__uint_as_float(x[q] << 16) * f, __uint_as_float(x[q] & 0xffff0000u) * f);
            st_shared128(base + k * 128 + (piece >> 3) * L::HALF + (((piece & 7) ^ rx) << 4), y[0], y[1], y[2], y[3]);
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.q_full[s]);
      }
      if (have_rest && !finish()) break;
      const float xmul = SCORE == SCORE_NONE ? p.scale_log2 * rf : 1.f;
      const float slope2 = SCORE == SCORE_ALIBI ? __ldg(p.slopes + (row_used ? hq : 0)) * kLog2e : 0.f;
      float m = -CUDART_INF_F, l = 0.f;
      bool ok = true;
      for (int i = a; i < z; ++i, ++sc, ++tile) {
        const int j0 = pf_key(u, i);
        ok = __all_sync(0xffffffffu, pf_wait(&sh.s_full[s], sc & 1u, Ctl{ctl.abort, p.status, p.timeout_ns * idle}, 20 + s));
        if (!ok) break;
        idle = 1;
        free_place(2 * tile);
        // d 128: that S was issued behind the last tile's P V
        if (!kSepP && i > a) free_place(2 * tile - 1);
        if (!Q4 && i + 1 == z && lane == 0 && quad == 0) ptx::mbar_arrive(&sh.q_empty[s]);
        ptx::tc_fence_after();
        float x[128];
#pragma unroll
        for (int b = 0; b < 4; ++b) ptx::tmem_ld32f(tS + 32 * b, &x[32 * b]);
        const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&sh.bad[tile & 15u]);
        const bool part = j0 + 127 > hi || (j0 < lo && j0 + 127 >= p.sink) || bad != 0u;
        const bool any_part = __any_sync(0xffffffffu, part);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int b = 0; b < 4; ++b) ptx::reg_fence32f(&x[32 * b]);
        if (kSepP) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.s_free[s]);
        }
        if (SCORE == SCORE_SOFTCAP) {
          // x = cap log2(e) tanh(s scale / cap): a polynomial while every |s| of the warp is in
          // its range, else 1 - 2 / (1 + e^2y), whose rounding costs 2^-20 cap whatever |s| is.
          // The warp's scores are other rows', other sequences' and unseen keys' too, so with a
          // cap whose 2^-20 would show (kPfCapAll) each score takes the form of its own range.
          float am[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 128; c += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) am[q] = ptx::max3(am[q], fabsf(x[c + q]), fabsf(x[c + 4 + q]));
          const float amax = fmaxf(fmaxf(am[0], am[1]), fmaxf(am[2], am[3])) * rf;
          if (__all_sync(0xffffffffu, amax <= p.sc_smax)) {
            const float2 sq0 = make_float2(p.sc_q[0], p.sc_q[0]), sq1 = make_float2(p.sc_q[1], p.sc_q[1]);
            const float2 sq2 = make_float2(p.sc_q[2], p.sc_q[2]), sq3 = make_float2(p.sc_q[3], p.sc_q[3]);
            const float2 rf2 = make_float2(rf, rf);
#pragma unroll
            for (int c = 0; c < 128; c += 2) {
              float2 sv = make_float2(x[c], x[c + 1]);
              if (Q4) sv = ptx::mul2(sv, rf2);
              const float2 y = ptx::mul2(sv, sv);
              float2 q = ptx::fma2(sq3, y, sq2);
              q = ptx::fma2(q, y, sq1);
              q = ptx::fma2(q, y, sq0);
              const float2 v = ptx::mul2(sv, q);
              x[c] = v.x;
              x[c + 1] = v.y;
            }
          } else {
            const float arg = p.cap_arg * rf;
            auto exact = [&](float v) {
              return fmaf(-2.0f * p.softcap, ptx::rcp(1.0f + ptx::ex2(v * arg)), p.softcap);
            };
            if (p.softcap <= kPfCapAll * kLog2e) {
#pragma unroll
              for (int c = 0; c < 128; ++c) x[c] = exact(x[c]);
            } else {
#pragma unroll
              for (int c = 0; c < 128; ++c) {
                const float sv = Q4 ? x[c] * rf : x[c], y = sv * sv;
                const float v = sv * fmaf(fmaf(fmaf(p.sc_q[3], y, p.sc_q[2]), y, p.sc_q[1]), y, p.sc_q[0]);
                const float w = exact(x[c]);
                x[c] = fabsf(sv) <= p.sc_smax ? v : w;
              }
            }
          }
        } else if (SCORE == SCORE_ALIBI) {
          // x = scale s + slope (j - pos), in log2 units
          const float2 sc2 = make_float2(p.scale_log2 * rf, p.scale_log2 * rf), sl2 = make_float2(slope2, slope2);
          const float off = slope2 * static_cast<float>(j0 - pos);
          const float2 off2 = make_float2(off, off);
#pragma unroll
          for (int c = 0; c < 128; c += 2) {
            const float2 t = ptx::fma2(make_float2(static_cast<float>(c), static_cast<float>(c + 1)), sl2, off2);
            const float2 v = ptx::fma2(make_float2(x[c], x[c + 1]), sc2, t);
            x[c] = v.x;
            x[c + 1] = v.y;
          }
        }
        if (__builtin_expect(any_part, 0)) {
          // 32 keys at a time as a word of bits: below hi, and from lo on or a sink
          const int chi = hi - j0, clo = lo - j0, csk = (p.window ? p.sink : 0) - j0;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            uint32_t w = pf_low_bits(chi + 1 - 32 * b) & (~pf_low_bits(clo - 32 * b) | pf_low_bits(csk - 32 * b));
            if (bad) w &= ~(((bad >> (8 * b) & 1u) ? 0xffffu : 0u) | ((bad >> (8 * b) & 2u) ? 0xffff0000u : 0u));
            if (!__any_sync(0xffffffffu, w != 0xffffffffu)) continue;
#pragma unroll
            for (int c = 0; c < 32; ++c) x[32 * b + c] = w & (1u << c) ? x[32 * b + c] : -CUDART_INF_F;
          }
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) mx[q] = fmaxf(x[q], x[4 + q]);
#pragma unroll
        for (int c = 8; c < 128; c += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = ptx::max3(mx[q], x[c + q], x[c + 4 + q]);
        const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * xmul;
        // the reference maximum is raised only by more than 8 (in log2 units)
        const float m_new = fmaxf(m, tmax);
        const bool raise = m_new > m + kRescaleThreshold || (m == -CUDART_INF_F && m_new != -CUDART_INF_F);
        const bool any_raise = __any_sync(0xffffffffu, raise);
        float alpha = 1.f;
        if (__builtin_expect(any_raise, 0)) {
          alpha = raise ? ptx::ex2(m - m_new) : 1.f;
          m = raise ? m_new : m;
          l *= alpha;
        }
        const float sub = (Q4 ? static_cast<float>(kPfLift) : 0.f) - (m == -CUDART_INF_F ? 0.f : m);
        const float2 negm = make_float2(sub, sub), xm2 = make_float2(xmul, xmul);
        // P and O may change once the previous P V is done (d 128: it was, before this S)
        if (kSepP && i > a) {
          ok = __all_sync(0xffffffffu, pf_wait(&sh.pv_done[s], (sc - 1) & 1u, ctl, 24 + s));
          if (!ok) break;
          free_place(2 * tile - 1);
        }
        ptx::tc_fence_after();
        if (__builtin_expect(i > a && any_raise, 0)) {
          // a few columns at a time: the row's scores hold most registers
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            ptx::tmem_ld16(tO + c, o);
            ptx::tmem_ld_wait();
            ptx::reg_fence16(o);
#pragma unroll
            for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
            ptx::tmem_st16(tO + c, o);
          }
        }
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint32_t pk[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const float2 arg = ptx::fma2(make_float2(x[b * 32 + 2 * q], x[b * 32 + 2 * q + 1]), xm2, negm);
            const float2 pv = make_float2(ptx::ex2(arg.x), ptx::ex2(arg.y));
            ls[q & 1] = ptx::add2(ls[q & 1], pv);
            pk[q] = Q4 ? pf_pack_f16(pv.x, pv.y) : ptx::pack_bf16x2(pv.x, pv.y);
          }
          ptx::tmem_st16(tP + b * 16, pk);
          if (b & 1) {
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(b == 1 ? &sh.p_lo[s] : &sh.p_hi[s]);
          }
        }
        const float2 lsum = ptx::add2(ls[0], ls[1]);
        l += lsum.x + lsum.y;
      }
      if (!ok) break;
      // a partial result: of a unit that an earlier block began (0), or that a later one ends (1)
      const bool whole = a == 0 && z == u.count;
      rest = Rest{m, l, whole ? static_cast<int64_t>(u.tok0 + tok)
                              : (static_cast<int64_t>(blockIdx.x) * 2 + (a > 0 ? 0 : 1)) * 2 + s,
                  tile - 1, hq, live, whole};
      have_rest = true;
      ++units;
    }
  } else if constexpr (Q4) {
    // -------------------------------------- 4 bits: Q, K and V tiles in fp16
    ptx::setmaxnreg_dec<L::LOAD_REGS>();
    const int r = tid - 384;  // key row of the tile
    const int row_off = (r >> 3) * L::GROUP + (r & 7) * 128;
    constexpr int W = D / 32;   // 16-byte words of a row's codes
    uint32_t e = 0, tile = 0;
    const uint32_t ring = ptx::smem_u32(smem + L::OFF_RING);
    each_unit([&](const PfUnit& u, int a, int z) {
      uint4 kc[W], vc[W];
      uint32_t ks[D / 64], vs[D / 64];
      bool bad = false;
      // this row's page for tile i; -1: negative in the table, -2: no row of the unit sees it
      auto lookup = [&](int i) -> int {
        const int j = pf_key(u, i) + r;
        return i < z && pf_seen(p, u, j) ? max(__ldg(p.table + u.b * p.table_stride + (j >> shift)), -1) : -2;
      };
      auto in_pool = [&](int page) { return page >= 0 && page < p.c.num_pages; };
      auto load_k = [&](int i, int page) {
        if (in_pool(page)) {
          const int64_t slot = ((static_cast<int64_t>(page) * p.c.Hkv + u.h) << shift) + ((pf_key(u, i) + r) & page_mask);
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.c.k) + slot * (D / 2));
#pragma unroll
          for (int q = 0; q < W; ++q) kc[q] = __ldg(src + q);
          const uint32_t* sc = reinterpret_cast<const uint32_t*>(p.c.ks + slot * (D / 16));
#pragma unroll
          for (int q = 0; q < D / 64; ++q) ks[q] = __ldg(sc + q);
        } else {
#pragma unroll
          for (int q = 0; q < W; ++q) kc[q] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int q = 0; q < D / 64; ++q) ks[q] = 0u;
        }
      };
      auto load_v = [&](int i, int page) {
        if (in_pool(page)) {
          const int64_t run = (static_cast<int64_t>(page) * p.c.Hkv + u.h) << shift;
          const int at = (pf_key(u, i) + r) & page_mask;
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.c.v) + (run + at) * (D / 2));
#pragma unroll
          for (int q = 0; q < W; ++q) vc[q] = __ldg(src + q);
          const uint8_t* sc = p.c.vs + run * (D / 16) + at;
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            uint32_t w = 0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) w |= static_cast<uint32_t>(__ldg(sc + (static_cast<int64_t>(4 * q + k) << shift))) << (8 * k);
            vs[q] = w;
          }
        } else {
#pragma unroll
          for (int q = 0; q < W; ++q) vc[q] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int q = 0; q < D / 64; ++q) vs[q] = 0u;
        }
      };
      // row r of a tile: 16 bytes (8 channels) at a time to their swizzled places
      auto put = [&](int st, const uint4 (&c)[W], const uint32_t (&s8)[D / 64]) {
        const uint32_t base = ring + st * L::TILE + row_off;
#pragma unroll
        for (int q = 0; q < W; ++q) {
          const uint32_t w[4] = {c[q].x, c[q].y, c[q].z, c[q].w};
          // channels 32 q ..: two blocks of 16
          const uint32_t two = cvt4::from_e4m3x2((s8[q / 2] >> (16 * (q & 1))) & 0xffffu);
          const uint32_t s0 = __byte_perm(two, 0u, 0x1010), s1 = __byte_perm(two, 0u, 0x3232);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t hv[4];
            cvt4::from_e2m1x8(w[k], hv);
            const uint32_t sc = k < 2 ? s0 : s1;
            const int piece = (q * 4 + k) & 7, half = (q * 4 + k) >> 3;
            st_shared128(base + half * 1024 + ((piece ^ (r & 7)) << 4), cvt4::hmul2(hv[0], sc), cvt4::hmul2(hv[1], sc),
                         cvt4::hmul2(hv[2], sc), cvt4::hmul2(hv[3], sc));
          }
        }
      };
      int page = lookup(a), page1 = lookup(a + 1);
      load_k(a, page);
      load_v(a, page);
      for (int i = a; i < z; ++i, ++tile, e += 2) {
        // page: this tile's; page1: the next one's
        const int page2 = lookup(i + 2);
        bad = page != -2 && !in_pool(page);
        const uint32_t bb = __ballot_sync(0xffffffffu, bad);
        if (lane == 0) {
          if (bb) atomicOr(p.status, 2u);
          reinterpret_cast<uint8_t*>(&sh.bad[tile & 15u])[warp - 12] =
              static_cast<uint8_t>(((bb & 0xffffu) ? 1u : 0u) | ((bb >> 16) ? 2u : 0u));
        }
        const int sk = static_cast<int>(e % NS), sv = static_cast<int>((e + 1) % NS);
        if (!__all_sync(0xffffffffu, pf_wait(&sh.kv_empty[sk], ((e / NS) & 1u) ^ 1u, ctl, 2))) return false;
        put(sk, kc, ks);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        const bool skip = p.dbg_skip_tile >= 0 && blockIdx.x == 0 && static_cast<int>(tile) == p.dbg_skip_tile;
        if (lane == 0 && !skip) ptx::mbar_arrive(&sh.kv_full[sk]);
        if (i + 1 < z) load_k(i + 1, page1);
        if (!__all_sync(0xffffffffu, pf_wait(&sh.kv_empty[sv], (((e + 1) / NS) & 1u) ^ 1u, ctl, 2))) return false;
        put(sv, vc, vs);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.kv_full[sv]);
        if (i + 1 < z) load_v(i + 1, page1);
        page = page1;
        page1 = page2;
      }
      return true;
    });
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// The rows behind the last sequence, spread over all threads of the grid: they belong to
// no unit, and nothing else of the call writes them.
template <int D>
__device__ __forceinline__ void fill_rest(const PrefillParams& p) {
  const int64_t last = min(max(__ldg(p.seq_offsets + p.B), 0), p.T);
  const int64_t pieces = (p.T - last) * p.Hq * (D / 8);  // of 8 channels
  const int64_t all = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < pieces; i += all) {
    const int64_t pair = i / (D / 8), row = last + pair / p.Hq, h = pair % p.Hq;
    const int c = static_cast<int>(i % (D / 8)) * 8;
    if (p.fill & FL_FILL_OUT)
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + row * p.o_t + h * p.o_h + c) = make_uint4(0u, 0u, 0u, 0u);
    if ((p.fill & FL_FILL_LSE) && c == 0) p.lse[row * p.Hq + h] = -CUDART_INF_F;
  }
}

// Joins the partial results of the units that pieces share: 8 blocks of 32 rows
// for every border between pieces; the first border inside of a unit does it.
template <int D>
__global__ void __launch_bounds__(128) paged_prefill_merge_kernel(const __grid_constant__ PrefillParams p) {
  // under the end of the first kernel, which began when all before it had ended
  if (p.fill) fill_rest<D>(p);
  ptx::wait_prerequisites();
  const int border = 1 + blockIdx.x / 8, part = blockIdx.x % 8;
  if (border >= p.grid) return;
  const int32_t* rec = p.rec + static_cast<int64_t>(border) * 8;
  if (!rec[0] || rec[4] != border - 1) return;
  const int s = part >> 2, r = (part & 3) * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  const int rtok = r / p.G, tok = s * p.RT + rtok;
  if (rtok >= p.RT || tok >= rec[2]) return;
  const int hq = rec[3] * p.G + r - rtok * p.G;
  const int last = rec[5];
  auto at = [&](int piece) { return (static_cast<int64_t>(piece) * 2 + (piece == border - 1 ? 1 : 0)) * 2 + s; };
  // one pass with a running maximum, so that a piece's log-sum-exp and output come
  // in one trip to memory; kJoin pieces at once
  constexpr int C = D / 16;                // float4 of this thread
  constexpr int kJoin = D == 64 ? 4 : 2;
  float4 o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -CUDART_INF_F, sum = 0.f;
  for (int i0 = border - 1; i0 <= last; i0 += kJoin) {
    float l[kJoin];
    float4 v[kJoin][C];
#pragma unroll
    for (int k = 0; k < kJoin; ++k) {
      const bool ok = i0 + k <= last;
      const int64_t piece = at(ok ? i0 + k : last);
      l[k] = p.lpart[piece * 128 + r];
      const float4* src = reinterpret_cast<const float4*>(p.opart) + (piece * (D / 4) + w * C) * 128 + r;
#pragma unroll
      for (int c = 0; c < C; ++c) v[k][c] = src[c * 128];
      if (!ok) l[k] = -CUDART_INF_F;
    }
    float m_new = m;
#pragma unroll
    for (int k = 0; k < kJoin; ++k) m_new = fmaxf(m_new, l[k]);
    const float ref = m_new == -CUDART_INF_F ? 0.f : m_new;
    const float old = ptx::ex2(m - ref);  // of nothing yet: 0
    m = m_new;
    sum *= old;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = make_float4(o[c].x * old, o[c].y * old, o[c].z * old, o[c].w * old);
#pragma unroll
    for (int k = 0; k < kJoin; ++k) {
      const float wt = ptx::ex2(l[k] - ref);
      sum += wt;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        o[c].x = fmaf(v[k][c].x, wt, o[c].x);
        o[c].y = fmaf(v[k][c].y, wt, o[c].y);
        o[c].z = fmaf(v[k][c].z, wt, o[c].z);
        o[c].w = fmaf(v[k][c].w, wt, o[c].w);
      }
    }
  }
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
  const int64_t row = static_cast<int64_t>(rec[1] + tok);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * p.o_t + hq * p.o_h + w * (D / 4);
#pragma unroll
  for (int c = 0; c < C; c += 2)
    *reinterpret_cast<uint4*>(out + 4 * c) =
        make_uint4(ptx::pack_bf16x2(o[c].x * inv, o[c].y * inv), ptx::pack_bf16x2(o[c].z * inv, o[c].w * inv),
                   ptx::pack_bf16x2(o[c + 1].x * inv, o[c + 1].y * inv), ptx::pack_bf16x2(o[c + 1].z * inv, o[c + 1].w * inv));
  if (w == 0 && p.lse) p.lse[row * p.Hq + hq] = (sum > 0.f || sum != sum ? m + __log2f(sum) : -CUDART_INF_F) * kLn2;
}

template <int FMT, int D, int SCORE>
cudaError_t launch_prefill_score(const CUtensorMap* maps, const PrefillParams& p, cudaStream_t s) {
  using L = PfLayout<FMT, D>;
  auto kern = paged_prefill_kernel<FMT, D, SCORE>;
  static OncePerDevice once;
  const cudaError_t checked = on_this_device(once, [&]() {
    cudaFuncAttributes a{};
    cudaError_t e = cudaFuncGetAttributes(&a, kern);
    if (e != cudaSuccess) return e;
    // the register split needs these at launch
    if (a.numRegs != L::LAUNCH_REGS) return cudaErrorInvalidDeviceFunction;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
  });
  if (checked != cudaSuccess) return checked;
  kern<<<p.grid, L::THREADS, L::SMEM, s>>>(maps[0], maps[1], maps[2], p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (p.grid < 2 && !p.fill)) return e;
  const unsigned borders = p.grid < 2 ? 1u : static_cast<unsigned>(p.grid - 1);
  return launch_chained(paged_prefill_merge_kernel<D>, borders * 8u, 128u, 0, s, p);
}

template <int FMT, int D>
cudaError_t launch_prefill(int score_mod, const CUtensorMap* maps, const PrefillParams& p, cudaStream_t s) {
  switch (score_mod) {
    case SCORE_NONE: return launch_prefill_score<FMT, D, SCORE_NONE>(maps, p, s);
    case SCORE_ALIBI: return launch_prefill_score<FMT, D, SCORE_ALIBI>(maps, p, s);
    case SCORE_SOFTCAP: return launch_prefill_score<FMT, D, SCORE_SOFTCAP>(maps, p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace fl
