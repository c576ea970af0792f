// Attention of packed new tokens over a paged cache (bf16 or f16, d = 128), causal at
// the tokens' places in their sequences, with grouped heads: from one token a
// sequence (decode) to long pieces of a prompt, mixed in one call.
//
//   o_r = sum_j softmax_j(q_r . k_j * scale) v_j over the keys j that row r sees,
//   lse_r = ln sum_j exp(q_r . k_j * scale),
// computed tile by tile with the online softmax, as in fwd_tc.cu.
//
// Rows.  The G = Hq / Hkv query heads of a key head read the same keys, so an item's
// rows are (token, head of the group) pairs: a tile of 128 rows holds 128 / G tokens
// of one sequence, and a K/V tile is loaded once for all of them.  An item is up to
// two row tiles of one (sequence, key head):
//   two tiles  -- both stream the same key tiles, one MMA/softmax ping-pong (as in
//                 fwd_tc.cu);
//   one tile   -- (single tokens, short or last pieces) the two softmax warpgroups
//                 take the even and the odd key tiles of the same rows, so the
//                 S -> softmax -> PV chain of one key tile overlaps the next one's;
//                 the epilogue joins the two states.
//
// Work split.  One persistent CTA per SM.  Items and their key tiles cost units
// (kTileUnits below); all items laid end to end are cut into equal runs of units, one per CTA,
// whatever the lengths: a long sequence with few rows is spread over many CTAs,
// many short ones share a CTA.  An item cut by a run's edge leaves normalised float32
// partials and their logsumexp in the workspace, and combine_kernel joins them (in
// the order of the keys: the result does not depend on timing).  Every CTA works the
// split out for itself from cu_tokens and seqlens, so no length crosses to the host.
//
// Cache.  K and V tiles come by TMA, one box per block and 64-column half; blocks
// with no visible key are not read.  Rows of a V tile outside the item's keys (a
// block's unused tail, a skipped block) stay out of the product: steps of 16 keys
// without a key are not issued, other such rows are zeroed in shared memory before
// the MMA, since their weights are zero but 0 * NaN is not.
//
// What bounds it, and what it measured (a run of calls, or a replayed graph of them, which take
// the same time; at 1965 MHz, the first 0.1 s or so, before the card's power limit of 1000 W lowers
// the clock; in brackets after a second of such calls, with the clock that was left):
//   2048 tokens of a prompt at 14336 .. 16383, 32 heads over 8: the tensor cores through
//     the S -> softmax -> PV chain of a two-tile item, as in fwd_tc.cu; 429 us, 1200 TFLOP/s
//     (508 us, 1014 TFLOP/s at 1620 MHz);
//   64 single tokens, 512 .. 8192 keys, 32 heads over 8: the cache's bytes; 195 us, 5.8 TB/s
//     (88 % of the copy rate; 230 us at 1515 MHz); an item's edges (Q, first S, last PV,
//     epilogue) cost as much as one or two key tiles, of the 118 a CTA takes here;
//   24 x 5 tokens, 100 .. 4000 keys, 16 heads over 16: 90 us, 5.3 TB/s (80 %), shorter items
//     (102 us at 1605 MHz);
//   512 single tokens over 600 keys: 316 us, 4.0 TB/s (61 %; 338 us at 1845 MHz): five key tiles
//     an item, the edges' chains no longer hidden by the next item's loads (two stages a ring);
//   17 ragged pieces under a window of 1024: 95 us, 515 TFLOP/s (102 us at 1830 MHz): a third of
//     the key tiles are partly masked, and a CTA has 27 in three or four items to level out;
//   8192 tokens of a fresh prompt, 32 heads over 8: 475 us, 1157 TFLOP/s (562 us at 1640 MHz);
//   one token over 512 keys: 14.2 us: launch, planning, a key tile's latency, the join.
// The kernel's text is kept near 90 KB with single issue sites and loops that are not
// unrolled: at 225 KB the sixteen warps' roles displaced one another in the instruction cache.
#include <atomic>

#include "cache_ops.h"
#include "common.cuh"
#include "dependent.cuh"
#include "kernels.h"

namespace fa {
namespace ext {

constexpr int BM = 128;                     // rows per tile
constexpr int BN = 128;                     // keys per tile
constexpr int D = 128;
constexpr int NS = 2;                       // stages of the K ring and of the V ring
constexpr int TILE_BYTES = BM * D * 2;
constexpr int HALF_BYTES = TILE_BYTES / 2;  // one 64-column half (128-byte rows, swizzled)
constexpr int NUM_THREADS = 512;
constexpr int WG_THREADS = 128;
constexpr int EPI_WG = 2;
constexpr int PLAN_WARP = 12;
constexpr int MMA_WARP = 13;
constexpr int K_WARP = 14;                  // Q and K tiles
constexpr int V_WARP = 15;                  // V tiles
constexpr int NP = 8;                       // pieces in flight between the planner and the other warps
constexpr int kPieceReaders = 15;           // warps that read a piece: MMA, K, V, 8 softmax, 4 epilogue
constexpr int kSoftmaxRegs = 184;
constexpr int kEpilogueRegs = 72;
constexpr int kOtherRegs = 72;
constexpr int kLaunchRegs = 128;            // 65536 / NUM_THREADS: what the split draws on
static_assert(2 * WG_THREADS * kSoftmaxRegs + WG_THREADS * kEpilogueRegs + WG_THREADS * kOtherRegs <=
                  NUM_THREADS * kLaunchRegs,
              "register split exceeds the launch budget");
constexpr float kRescaleThreshold = 8.0f;   // log2 units: P stays below 2^8
// Costs in units of about 0.7 us.  A key tile of a one-tile item took 1.3-1.5 us (its bytes
// at the memory's rate), of a two-tile item 1.8-2.9 us; weights of 2 and 3 served mixed
// batches no better than 2 and 2 (ragged batch without a window 145 and 136 us), and equal
// ones let a run be a single tile.  An item itself: 3 and 5 (4 and 7: 2 % slower on single
// tokens, 2 and 4: 2 % slower on ragged batches).
constexpr int kTileUnits = 2, kItemUnits1 = 3, kItemUnits2 = 5;  // items of one, two row tiles
// A CTA takes at least so many.  Every run inside an item then holds the first unit of some
// key tile, so that each of the CTAs between an item's first and last has a piece of it
// (combine_kernel reads them all).
constexpr int kMinUnits = kTileUnits;
// Items of a sequence that one lane of the planner adds up; more take the whole warp.
constexpr int kLaneItems = 16;
// The planner keeps the units of so many sequences; it works those of more out twice.
constexpr int kPlanSeqs = 1024;
// Epilogue: an item of so many rows at most (one warp's) has its first finished slot put
// aside in shared memory.
constexpr int kAsideRows = 32;

// A wait gives up after so many cycles.
constexpr unsigned kWaitCycles = 2000000000u;

// A run of key tiles [j0, j1) of one item, as the planner hands it to the other warps.
// Arrays go by slot: a one-tile item's key tiles take the slots in turn, going on from the
// item before; a two-tile item's row tiles have one each.
struct Piece {
  int j0, j1;
  int single;                  // one row tile
  int stop;                    // no more pieces
  int b, kvh;
  int key_lo, key_hi;          // keys of the sequence that some row of the item sees
  int tok0, ntok;              // the item's tokens in the packed batch
  int part;                    // workspace slot of the partial result, -1: the piece is the whole item
  int tile0;                   // the CTA's number of key tile j0: its place in the rings
  int slot0;                   // a one-tile item's slot for key tile j0
  int pad;
  int first[2], end[2];        // key tiles of the slot: first, end; every second one of a one-tile item
  int rows[2];                 // rows of the slot's row tile that hold a token
  int pos[2];                  // position of its first token
  int all_lo[2], all_hi[2];    // keys that every row of it sees
  __device__ __forceinline__ bool any(int t) const { return first[t] < end[t]; }
};

// Dynamic shared memory, 1024-byte aligned: Q tiles, K ring, V ring, then kAsideRows rows
// of float32 that the epilogue puts aside.
constexpr int kKOff = 2 * TILE_BYTES;
constexpr int kVOff = kKOff + NS * TILE_BYTES;
constexpr int kAsideOff = kVOff + NS * TILE_BYTES;
constexpr size_t kSmemBytes = kAsideOff + kAsideRows * D * 4 + 1024;

// Heads per key head and tokens per row tile, 128 / G.
struct Geo {
  int G, tpt;
};

struct Seq {
  int tok0, nq, n;  // first packed token, new tokens, keys
};
// A CTA's run of units [begin, end) of `length` (the last one's may be shorter), and the
// sequence in which it starts: its number, units before it and units per key head.
struct Run {
  long long begin, end, length;
  long long before, per_head;
  int b;
};

// Everything else sits in static shared memory, whose addresses are constants: pointers
// to it cost no registers.
struct Ctl {
  alignas(16) uint32_t bad[4][BN / 32];  // keys of a tile whose block lies outside the pool (read as uint4)
  Piece piece[NP];
  // Barriers, by the arrivals that they count: one, a warpgroup's, the piece readers'.
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[NS], k_empty[NS];
  uint64_t v_full[NS], v_empty[NS];
  uint64_t s_full[2], o_full[2];
  uint64_t piece_full[NP];
  uint64_t mma_done;
  uint64_t p_full[2], o_free[2];
  uint64_t st_full[2], st_empty[2];
  uint64_t piece_empty[NP];
  float stat_m[2][BM], stat_l[2][BM];
  Run run;
  long long units[kPlanSeqs];        // per key head, of each sequence
  Geo geo;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(offsetof(Ctl, bad) % alignof(uint4) == 0 && alignof(Ctl) % alignof(uint4) == 0, "bad is read in 16-byte pieces");
static_assert(kSmemBytes + sizeof(Ctl) + 64 <= 227 * 1024, "shared memory");

__device__ __forceinline__ Seq seq_of(const ExtendArgs& a, int b) {
  Seq s;
  if (a.cu_tokens == nullptr) {
    s.tok0 = b;
    s.nq = 1;
  } else {
    s.tok0 = min(max(a.cu_tokens[b], 0), a.T);
    s.nq = min(max(a.cu_tokens[b + 1], s.tok0), a.T) - s.tok0;
  }
  s.n = min(max(a.seqlens[b], 0), a.cap);
  return s;
}

// Keys [lo, hi) that tokens at positions pf .. pl of a sequence with n keys see in all
// (empty: lo = hi = 0).
__device__ __forceinline__ void key_range(const ExtendArgs& a, int pf, int pl, int n, int& lo, int& hi) {
  hi = a.causal ? min(n, pl + 1) : n;
  lo = a.window > 0 ? max(0, pf - a.window + 1) : 0;
  if (hi <= lo) lo = hi = 0;
}
// Key tiles of item p (tokens [2 tpt p, 2 tpt (p + 1)) of the sequence).
__device__ __forceinline__ int item_tiles(const ExtendArgs& a, const Geo& g, const Seq& s, int p, int& lo, int& hi) {
  const int i0 = p * 2 * g.tpt, i1 = min(s.nq, i0 + 2 * g.tpt);
  key_range(a, s.n - s.nq + i0, s.n - s.nq + i1 - 1, s.n, lo, hi);
  return hi > lo ? (hi + BN - 1) / BN - lo / BN : 0;
}
// Units of item p of the sequence ahead of its first key tile, and in all.
__device__ __forceinline__ int head_cost(const Geo& g, const Seq& s, int p) {
  return s.nq - p * 2 * g.tpt > g.tpt ? kItemUnits2 : kItemUnits1;
}
__device__ __forceinline__ int item_units(const ExtendArgs& a, const Geo& g, const Seq& s, int p) {
  int lo, hi;
  return head_cost(g, s, p) + item_tiles(a, g, s, p, lo, hi) * kTileUnits;
}
__device__ __forceinline__ int items_of(const Geo& g, int nq) { return (nq + 2 * g.tpt - 1) / (2 * g.tpt); }

// Units of all items of one key head of each lane's sequence (lane: its own `s`, nq = 0
// for none).  Sequences with many items are summed by the whole warp.
__device__ __forceinline__ long long head_units(const ExtendArgs& a, const Geo& g, const Seq& s, int lane) {
  const int np = items_of(g, s.nq);
  long long u = 0;
  if (np <= kLaneItems) {
#pragma unroll 1
    for (int p = 0; p < np; ++p) u += item_units(a, g, s, p);
  }
  unsigned many = __ballot_sync(0xffffffffu, np > kLaneItems);
#pragma unroll 1
  while (many) {
    const int src = __ffs(many) - 1;
    many &= many - 1;
    const Seq o{__shfl_sync(0xffffffffu, s.tok0, src), __shfl_sync(0xffffffffu, s.nq, src),
                __shfl_sync(0xffffffffu, s.n, src)};
    const int onp = items_of(g, o.nq);
    long long v = 0;
#pragma unroll 1
    for (int p = lane; p < onp; p += 32) v += item_units(a, g, o, p);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
    if (lane == src) u = v;
  }
  return u;
}

// The piece's fields by slot; pos0: the position of its first token.
__device__ __forceinline__ void fill_slots(const ExtendArgs& a, const Geo& g, Piece& p, int pos0) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int i0 = p.single ? 0 : t * g.tpt, i1 = min(p.ntok, i0 + g.tpt);
    p.rows[t] = (i1 - i0) * g.G;
    p.pos[t] = pos0 + i0;
    int lo = p.key_lo, hi = p.key_hi;
    p.all_lo[t] = lo;
    p.all_hi[t] = hi;
    if (a.causal) {
      hi = min(hi, pos0 + i1);
      p.all_hi[t] = min(p.all_hi[t], pos0 + i0 + 1);
    }
    if (a.window > 0) {
      lo = max(lo, pos0 + i0 - a.window + 1);
      p.all_lo[t] = max(p.all_lo[t], pos0 + i1 - a.window);
    }
    if (p.single) {
      p.first[t] = p.j0 + (t ^ p.slot0);
      p.end[t] = p.j1;
    } else {
      p.first[t] = hi > lo ? max(p.j0, lo / BN) : p.j0;
      p.end[t] = hi > lo ? min(p.j1, (hi + BN - 1) / BN) : p.j0;
    }
  }
}

__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | (2u << 29); }

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void commit_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// S = Q K^T and O += P V for one tile; operand layouts as in fwd_tc.cu.
template <class T>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t q_addr, uint32_t k_addr) {
  constexpr uint32_t h = HALF_BYTES >> 4, idesc = idesc_f32acc<T>(BM, BN, 0, 0);
  mma8_ss<idesc, 2, 4, 6, h, h + 2, h + 4, h + 6>(d_tmem, desc_lo(q_addr, 16), desc_lo(k_addr, 16), desc_hi(1024), 0u);
}
template <class T>
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_addr, uint32_t accumulate) {
  constexpr uint32_t idesc = idesc_f32acc<T>(BM, D, 0, 1), col_step = 8, v_step = (16 * 128) >> 4;
  mma8_ts<idesc, col_step, v_step>(d_tmem, p_tmem, desc_lo(v_addr, HALF_BYTES), desc_hi(1024), accumulate);
}

// ceil(a / b) for 0 <= a < 2^48, 0 < b < 2^16, by two 32-bit divisions (a 64-bit one takes
// about 150 instructions, and a launch's first microseconds are one warp's chain of them).
__device__ __forceinline__ long long div_up(long long a, unsigned b) {
  const unsigned hi = static_cast<unsigned>((a + b - 1) >> 16), lo = static_cast<unsigned>(a + b - 1) & 0xffffu;
  const unsigned q = hi / b;
  return (static_cast<long long>(q) << 16) + ((hi - q * b) << 16 | lo) / b;
}
// This CTA's run, found by one warp, 32 sequences at a time.  The units of the first
// kPlanSeqs are kept for the second walk.  Out of line, and called ahead of the register
// split: its code runs once and stays away from the roles' loops.
__device__ __noinline__ void find_run(const ExtendArgs& a, Ctl& sm, int lane) {
  const Geo g{a.Hq / a.Hkv, BM / (a.Hq / a.Hkv)};
  long long total = 0, length = 0, begin = 0, before = 0;
#pragma unroll 1
  for (int walk = 0; walk < 2; ++walk) {
#pragma unroll 1
    for (int c = 0; c < a.B && (walk == 0 || before <= begin); c += 32) {
      long long units;
      if (walk == 1 && c < kPlanSeqs) {
        units = sm.units[c + lane];
      } else {
        Seq s{0, 0, 0};
        if (c + lane < a.B) s = seq_of(a, c + lane);
        units = head_units(a, g, s, lane);
        if (c < kPlanSeqs) sm.units[c + lane] = units;
      }
      const long long cost = units * a.Hkv;
      long long inc = cost;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, x);
        if (lane >= x) inc += o;
      }
      if (walk == 1 && before + inc - cost <= begin && begin < before + inc) {
        sm.run.before = before + inc - cost;
        sm.run.per_head = units;
        sm.run.b = c + lane;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (walk == 0) {
      total = before;
      before = 0;
      length = max(div_up(total, gridDim.x), static_cast<long long>(kMinUnits));
      begin = blockIdx.x * length;
    }
  }
  if (lane == 0) {
    sm.run.begin = begin;
    sm.run.end = min(total, begin + length);
    sm.run.length = length;
  }
  __syncwarp();
}

#define FA_TMEM_LD16(taddr, r)                                                                       \
  asm volatile(                                                                                      \
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"   \
      "%15}, [%16];"                                                                                 \
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),          \
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),      \
        "=r"(r[14]), "=r"(r[15])                                                                     \
      : "r"(taddr))

// One step of 16 keys of O += P V.
template <class T>
__device__ __forceinline__ void issue_pv_step(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_addr, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b64 bd;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 bd, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(p_tmem), "r"(desc_lo(v_addr, HALF_BYTES)), "r"(desc_hi(1024)), "r"(accumulate),
      "n"(idesc_f32acc<T>(BM, D, 0, 1))
      : "memory");
}

// 16 columns of a row's O, scaled and (both) joined with the other slot's; zero for a row
// without a key, whatever its O holds.
__device__ __forceinline__ void load_o16(uint32_t tO, uint32_t tO1, bool both, bool none, float f0, float f1, float (&o)[16]) {
  uint32_t r[16];
  FA_TMEM_LD16(tO, r);
  if (both) {
    uint32_t r1[16];
    FA_TMEM_LD16(tO1, r1);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = fmaf(__uint_as_float(r1[e]), f1, __uint_as_float(r[e]) * f0);
  } else {
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(r[e]) * f0;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] = none ? 0.f : o[e];
}

// The bounded wait of common.cuh for a whole warp, in fewer instructions: there are more
// than a dozen waits here.  (A suspend-time hint on try_wait, to leave the issue slots to the
// softmax warps, measured 3 % slower.)
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  bool ok = true;
  const unsigned t0 = static_cast<unsigned>(clock());
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    // About a second at the B200's clocks; the kernel's end reports it.
    if (*abort_flag || static_cast<unsigned>(clock()) - t0 > kWaitCycles) {
      *abort_flag = 1;
      ok = false;
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __noinline__ bool wait_out_of_line(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return wait_inline(bar, parity, abort_flag);
}
// One try in line, the loop in one place for all: the MMA warp's steps are a chain of such
// waits, most of them over already (5 drafted tokens 94 -> 90 us, ragged window 99 -> 95, 64
// single tokens 200 -> 195).  The softmax warps, whose registers a call does not fit, take
// wait_inline (a try ahead of its loop gained them nothing).
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_out_of_line(bar, parity, abort_flag);
}

// A warp's view of the planner's ring of pieces.  Pieces stay in shared memory until the
// warp releases them: what a role needs of one now and then is read there, since a
// spilled register costs a local load, and with this much shared memory in use little
// L1 is left to catch it (measured: 60 bytes of spills in the MMA and producer warps
// took a quarter of the kernel's time).
struct Pieces {
  Ctl* sm;
  volatile int* abort_flag;
  __device__ __forceinline__ const Piece& at(int i) const { return sm->piece[i % NP]; }
  // Waits for piece i; false at the end (or when the CTA gives up).
  template <bool INLINE = false>
  __device__ __forceinline__ bool wait(int i) const {
    const uint32_t bar = smem_u32(&sm->piece_full[i % NP]), parity = (i / NP) & 1;
    return (INLINE ? wait_inline(bar, parity, abort_flag) : wait_bar(bar, parity, abort_flag)) && !at(i).stop;
  }
  __device__ __forceinline__ void release(int i, int lane) const {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm->piece_empty[i % NP]));
  }
};

// Zeroes rows [r0, r1) of a V tile.  All lanes: sixteen to a row.
__device__ __forceinline__ void zero_v_rows(uint32_t v_addr, int r0, int r1, int lane) {
  const uint32_t dst = v_addr + (lane >> 3 & 1) * HALF_BYTES + (lane & 7) * 16;
#pragma unroll 1
  for (int r = r0 + (lane >> 4); r < r1; r += 2)
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + r * 128), "r"(0u) : "memory");
}
// Zeroes the rows of blocks outside the pool (bit r of `bad`).
__device__ __forceinline__ void zero_bad_rows(uint32_t v_addr, const uint32_t* bad, int lane) {
#pragma unroll 1
  for (int r = 0; r < BN; ++r)
    if (bad[r >> 5] >> (r & 31) & 1u) zero_v_rows(v_addr, r, r + 1, lane);
}

template <class T>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    extend_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ ExtendArgs args, int q_box_tokens) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl sm;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int wg = warp >> 2;
  {
    // One barrier a thread.
    uint64_t* bars = sm.q_full;
    constexpr int n1 = (offsetof(Ctl, p_full) - offsetof(Ctl, q_full)) / 8, n2 = (offsetof(Ctl, piece_empty) - offsetof(Ctl, q_full)) / 8;
    if (threadIdx.x < n2 + NP) {
      mbar_init(smem_u32(bars + threadIdx.x), threadIdx.x < n1 ? 1 : threadIdx.x < n2 ? WG_THREADS : kPieceReaders);
      fence_barrier_init();
    }
  }
  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    const int G = args.Hq / args.Hkv;
    sm.geo = Geo{G, BM / G};
  }
  if (warp == MMA_WARP) {
    tmem_alloc(smem_u32(&sm.tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == K_WARP && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // Everything before this overlaps the end of the kernel ahead in the stream.
  wait_for_previous_kernel();
  let_next_kernel_start();
  if (warp == PLAN_WARP) find_run(args, sm, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  volatile int* abort_flag = &sm.abort_flag;
  const Pieces pieces{&sm, abort_flag};
  // Each role reads these for itself: a value held across the roles is one register less
  // for the role that has none to spare.
  auto tiles_base = [&]() { return (smem_u32(smem_raw) + 1023u) & ~1023u; };
  auto geometry = [&]() { return Geo{*const_cast<volatile int*>(&sm.geo.G), *const_cast<volatile int*>(&sm.geo.tpt)}; };
  auto tmem_base = [&]() { return *const_cast<volatile uint32_t*>(&sm.tmem_base); };

  if (wg == 3) {
    regs_dec<kOtherRegs>();
    if (warp == PLAN_WARP) {
      // ---------------------------------------------------------- planner
      // Finds the run, walks it item by item, hands out its pieces and loads their Q tiles.
      const Geo geo = geometry();
      const uint32_t tiles = tiles_base();
      ExtendDesc open{0, 0, 0, -1};  // the item that begins here and ends in another CTA
      int ip = 0, tile0 = 0, slot0 = 0;  // pieces handed out, their key tiles, the next slot in turn
      int iq = 0;                    // pieces whose Q is on its way
      int nq0 = 0, nq1 = 0;          // Q tiles loaded, per slot
      bool ok = true;
      // A one-tile item uses one Q slot, in turn with the next one's, so that its Q tile is
      // there before the last item is done with its own.
      auto load_q = [&]() {
        const Piece& p = pieces.at(iq);
#pragma unroll 1
        for (int t = 0; t < (p.single ? 1 : 2); ++t) {
          if (!p.single && !p.any(t)) continue;
          const int qs = p.single ? iq & 1 : t;
          const int used = qs ? nq1++ : nq0++;
          if (used > 0) ok = wait_bar(smem_u32(&sm.q_empty[qs]), (used - 1) & 1, abort_flag);
          if (!ok) return;
          if (lane == 0) {
            const uint32_t bar = smem_u32(&sm.q_full[qs]), bytes = q_box_tokens * geo.G * 256;
            uint32_t dst = tiles + qs * TILE_BYTES;
            const int end = p.tok0 + min(p.ntok, (t + 1) * geo.tpt);
#pragma unroll 1
            for (int tok = p.tok0 + t * geo.tpt; tok < end; tok += q_box_tokens, dst += bytes / 2) {
              mbar_expect_tx(bar, bytes);
              tma_load_3d(dst, &tm_q, bar, 0, p.kvh * geo.G, tok);
              tma_load_3d(dst + HALF_BYTES, &tm_q, bar, 64, p.kvh * geo.G, tok);
            }
            mbar_arrive(bar);
          }
          __syncwarp();
        }
        ++iq;
      };
      const long long u_begin = sm.run.begin, u_end = sm.run.end, run = sm.run.length;
      int b = 0, h = 0, p = 0;       // the item: sequence, key head, number
      Seq s{0, 0, 0};
      long long u0 = u_end;          // its first unit (an empty run: past the end)
      auto next_item = [&]() {
        if (++p * 2 * geo.tpt < s.nq) return;
        p = 0;
        if (++h < args.Hkv) return;
        h = 0;
        // Sequences without new tokens have no items; the run ends before they run out.
#pragma unroll 1
        do {
          if (++b >= args.B) return;
          s = seq_of(args, b);
        } while (s.nq == 0);
      };
      if (u_begin < u_end) {
        b = sm.run.b;
        s = seq_of(args, b);
        const long long into = u_begin - sm.run.before, per_head = sm.run.per_head;
        // h = into / per_head, bit by bit where 32-bit division does not serve.
        if (into <= 0xffffffffLL) {
          if (into >= per_head) h = static_cast<int>(static_cast<unsigned>(into) / static_cast<unsigned>(per_head));
        } else {
#pragma unroll 1
          for (int bit = 1 << 30; bit > 0; bit >>= 1)
            if ((h | bit) * per_head <= into) h |= bit;
        }
        // The item of key head h in which the run starts, 32 items at a time.
        long long rem = into - h * per_head;
#pragma unroll 1
        for (const int np = items_of(geo, s.nq); p < np; p += 32) {
          int inc = p + lane < np ? item_units(args, geo, s, p + lane) : 0;
          const int own = inc;
#pragma unroll
          for (int x = 1; x < 32; x <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, x);
            if (lane >= x) inc += o;
          }
          const unsigned past = __ballot_sync(0xffffffffu, inc > rem);
          if (past) {
            const int at = __ffs(past) - 1;
            rem -= __shfl_sync(0xffffffffu, inc - own, at);
            p += at;
            break;
          }
          rem -= __shfl_sync(0xffffffffu, inc, 31);
        }
        u0 = u_begin - rem;
      }
      // One turn: the next piece of the run, or the end, goes out.
#pragma unroll 1
      for (bool stop = false; ok && !stop;) {
        int nt = 0, lo = 0, hi = 0, k0 = 0, k1 = 0;
        int head = 0;
        // To the next item with a key tile in the run.
#pragma unroll 1
        while (true) {
          stop = u0 >= u_end;
          if (stop) break;
          nt = item_tiles(args, geo, s, p, lo, hi);
          head = head_cost(geo, s, p);
          // Tile k of the item begins at unit t0 + k kTileUnits, and the run that holds this unit
          // takes it; unit u0 only says who writes an item without keys.
          const long long t0 = u0 + head;
          auto tile_at = [&](long long u) {
            const int x = static_cast<int>(min(max(u - t0, 0LL), static_cast<long long>(nt) * kTileUnits));
            return (x + kTileUnits - 1) / kTileUnits;
          };
          k0 = tile_at(u_begin);
          k1 = tile_at(u_end);
          if (k0 < k1) break;
          if (nt == 0 && u0 >= u_begin) {
            // No row of the item sees a key (an empty cache, more tokens than keys): written here.
            const int i0 = p * 2 * geo.tpt, rows = min(s.nq - i0, 2 * geo.tpt) * geo.G;
#pragma unroll 1
            for (int r = lane >> 4; r < rows; r += 2) {
              const int tok = r / geo.G;
              const long long at = static_cast<long long>(s.tok0 + i0 + tok) * args.Hq + h * geo.G + r - tok * geo.G;
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(args.o) + at * D + (lane & 15) * 8) = make_uint4(0u, 0u, 0u, 0u);
              if (args.lse != nullptr && (lane & 15) == 0) args.lse[at] = -INFINITY;
            }
          }
          u0 += head + static_cast<long long>(nt) * kTileUnits;
          next_item();
        }
        // A free place in the ring.  Q follows two pieces behind, that of the first two at once.
#pragma unroll 1
        while (ok && iq < (ip <= 2 ? ip : ip - 2)) load_q();
        if (ok && ip >= NP) ok = wait_bar(smem_u32(&sm.piece_empty[ip % NP]), ((ip / NP) - 1) & 1, abort_flag);
        if (!ok) break;
        Piece& out = sm.piece[ip % NP];
        if (stop) {
          out.stop = 1;
        } else {
          const bool single = s.nq - p * 2 * geo.tpt <= geo.tpt;
          if (!single) slot0 = 0;
          if (lane == 0) {
            const int i0 = p * 2 * geo.tpt;
            out.tok0 = s.tok0 + i0;
            out.ntok = min(s.nq - i0, 2 * geo.tpt);
            out.kvh = h;
            out.b = b;
            out.j0 = lo / BN + k0;
            out.j1 = lo / BN + k1;
            out.key_lo = lo;
            out.key_hi = hi;
            out.single = single;
            out.tile0 = tile0;
            out.slot0 = slot0;
            out.part = k0 == 0 && k1 == nt ? -1 : 2 * static_cast<int>(blockIdx.x) + (k0 == 0 ? 1 : 0);
            out.stop = 0;
            fill_slots(args, geo, out, s.n - s.nq + i0);
            if (k0 == 0 && k1 < nt) {
              // The run that holds the last tile's unit, which lies at or past this one's end.
              const long long past = u0 + head + (nt - 1LL) * kTileUnits - u_end;
              const int runs = run > past ? 0 : static_cast<int>(static_cast<unsigned>(past) / static_cast<unsigned>(run));
              open = ExtendDesc{out.tok0, out.ntok, h, static_cast<int>(blockIdx.x) + 1 + runs};
            }
          }
          tile0 += k1 - k0;
          if (single) slot0 = (slot0 + k1 - k0) & 1;
          u0 += head + static_cast<long long>(nt) * kTileUnits;
          next_item();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.piece_full[ip % NP]));
        ++ip;
      }
#pragma unroll 1
      while (ok && iq < ip - 1) load_q();
      if (lane == 0) args.desc[blockIdx.x] = open;
      if (nq0 > 0) mbar_wait_drain(smem_u32(&sm.q_full[0]), (nq0 - 1) & 1);
      if (nq1 > 0) mbar_wait_drain(smem_u32(&sm.q_full[1]), (nq1 - 1) & 1);
    } else if (warp == K_WARP || warp == V_WARP) {
      // ---------------------------------------------------------- K, V producers
      // A warp each, so that K tiles run ahead of the V tiles that wait for a softmax.
      // Lane l holds the tile's block-table entries l, l + 32, ..., fetched one tile ahead
      // (across items too); the boxes go out one after another from one elected lane.
      const uint32_t tiles = tiles_base();
      const bool is_k = warp == K_WARP;
      const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
      uint64_t* full = is_k ? sm.k_full : sm.v_full;
      uint64_t* empty = is_k ? sm.k_empty : sm.v_empty;
      const uint32_t ring = tiles + (is_k ? kKOff : kVOff);
      const int rows = min(1 << args.block_shift, BN);  // keys per box
      const int nblk = BN / rows;                       // blocks per tile: 1 .. 128
      // Does block `blk` of tile j hold keys of the item?
      auto wanted = [&](const Piece& w, int j, int blk) {
        const int key = j * BN + blk * rows;
        return blk < nblk && key < w.key_hi && key + rows > w.key_lo;
      };
      auto lookup = [&](const Piece& w, int j, int blk) {
        return wanted(w, j, blk) ? args.block_table[static_cast<long long>(w.b) * args.max_blocks + ((j * BN + blk * rows) >> args.block_shift)] : 0;
      };
      int n = 0;           // tiles loaded so far
      bool ok = true;
      // Loads tile j; `id`: this lane's entry of the tile's first 32 blocks (the rest, of
      // blocks of one or two keys, is looked up here).
      auto load_tile = [&](const Piece& p, int j, int id) {
        const int s = n % NS;
        if (n >= NS) ok = wait_bar(smem_u32(&empty[s]), ((n / NS) - 1) & 1, abort_flag);
        if (!ok) return;
        const uint32_t bar = smem_u32(&full[s]);
        // Tile n - 4 is done with these words: K's stage was that of tile n - 2, whose S
        // followed the PV of tile n - 4 or a later one in the same slot.
        if (is_k && lane < BN / 32) sm.bad[n & 3][lane] = 0u;
        __syncwarp();
        const int y = (j * BN) & ((1 << args.block_shift) - 1) & ~(rows - 1);
#pragma unroll 1
        for (int b0 = 0; b0 < nblk; b0 += 32) {
          const int blk = b0 + lane;
          if (b0 > 0) id = lookup(p, j, blk);
          const bool want = wanted(p, j, blk), good = want && id >= 0 && id < args.num_blocks;
          if (__any_sync(0xffffffffu, want && !good)) {
            if (want && !good) {  // a run of keys inside a word, or whole words
              const uint32_t run = rows >= 32 ? 0xffffffffu : ((1u << rows) - 1u) << (blk * rows & 31);
              for (int w = blk * rows / 32; is_k && w < max(1, rows / 32) + blk * rows / 32; ++w) atomicOr(&sm.bad[n & 3][w], run);
              atomicOr(&g_status, kStatusBadBlock);
            }
          }
          unsigned live = __ballot_sync(0xffffffffu, good);
          if (lane == 0) mbar_expect_tx(bar, __popc(live) * rows * 256u);
          __syncwarp();
#pragma unroll 1
          for (; live; live &= live - 1) {
            const int src = __ffs(live) - 1;
            const int z = __shfl_sync(0xffffffffu, id, src) * args.Hkv + p.kvh;
            const uint32_t dst = ring + s * TILE_BYTES + (b0 + src) * rows * 128;
            if (elect_one()) {
              tma_load_3d(dst, tm, bar, 0, y, z);
              tma_load_3d(dst + HALF_BYTES, tm, bar, 64, y, z);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
        ++n;
      };
      // Piece i's number, -1: there is none.
      auto find = [&](int i) { return pieces.wait(i) ? i : -1; };
      // One tile a turn: the next one's entries are asked for, then this one is loaded.
      int ip = find(0), j = 0, id = 0;
      if (ip >= 0) {
        j = pieces.at(ip).j0;
        id = lookup(pieces.at(ip), j, lane);
      }
#pragma unroll 1
      while (ok && ip >= 0) {
        int in = ip, jn = j + 1, next = 0;
        if (jn == pieces.at(ip).j1) {
          in = find(ip + 1);
          if (in >= 0) jn = pieces.at(in).j0;
        }
        if (in >= 0) next = lookup(pieces.at(in), jn, lane);
        load_tile(pieces.at(ip), j, id);
        if (in != ip) pieces.release(ip, lane);
        ip = in;
        j = jn;
        id = next;
      }
#pragma unroll 1
      for (int i = max(0, n - NS); i < n; ++i) mbar_wait_drain(smem_u32(&full[i % NS]), (i / NS) & 1);
    } else {
      // ---------------------------------------------------------- MMA issuer
      // The whole warp runs this (warp-uniform waits); MMAs and commits go out from one
      // elected lane.  The work is one stream of steps through the items: a one-tile item
      // has a step per key tile, a two-tile item two, one per slot.  S of step w + 2 goes out
      // after PV of step w, in the same slot, so the softmaxes of two steps overlap, of
      // successive items too.  Phase bits, bit t for slot t: Q_PH q_full, P_PH p_full and
      // O_PH o_free to wait for next; O_USED: an item has used O_t.
      const uint32_t tiles = tiles_base(), tmem = tmem_base();
      enum : uint32_t { Q_PH = 0, P_PH = 2, O_PH = 4, O_USED = 6 };
      uint32_t ph = 0;
      auto bit = [&](uint32_t i) { return (ph >> i) & 1u; };
      bool ok = true;
      auto free_tile = [&](uint64_t* empty, int g) { commit_elect(smem_u32(empty + g % NS)); };
      // A place in the stream: piece, key tile, slot, the tile's number in the CTA; the key
      // tiles [a, b) of its slot and [a2, b2) of the other one, the piece's last (exclusive).
      // Kept in registers: a step reads them some ten times, and a dependent shared-memory
      // read a time made the steps 1500 cycles longer.
      struct Step {
        int i, j, t, g, a, b, a2, b2, j1;
        bool single, fresh;  // fresh: the piece's first step
      };
      auto open_piece = [&](Step& at) {
        const Piece& p = pieces.at(at.i);
        at.j = p.j0;
        at.j1 = p.j1;
        at.t = p.slot0;
        at.g = p.tile0;
        at.single = p.single;
        at.fresh = true;
        at.a = p.first[at.t];
        at.b = p.end[at.t];
        at.a2 = p.first[at.t ^ 1];
        at.b2 = p.end[at.t ^ 1];
      };
      // Is this the step's key tile's last step?  (Two-tile items: slot 1's.)
      auto last_of_tile = [&](const Step& at) { return at.single || at.t == 1; };
      // Does the step's slot have its key tile?
      auto real = [&](const Step& at) { return at.j >= at.a && at.j < at.b; };
      // To the next step of the piece; false past its last.
      auto advance = [&](Step& at) {
        const int next_tile = last_of_tile(at) ? 1 : 0;
        at.t ^= 1;
        at.j += next_tile;
        at.g += next_tile;
        at.fresh = false;
        const int a = at.a, b = at.b;
        at.a = at.a2;
        at.b = at.b2;
        at.a2 = a;
        at.b2 = b;
        return at.j < at.j1;
      };
      auto k_landed = [&](int g) {
        return wait_bar(smem_u32(&sm.k_full[g % NS]), static_cast<uint32_t>((g / NS) & 1), abort_flag);
      };
      auto v_landed = [&](int g) {
        return wait_bar(smem_u32(&sm.v_full[g % NS]), static_cast<uint32_t>((g / NS) & 1), abort_flag);
      };
      auto p_there = [&](int t) {
        if (!wait_bar(smem_u32(&sm.p_full[t]), bit(P_PH + t), abort_flag)) return false;
        ph ^= 1u << (P_PH + t);
        tc_fence_after();
        return true;
      };
      auto any_bad = [&](int g) {
        const uint4 bad = *reinterpret_cast<const uint4*>(sm.bad[g & 3]);
        return (bad.x | bad.y | bad.z | bad.w) != 0u;
      };
      Step sc{}, oc{};  // the next S, the next PV
      bool o_open = false;  // oc's piece is open
      int ahead = 0;                         // steps that S is ahead of PV
      bool s_more = pieces.wait(0);
      if (s_more) open_piece(sc);
      bool hold = false;  // the next S's slot is the last one's: it waits for that one's PV
      int2 steps = make_int2(0, 0);
#pragma unroll 1
      while (ok && (s_more || ahead > 0)) {
        const bool do_o = ahead == 2 || !s_more || (hold && ahead == 1);
        const bool do_s = s_more && !(hold && ahead - do_o > 0);
        if (do_o && !o_open) {
          open_piece(oc);
          o_open = true;
        }
        if (do_o && do_s && sc.i == oc.i && oc.t == 0 && !oc.single) {
          // Inside a two-tile item, away from its edges: the same steps without their questions.
          const int end = min(oc.b, oc.b2) - 2;
          if (oc.j < end && oc.j > max(oc.a, oc.a2)) {
            int g = oc.g;
            const int g_end = g + end - oc.j;
#pragma unroll 1
            for (; g < g_end; ++g) {
              ok = v_landed(g) && k_landed(g + 1);
              if (!ok || any_bad(g)) break;
              const uint32_t k = tiles + kKOff + (g + 1) % NS * TILE_BYTES, v = tiles + kVOff + g % NS * TILE_BYTES;
#pragma unroll 1
              for (int t = 0; t < 2; ++t) {
                if (!(ok = p_there(t))) break;
                issue_pv<T>(tmem + 256 + 128 * t, tmem + 128 * t, v, 1u);
                if (t) free_tile(sm.v_empty, g);
                issue_qk<T>(tmem + 128 * t, tiles + t * TILE_BYTES, k);
                commit_elect(smem_u32(&sm.s_full[t]));
              }
              if (!ok) break;
              free_tile(sm.k_empty, g + 1);
            }
            if (!ok) break;
            const int done = g - oc.g;
            oc.j += done;
            oc.g += done;
            sc.j += done;
            sc.g += done;
          }
        }
        if (do_s) {
          // K and, for its first use, Q have landed: waited for ahead of the PV, so that the
          // two follow one another into the tensor pipe.
          if (sc.single ? sc.fresh : sc.j == sc.a && sc.j < sc.b) {
            const int qs = sc.single ? sc.i & 1 : sc.t;
            ok = wait_bar(smem_u32(&sm.q_full[qs]), bit(Q_PH + qs), abort_flag);
            ph ^= 1u << (Q_PH + qs);
          }
          ok = ok && k_landed(sc.g);
          if (!ok) break;
        }
        if (do_o) {
          const int t = oc.t;
          const uint32_t v = tiles + kVOff + oc.g % NS * TILE_BYTES;
          if (oc.single || t == 0) {
            // V has landed.  Rows without a key of the item are kept out of the product: whole
            // steps of 16 keys are not issued (`steps`: first and end), the others' rows, and
            // those of blocks outside the pool, are cleared.
            ok = v_landed(oc.g);
            if (!ok) break;
            int lo = 0, hi = BN;
            if (oc.fresh || oc.j + 1 == oc.j1) {
              const Piece& p = pieces.at(oc.i);
              lo = max(0, p.key_lo - oc.j * BN);
              hi = min(BN, p.key_hi - oc.j * BN);
            }
            steps = make_int2(lo >> 4, (hi + 15) >> 4);
            const bool bad = any_bad(oc.g);
            if ((lo & 15) != 0 || (hi & 15) != 0 || bad) {
              zero_v_rows(v, lo & ~15, lo, lane);
              zero_v_rows(v, hi, (hi + 15) & ~15, lane);
              if (bad) zero_bad_rows(v, sm.bad[oc.g & 3], lane);
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          if (real(oc)) {
            // The slot's first PV of the item overwrites O_t (which the epilogue must have read
            // out), its last publishes it.
            const bool first = oc.j == oc.a, last = oc.j + (oc.single ? 2 : 1) >= oc.b;
            if (first && bit(O_USED + t)) {
              ok = wait_bar(smem_u32(&sm.o_free[t]), bit(O_PH + t), abort_flag);
              ph ^= 1u << (O_PH + t);
            }
            ok = ok && p_there(t);
            if (!ok) break;
            if (steps.x == 0 && steps.y == BN / 16) {
              issue_pv<T>(tmem + 256 + 128 * t, tmem + 128 * t, v, first ? 0u : 1u);
            } else {
#pragma unroll 1
              for (int i = steps.x; i < steps.y; ++i)
                issue_pv_step<T>(tmem + 256 + 128 * t, tmem + 128 * t + 8 * i, v + i * 16 * 128, first && i == steps.x ? 0u : 1u);
            }
            if (last) {
              commit_elect(smem_u32(&sm.o_full[t]));
              ph |= 1u << (O_USED + t);
            }
          }
          if (last_of_tile(oc)) free_tile(sm.v_empty, oc.g);
          --ahead;
          if (!advance(oc)) {
            pieces.release(oc.i++, lane);
            o_open = false;
          }
        }
        if (do_s) {
          if (real(sc)) {
            const int qs = sc.single ? sc.i & 1 : sc.t;
            issue_qk<T>(tmem + 128 * sc.t, tiles + qs * TILE_BYTES, tiles + kKOff + sc.g % NS * TILE_BYTES);
            commit_elect(smem_u32(&sm.s_full[sc.t]));
            if (sc.j + 1 == sc.b) commit_elect(smem_u32(&sm.q_empty[qs]));
          }
          if (last_of_tile(sc)) free_tile(sm.k_empty, sc.g);
          ++ahead;
          hold = false;
          if (!advance(sc)) {
            const int t = sc.t ^ 1;  // the slot of the step just issued
            ++sc.i;
            s_more = pieces.wait(sc.i);
            if (s_more) {
              open_piece(sc);
              hold = sc.t == t;
            }
          }
        }
      }
      // All MMAs issued by this warp must complete before TMEM is freed.
      commit_elect(smem_u32(&sm.mma_done));
      mbar_wait_drain(smem_u32(&sm.mma_done), 0);
      __syncwarp();
    }
  } else if (wg == EPI_WG) {
    // ------------------------------------------------------------ epilogue
    // Thread = one row of a tile.  O comes out of TMEM 16 columns at a time, is scaled
    // (and, for a one-tile item, the two slots' states are joined) and written: 16-bit O,
    // or float32 partials.
    regs_dec<kEpilogueRegs>();
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const Geo geo = geometry();
    const int row_tok = row / geo.G;
    const uint32_t tmem = tmem_base();
    // This lane's row put aside; 16-byte chunk i of it sits at chunk i ^ lane.
    const uint32_t aside = tiles_base() + kAsideOff + lane * (D * 4);
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    uint32_t ph = 0;  // phase of o_full (and st_full) to wait for next, bit t for slot t
    bool ok = true;
#pragma unroll 1
    for (int ip = 0; ok && pieces.wait(ip); pieces.release(ip++, lane)) {
      const Piece& p = pieces.at(ip);
      const int slot = p.part;
#pragma unroll 1
      for (int rt = 0; rt < (p.single ? 1 : 2) && ok; ++rt) {
        // t: the slot; of a one-tile item's two, the one whose last tile comes last.
        const int nt = p.j1 - p.j0;
        const int t = p.single ? (p.slot0 + nt - 1) & 1 : rt;
        const bool both = p.single && nt > 1;
        const int mine = p.rows[rt] - wq * 32;  // rows of this warp's 32 that hold a token, if positive
        // This row's place in the output or, for a piece, in the workspace.
        long long at;
        if (slot < 0) {
          at = static_cast<long long>(p.tok0 + rt * geo.tpt + row_tok) * args.Hq + p.kvh * geo.G + row - row_tok * geo.G;
        } else {
          at = static_cast<long long>(slot) * args.slot_rows + rt * BM + row;
        }
        float* lse = slot < 0 ? args.lse : args.ws_lse;
        if (!p.any(t)) {
          // A row tile without keys beside one that has some: its rows see nothing; of a piece,
          // they may see something in another one.
          if (lane < mine) {
            if (lse != nullptr) lse[at] = -INFINITY;
            if (slot < 0) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(args.o) + at * D);
#pragma unroll 1
              for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          continue;
        }
        float m1 = -INFINITY, l1 = 0.f;
        bool put_aside = false;
        if (both) {
          // The other slot is done one tile earlier.  With few rows its O is put aside, so that
          // the next item's first tile finds the slot free.
          ok = wait_bar(smem_u32(&sm.o_full[t ^ 1]), ph >> (t ^ 1) & 1u, abort_flag) &&
               wait_bar(smem_u32(&sm.st_full[t ^ 1]), ph >> (t ^ 1) & 1u, abort_flag);
          if (!ok) break;
          ph ^= 1u << (t ^ 1);
          tc_fence_after();
          m1 = sm.stat_m[t ^ 1][row];
          l1 = sm.stat_l[t ^ 1][row];
          mbar_arrive(smem_u32(&sm.st_empty[t ^ 1]));
          put_aside = p.rows[0] <= kAsideRows;
          if (put_aside) {
            if (mine > 0) {
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t r[32];
                FA_TMEM_LD32(tmem + lane_off + 256 + (t ^ 1) * 128 + c, r);
                tmem_ld_wait();
                if (lane < mine) {
#pragma unroll
                  for (int v = 0; v < 8; ++v)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(aside + ((c / 4 + v) ^ lane) * 16),
                                 "r"(r[4 * v]), "r"(r[4 * v + 1]), "r"(r[4 * v + 2]), "r"(r[4 * v + 3])
                                 : "memory");
                }
              }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&sm.o_free[t ^ 1]));
          }
        }
        ok = wait_bar(smem_u32(&sm.o_full[t]), ph >> t & 1u, abort_flag) &&
             wait_bar(smem_u32(&sm.st_full[t]), ph >> t & 1u, abort_flag);
        if (!ok) break;
        ph ^= 1u << t;
        tc_fence_after();
        float m = sm.stat_m[t][row], l = sm.stat_l[t][row];
        mbar_arrive(smem_u32(&sm.st_empty[t]));
        float f0 = 1.f, f1 = 0.f;
        if (both) {
          const float mm = fmaxf(m, m1);
          f0 = m == -INFINITY ? 0.f : ex2_approx((m - mm) * args.scale_log2);
          f1 = m1 == -INFINITY ? 0.f : ex2_approx((m1 - mm) * args.scale_log2);
          l = f0 * l + f1 * l1;
          m = mm;
        }
        // l > 0: the row saw keys; l = 0: none; NaN marks a NaN score.
        const bool none = l == 0.f;
        if (lane < mine && lse != nullptr) lse[at] = l > 0.f ? m * args.scale + logf(l) : (none ? -INFINITY : l);
        const float inv = l > 0.f ? 1.f / l : (none ? 0.f : l);
        f0 *= inv;
        f1 *= inv;
        const uint32_t tO = tmem + lane_off + 256 + t * 128;
        const uint32_t tO1 = tmem + lane_off + 256 + (t ^ 1) * 128;
        const bool part = slot >= 0;
        char* out = part ? reinterpret_cast<char*>(args.ws_o) : static_cast<char*>(args.o);
        at *= part ? D * 4 : D * 2;  // bytes from here on
        if (mine > 0) {
          // Each lane writes its own row, 32 or 64 bytes a step.  (Rows put aside in shared memory and
          // written in runs were no faster: 107 us for 108 on the ragged batch; few rows joined there
          // and written whole, so that both slots are free at once: 512 single tokens 316 -> 310 us,
          // but 5 drafted tokens 90.2 -> 91.5 and one token 14.3 -> 14.8.)
          char* dst = out + at;
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            load_o16(tO + c, tO1 + c, both && !put_aside, none, f0, f1, o);
            if (lane < mine) {
              if (put_aside && !none) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                  float4 x;
                  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                               : "r"(aside + ((c / 4 + v) ^ lane) * 16));
                  o[4 * v] = fmaf(x.x, f1, o[4 * v]);
                  o[4 * v + 1] = fmaf(x.y, f1, o[4 * v + 1]);
                  o[4 * v + 2] = fmaf(x.z, f1, o[4 * v + 2]);
                  o[4 * v + 3] = fmaf(x.w, f1, o[4 * v + 3]);
                }
              }
              if (part) {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                  *reinterpret_cast<float4*>(dst + c * 4 + v * 16) = make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
              } else {
#pragma unroll
                for (int v = 0; v < 2; ++v)
                  *reinterpret_cast<uint4*>(dst + c * 2 + v * 16) =
                      make_uint4(pack2<T>(o[8 * v], o[8 * v + 1]), pack2<T>(o[8 * v + 2], o[8 * v + 3]),
                                 pack2<T>(o[8 * v + 4], o[8 * v + 5]), pack2<T>(o[8 * v + 6], o[8 * v + 7]));
              }
            }
          }
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&sm.o_free[t]));
        if (both && !put_aside) mbar_arrive(smem_u32(&sm.o_free[t ^ 1]));
      }
    }
  } else {
    // ------------------------------------------------------------ softmax warps
    // Warpgroup t is the softmax of slot t: thread = row, all 128 score columns of a key
    // tile in registers (as in fwd_tc.cu).  A warp without a valid row only keeps step.
    regs_inc<kSoftmaxRegs>();
    const uint32_t tmem = tmem_base();
    const int t = wg;
    const int wq = warp & 3;
    const int row = wq * 32 + lane, row_tok = row / geometry().G;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + t * 128;
    const uint32_t tO = tS + 256;
    const float sl2 = args.scale_log2;
    // Phase bits: S_PH s_full to wait for next, ST_PH st_empty, ST_ANY an item was published.
    enum : uint32_t { S_PH = 1, ST_PH = 2, ST_ANY = 4 };
    uint32_t ph = ST_PH;
    bool ok = true;
#pragma unroll 1
    for (int ip = 0; ok && pieces.wait<true>(ip); ++ip) {
      // Keys that this row sees, [row_lo, row_hi), and that every row of the tile sees,
      // [all_lo, all_hi): key tiles inside the latter need no mask.
      int row_lo, row_hi, all_lo, all_hi;
      int j, end, step, bad_at;  // bad_at + j: the key tile's number in the CTA
      bool busy;
      {
        const Piece& p = pieces.at(ip);
        j = p.first[t];
        end = p.end[t];
        step = p.single ? 2 : 1;
        bad_at = p.tile0 - p.j0;
        busy = wq * 32 < p.rows[t];
        row_lo = p.key_lo;
        row_hi = p.key_hi;
        all_lo = p.all_lo[t];
        all_hi = p.all_hi[t];
        const int pos = p.pos[t] + row_tok;
        if (args.causal) row_hi = min(row_hi, pos + 1);
        if (args.window > 0) row_lo = max(row_lo, pos - args.window + 1);
        pieces.release(ip, lane);
      }
      if (j >= end) continue;
      float m = -INFINITY, l = 0.f;
      bool nan_row = false, begun = false;
#pragma unroll 1
      for (; j < end; j += step) {
        ok = wait_inline(smem_u32(&sm.s_full[t]), ph & S_PH, abort_flag);
        if (!ok) break;
        ph ^= S_PH;
        if (!busy) {
          mbar_arrive(smem_u32(&sm.p_full[t]));
          continue;
        }
        tc_fence_after();
        const int kb = j * BN;
        const uint4 bad = *reinterpret_cast<const uint4*>(sm.bad[(bad_at + j) & 3]);
        const bool any_bad = (bad.x | bad.y | bad.z | bad.w) != 0u;
        if (kb + BN > all_hi || kb < all_lo || any_bad) {
          // Visible keys of this row: columns [c_lo, c_hi), without the blocks outside the pool.
          const int c_lo = max(0, row_lo - kb), c_hi = max(min(BN, row_hi - kb), c_lo);
#pragma unroll 1
          for (int c = 0; c < BN / 32; ++c) {
            // Bit e: column 32 c + e is visible.
            const int lo = min(max(c_lo - 32 * c, 0), 32), hi = min(max(c_hi - 32 * c, 0), 32);
            const uint32_t seen = (hi == 32 ? 0xffffffffu : (1u << hi) - 1u) & (lo == 32 ? 0u : 0xffffffffu << lo) &
                                  ~sm.bad[(bad_at + j) & 3][c];
            if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
            uint32_t r[32];
            FA_TMEM_LD32(tS + 32 * c, r);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = seen >> e & 1u ? r[e] : __float_as_uint(-INFINITY);
            FA_TMEM_ST32(tS + 32 * c, r);
          }
          tmem_st_wait();
        }
        uint32_t s[BN];
        FA_TMEM_LD32(tS + 0, (s + 0));
        FA_TMEM_LD32(tS + 32, (s + 32));
        FA_TMEM_LD32(tS + 64, (s + 64));
        FA_TMEM_LD32(tS + 96, (s + 96));
        tmem_ld_wait();
        float mm[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          mm[q] = fmax3_nan(__uint_as_float(s[q]), __uint_as_float(s[q + 8]), -INFINITY);
#pragma unroll
        for (int c = 16; c < BN; c += 16)
#pragma unroll
          for (int q = 0; q < 8; ++q)
            mm[q] = fmax3_nan(mm[q], __uint_as_float(s[c + q]), __uint_as_float(s[c + 8 + q]));
        const float mx = fmax3_nan(fmax3_nan(mm[0], mm[1], mm[2]), fmax3_nan(mm[3], mm[4], mm[5]),
                                   fmax3_nan(mm[6], mm[7], -INFINITY));
        nan_row |= (mx != mx);
        const float m_new = fmaxf(m, mx);
        const bool need = (m_new - m) * sl2 > kRescaleThreshold;
        float alpha = 1.f;
        if (need) {
          alpha = ex2_approx((m - m_new) * sl2);
          m = m_new;
          l *= alpha;
        }
        if (begun && __any_sync(0xffffffffu, need)) {
          // O_t's last update is complete: S_t of this tile was issued after it.
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t r[32];
            FA_TMEM_LD32(tO + 32 * c, r);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            FA_TMEM_ST32(tO + 32 * c, r);
          }
        }
        begun = true;
        const float ms = (m == -INFINITY) ? 0.f : m * sl2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2), nms2 = f2_pack(-ms, -ms);
        uint64_t acc[4] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f), f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t x2 = f2_fma(f2_pack(__uint_as_float(s[32 * c + e]), __uint_as_float(s[32 * c + e + 1])),
                                       sl2x2, nms2);
            float x0, x1;
            f2_unpack(x2, x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            acc[(e >> 1) & 3] = f2_add(acc[(e >> 1) & 3], f2_pack(p0, p1));
            // P in 16 bits, the MMA's type: relative error up to 2^-8 (bf16; fp16 2^-11) a weight,
            // the size of the output's own rounding, less where many keys share the weight; l adds
            // the unrounded values.  Measured against 64 bits (bf16, relative norm): 0.0021 to 0.0023,
            // the output's rounding alone 0.0017.
            pk[e >> 1] = pack2<T>(p0, p1);
          }
          asm volatile(
              "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
                  tS + 16 * c),
              "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3]), "r"(pk[4]), "r"(pk[5]), "r"(pk[6]), "r"(pk[7]),
              "r"(pk[8]), "r"(pk[9]), "r"(pk[10]), "r"(pk[11]), "r"(pk[12]), "r"(pk[13]), "r"(pk[14]), "r"(pk[15])
              : "memory");
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(&sm.p_full[t]));
        {
          const uint64_t s01 = f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3]));
          float a0, a1;
          f2_unpack(s01, a0, a1);
          l += a0 + a1;
        }
      }
      if (!ok) break;
      if (ph & ST_ANY) ok = wait_inline(smem_u32(&sm.st_empty[t]), (ph & ST_PH) != 0u, abort_flag);
      if (!ok) break;
      ph = (ph ^ ST_PH) | ST_ANY;
      sm.stat_m[t][row] = m;
      sm.stat_l[t][row] = nan_row ? __uint_as_float(0x7fc00000u) : l;
      mbar_arrive(smem_u32(&sm.st_full[t]));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && sm.abort_flag) atomicOr(&g_status, kStatusTimeout);
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(sm.tmem_base, 512);
  }
}

// Joins the partial results of an item that several CTAs share: with lse_s of piece s,
// lse = ln sum exp(lse_s), o = sum exp(lse_s - lse) o_s, in the order of the pieces.  Block
// x looks at the item that begins in CTA x and ends in a later one, if there is one.  A
// warp takes four rows at a time, eight lanes reading a row's logsumexps, all lanes its o,
// so that four rows' loads are in flight.  Bound by the latency of those loads, the partials
// being in L2: 17.4 us after the 2048-token piece with cold caches (one row a warp: 22.6 us).
constexpr int CB_WARPS = 8, CB_ROWS = 4;
template <class T>
__global__ void __launch_bounds__(CB_WARPS * 32) combine_kernel(const __grid_constant__ ExtendArgs args) {
  wait_for_previous_kernel();
  let_next_kernel_start();
  const ExtendDesc d = args.desc[blockIdx.x];
  if (d.last < 0) return;
  const int lane = threadIdx.x & 31;
  const int G = args.Hq / args.Hkv, tpt = BM / G, rows = d.ntok * G;
  const int first = blockIdx.x, pieces = d.last - first + 1;
  const float nan = __uint_as_float(0x7fc00000u);
  // With no more rows than a block has warps each warp takes one.
  const int nk = rows <= CB_WARPS ? 1 : CB_ROWS;
  for (int r0 = (blockIdx.y * CB_WARPS + (threadIdx.x >> 5)) * nk; r0 < rows; r0 += gridDim.y * CB_WARPS * nk) {
    // This lane's row of the four: its place in a slot and in the output.
    const int mine = nk == 1 ? 0 : lane >> 3;
    const int r = min(r0 + mine, rows - 1), tok = r / G, t = tok >= tpt ? 1 : 0;
    const int srow = t * BM + r - t * tpt * G;
    const long long out = static_cast<long long>(d.tok0 + tok) * args.Hq + d.kvh * G + r - tok * G;
    // Piece s of the item lies in this slot of the workspace.
    auto slot_at = [&](int s) { return static_cast<long long>(s == 0 ? 2 * first + 1 : 2 * (first + s)) * args.slot_rows; };
    float M = -INFINITY;
    for (int s = lane & 7; s < pieces; s += 8) {
      const float v = args.ws_lse[slot_at(s) + srow];
      M = M != M || v != v ? nan : fmaxf(M, v);
    }
#pragma unroll
    for (int x = 4; x > 0; x >>= 1) {
      const float v = __shfl_xor_sync(0xffffffffu, M, x);
      M = M != M || v != v ? nan : fmaxf(M, v);
    }
    float W = 0.f;  // this lane's row's
    float4 acc[CB_ROWS];
#pragma unroll
    for (int k = 0; k < CB_ROWS; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < pieces; s0 += 8) {
      const int s = s0 + (lane & 7);
      const float w_l = s < pieces && M != -INFINITY ? __expf(args.ws_lse[slot_at(s) + srow] - M) : 0.f;
      const int n = min(8, pieces - s0);
#pragma unroll 2
      for (int i = 0; i < n; ++i) {
        const float* o = args.ws_o + slot_at(s0 + i) * D + lane * 4;
        W += __shfl_sync(0xffffffffu, w_l, (lane & 24) + i);
        float w[CB_ROWS];
        float4 v[CB_ROWS];
#pragma unroll
        for (int k = 0; k < CB_ROWS; ++k) {
          w[k] = __shfl_sync(0xffffffffu, w_l, 8 * k + i);
          const int row = __shfl_sync(0xffffffffu, srow, 8 * k);
          // A piece without a visible key wrote no o.
          v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < nk && w[k] != 0.f) v[k] = *reinterpret_cast<const float4*>(o + row * D);
        }
#pragma unroll
        for (int k = 0; k < CB_ROWS; ++k) {
          acc[k].x = fmaf(w[k], v[k].x, acc[k].x);
          acc[k].y = fmaf(w[k], v[k].y, acc[k].y);
          acc[k].z = fmaf(w[k], v[k].z, acc[k].z);
          acc[k].w = fmaf(w[k], v[k].w, acc[k].w);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < CB_ROWS; ++k) {
      const float Wk = __shfl_sync(0xffffffffu, W, 8 * k);
      const long long at = __shfl_sync(0xffffffffu, out, 8 * k);
      const float inv = Wk == 0.f ? 0.f : 1.f / Wk;  // a NaN logsumexp makes the row NaN
      if (k < nk && r0 + k < rows)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(args.o) + at * D + lane * 4) =
            make_uint2(pack2<T>(acc[k].x * inv, acc[k].y * inv), pack2<T>(acc[k].z * inv, acc[k].w * inv));
    }
    if ((lane & 7) == 0 && (lane >> 3) < nk && r0 + mine < rows && args.lse != nullptr) args.lse[out] = W == 0.f ? -INFINITY : M + logf(W);
  }
}

}  // namespace ext

cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t stream) {
  using namespace ext;
  const int G = a.Hq / a.Hkv, tpt = BM / G;
  // Q boxes: the largest divisor of a tile's tokens that keeps a box within 32 rows.
  int box = 1;
  for (int i = 1; i <= tpt; ++i)
    if (tpt % i == 0 && i * G <= 32) box = i;
  const int bs = 1 << a.block_shift;
  CUtensorMap tq, tk, tv;
  const long long qd[3] = {D, a.Hq, a.T}, qs[2] = {D * 2, a.q_stride * 2};
  const int qb[3] = {64, G, box};
  const long long pd[3] = {D, bs, static_cast<long long>(a.num_blocks) * a.Hkv}, ps[2] = {D * 2, static_cast<long long>(bs) * D * 2};
  const int pb[3] = {64, bs < BN ? bs : BN, 1};
  if (!make_tmap_3d_half(&tq, a.q, qd, qs, qb, a.f16) || !make_tmap_3d_half(&tk, a.kpool, pd, ps, pb, a.f16) ||
      !make_tmap_3d_half(&tv, a.vpool, pd, ps, pb, a.f16))
    return cudaErrorInvalidValue;
  auto kernel = a.f16 ? extend_kernel<F16> : extend_kernel<Bf16>;
  // With fewer registers than the split draws on, setmaxnreg.inc would wait forever.  One
  // build has one answer, so it is asked for once.
  static std::atomic<bool> fits[2];
  cudaError_t e = cudaSuccess;
  if (!fits[a.f16 != 0].load(std::memory_order_relaxed)) {
    cudaFuncAttributes fattr{};
    e = cudaFuncGetAttributes(&fattr, reinterpret_cast<const void*>(kernel));
    if (e != cudaSuccess) return e;
    if (fattr.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
    fits[a.f16 != 0].store(true, std::memory_order_relaxed);
  }
  e = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), kSmemBytes);
  if (e != cudaSuccess) return e;
  int sms = 0;
  e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(sms < kExtendMaxCtas ? sms : kExtendMaxCtas);
  e = launch_dependent(kernel, dim3(grid), dim3(NUM_THREADS), kSmemBytes, stream, tq, tk, tv, a, box);
  if (e != cudaSuccess) return e;
  const dim3 cgrid(grid, (a.slot_rows + CB_WARPS * CB_ROWS - 1) / (CB_WARPS * CB_ROWS));
  return launch_dependent(a.f16 ? combine_kernel<F16> : combine_kernel<Bf16>, cgrid, dim3(CB_WARPS * 32), 0, stream, a);
}

cudaError_t take_status_extend(unsigned int* out) { return take_local_status(out); }

}  // namespace fa
