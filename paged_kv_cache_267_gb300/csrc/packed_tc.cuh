// Attention of a ragged step over the paged cache, on the 5th-generation tensor
// cores: packed prompts and chunks (causal), and drafted trees (each row attends to
// the cache before the drafted tokens and to its ancestors among them).
//
// The rows of an item (packed_plan.cuh) are the (token, head) pairs of a unit of one
// sequence and one KV head, as matrix Q [rows x D]; with K/V tiles of kKv tokens,
//   S = Q K^T,  P = 2^(S c - m),  O += P V,  l += sum P
// with a running reference m per row, which moves only when a score exceeds it by
// more than 2^8, and out = O / l.
//
// Roles: one warp works out the CTA's items, in a ring that all others read them from,
// and streams K tiles, one streams V tiles (TMA through the block table), one loads Q and
// issues the products S, one issues the products O, groups of four softmax warps serve a
// 128-row tile each (one row a thread), and four warps store the results, so that a group
// goes on with its next item while the last one's output is written. (With one warp for
// all products, its own waits and instruction fetches, 700 cycles a job beside 1,050 of
// tensor work, came in the way of both.)
// A job is the product of a row tile and a K/V tile; jobs alternate between the two
// groups (a unit of more than 128 rows: each group has its rows and every tile; one of
// at most 128: both groups have the same rows, each every other tile, joined by the
// storing warps). S runs two jobs ahead of the softmax, across items. head_dim 256 has one
// group, whose S has two buffers (its O fills half of the tensor memory).
//
// Bound: a K/V tile of two row tiles is 2,112 cycles of tensor work (M128 N128 K16: 66)
// and takes 2,650, as S, softmax and O of a row tile follow each other in one buffer and
// only the other group's fill the gaps; one prompt of 16,384 tokens, 32 heads: 1.46 to 1.51
// ms, 1,460 to 1,510 TFLOP/s under the limit of 1.4 kW. An item costs about 7,000 cycles
// besides (e4m3: 11,000): Q's load behind the last products and its conversion, the masked
// tiles, O read out. What the warps run must stay small: some 5,000 instructions a kernel
// share the instruction cache, and one copy of each piece of code in place of two or three
// gave 4 to 13%.
//
// Masks: a row's attended positions in a tile are a bit word per 32 tokens (a range,
// and for a tree the ancestor bits moved to the tile); tiles that every row of a
// warp attends to in full take no mask. V rows outside of the unit's range are zeroed,
// as they may hold anything; where a tile is masked for some row, its V is looked
// through for infinities and NaN, which a weight of zero would not keep out of the
// other rows, and such a tile is added up without the tensor cores.
//
// FP8 caches: S is a product of e4m3 values, K as it is cached and Q as a sum of two (bf16)
// or three (f16) of them, made in its place by the storing warps; two terms at twice the
// rate cost as much as one 16-bit product, and K needs no conversion. (With K converted to
// f16 as V is, 19 trees of 32 tokens on 16,384 took 221 us instead of 157, 1,024 rows at
// head_dim 256 600 instead of 412.) The weights have to span more than e4m3 does, so V's
// tiles become f16 (exact), in two buffers, by the storing warps, which store an item's
// results between the next one's first tiles.
#pragma once

#include <float.h>

#include "attn_tc.cuh"
#include "packed_ops.h"
#include "pa_internal.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;
constexpr int kGroupThreads = 128;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;  // bound of every wait (2 s)
constexpr uint64_t kDrainNs = 200000000ull;  // and of those after one ran out
constexpr float kFloor = -3e38f;             // reference-max start
constexpr float kRescaleAbove = 8.f;         // log2 units
// f16 weights are 2^7 times as large against their reference: at most 2^15, and
// subnormal below 2^-21 of it instead of 2^-14.
constexpr float kF16Lift = 7.f;              // log2 units
constexpr unsigned kFull = 0xffffffffu;
constexpr int kItemRing = 3;                 // items known at once
// Who works out a CTA's items: the plan kernel, or the CTA itself (small steps), by cutting
// the space of places or taking whole pairs. (Kernels of their own: each would hold the
// others' registers, 131 us instead of 119 for one tree on 131,072 tokens.)
enum { kPlanned = 0, kSmallCut = 1, kSmallWhole = 2 };

template <int QT, int D, bool FP8>
struct Cfg {
  static constexpr int kGroups = packed_shape(D).rows;  // softmax groups
  static constexpr int kKv = packed_shape(D).kv;        // tokens a tile
  static constexpr int kSlices = kKv / 16;
  static constexpr int kBoxes = D / 64;  // 64-dim boxes of a 16-bit tile
  // FP8: Q as a sum of e4m3 values, as many as its type's bits need
  static constexpr int kTerms = FP8 ? (QT == kBF16 ? 2 : 3) : 1;
  static constexpr int kKStages = FP8 ? (kTerms == 2 ? 3 : 2) : (D == 64 ? 4 : 2);
  static constexpr int kVStages = FP8 ? 2 : (D == 64 ? 4 : 3);
  static constexpr int kStages = kKStages > kVStages ? kKStages : kVStages;
  // Barriers: K and V rings (full, empty); per S buffer: computed, half of P written, the
  // other half, product with V complete; Q loaded, ready (items in turn) and done with; per
  // group: last product of an item complete, O and statistics read, statistics written,
  // a tile's V looked through; FP8: converted V (two buffers) written and read; items
  // known and read; the ends of the two product warps.
  enum {
    kBarKFull = 0,
    kBarKEmpty = kBarKFull + kStages,
    kBarVFull = kBarKEmpty + kStages,
    kBarVEmpty = kBarVFull + kStages,
    kBarS = kBarVEmpty + kStages,
    kBarP = kBarS + 2,
    kBarP2 = kBarP + 2,
    kBarO = kBarP2 + 2,
    kBarQRaw = kBarO + 2,
    kBarQFull = kBarQRaw + 1,
    kBarQFree = kBarQFull + 2,
    kBarOFull = kBarQFree + 1,
    kBarOFree = kBarOFull + 2,
    kBarStat = kBarOFree + 2,
    kBarLook = kBarStat + 2,
    kBarCVFull = kBarLook + 2,
    kBarCVFree = kBarCVFull + 2,
    kBarItem = kBarCVFree + 2,
    kBarItemFree = kBarItem + kItemRing,
    kBarDrain = kBarItemFree + kItemRing,
    kNumBars = kBarDrain + 2
  };
  static constexpr int kStoreWarp = 4 * kGroups, kMmaS = kStoreWarp + 4,
                       kLoadK = kMmaS + 2, kLoadV = kMmaS + 3;  // (the products O behind S)
  static constexpr int kThreads = (kMmaS + 4) * 32;
  // Registers a thread: what the block is launched with, and what the softmax warps, the
  // storing warps and all others make of it where that is too little for the softmax.
  // (A spill costs far more than its instruction here: beside 220 KB of shared memory
  // the L1 cache holds little, and what the storing warps had spilt at 64 made them ten
  // times slower.)
  static constexpr bool kSplitRegs = kThreads == 512;
  static constexpr int kLaunchRegs = kSplitRegs ? 128 : 168;
  static constexpr int kSoftmaxRegs = FP8 ? 176 : 184, kStoreRegs = FP8 ? 96 : 80, kOtherRegs = 64;
  static_assert(kThreads == 384 || (kThreads == 512 && kGroups == 2 && 2 * kSoftmaxRegs + kStoreRegs +
                                                                           kOtherRegs == 4 * kLaunchRegs),
                "registers of the block");
  static constexpr uint32_t kQBox = kRows * 128, kQBytes = (FP8 ? kTerms * D / 128 : kBoxes) * kQBox;  // one row tile's Q
  static constexpr uint32_t kBox = kKv * 128, kTile = kBoxes * kBox;        // 16-bit K or V tile
  static constexpr uint32_t kRawBoxes = FP8 ? D / 128 : kBoxes;             // 128-byte boxes
  static constexpr uint32_t kRing = kRawBoxes * kBox;                       // ring tile
  // small things first, then the tiles, which start on 1 KB
  static constexpr uint32_t kBar = 0, kSlot = (8 * kNumBars + 15) & ~15, kSkip = kSlot + 8, kLook = kSkip + 8,
                            kItem = kLook + 32, kShift = kItem + 48 * kItemRing,
                            kStat = kShift + (FP8 ? 2 * kGroups * kRows : 0),
                            kSmall = kStat + kGroups * 2 * kRows * 4;
  static constexpr uint32_t kQ = (kSmall + 1023) / 1024 * 1024, kK = kQ + kGroups * kQBytes,
                            kV = kK + kKStages * kRing, kVc = kV + kVStages * kRing,
                            kBytes = kVc + (FP8 ? 2 * kTile : 0);
  // where term t of Q's head dims 128 b .. 128 b + 127 is, in boxes: terms 0 and 1 in the
  // place of the 16-bit values that they are made of
  __device__ static constexpr int q_region(int t, int b) { return t < 2 ? 2 * b + t : D / 64 + b; }
  static constexpr uint32_t kColS = 0, kColO = 2 * kKv;
  static_assert(kLook % 16 == 0 && kItem % 16 == 0 && kStat % 8 == 0, "alignment of what is read at once");
  static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
  static_assert(kColO + kGroups * D <= kTmemCols, "tensor memory");
};

__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity) {
  return mbar_wait_bounded(bar, parity & 1, kWaitNs);
}
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity) {
  return __all_sync(kFull, wait_one(bar, parity));
}

// Products issued by a whole warp in step: every lane comes here with the same values,
// which then sit in uniform registers, and one elected lane issues. (Issued by one lane
// of a diverged warp, each product took 60 to 90 cycles to move its descriptors, 1,300 a
// job of 1,024 cycles of tensor work.) Four M128 steps of 32 bytes (K16, of e4m3 K32) over
// one swizzled box, A and B in shared memory; the first accumulates iff acc0 != 0.
template <bool F8>
__device__ __forceinline__ void mma4_ss_all(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t acc0) {
  if constexpr (F8) {
  asm volatile(
        "{\n.reg .pred p0, p1, e;\n.reg .b64 ad, bd;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p0, %4, 0;\nsetp.eq.b32 p1, 0, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p0;\n"
        "add.u64 ad, %1, 2;\nadd.u64 bd, %2, 2;\n"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %3, p1;\n"
        "add.u64 ad, %1, 4;\nadd.u64 bd, %2, 4;\n"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %3, p1;\n"
        "add.u64 ad, %1, 6;\nadd.u64 bd, %2, 6;\n"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %3, p1;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc0)
        : "memory");
  } else {
  asm volatile(
        "{\n.reg .pred p0, p1, e;\n.reg .b64 ad, bd;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p0, %4, 0;\nsetp.eq.b32 p1, 0, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p0;\n"
        "add.u64 ad, %1, 2;\nadd.u64 bd, %2, 2;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %3, p1;\n"
        "add.u64 ad, %1, 4;\nadd.u64 bd, %2, 4;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %3, p1;\n"
        "add.u64 ad, %1, 6;\nadd.u64 bd, %2, 6;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %3, p1;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc0)
        : "memory");
  }
}
// 2 or 4 M128 K16 steps with A in tensor memory: step k reads A 8 k columns on and B 16 k
// rows (2048 k bytes) on.
template <int STEPS>
__device__ __forceinline__ void mma_ts_all(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc0) {
  static_assert(STEPS == 2 || STEPS == 4, "steps");
  if constexpr (STEPS == 4) {
    asm volatile(
        "{\n.reg .pred p0, p1, e;\n.reg .b32 ac;\n.reg .b64 bd;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p0, %4, 0;\nsetp.eq.b32 p1, 0, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p0;\n"
        "add.u32 ac, %1, 8;\nadd.u64 bd, %2, 128;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ac], bd, %3, p1;\n"
        "add.u32 ac, %1, 16;\nadd.u64 bd, %2, 256;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ac], bd, %3, p1;\n"
        "add.u32 ac, %1, 24;\nadd.u64 bd, %2, 384;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ac], bd, %3, p1;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc0)
        : "memory");
  } else {
    asm volatile(
        "{\n.reg .pred p0, p1, e;\n.reg .b32 ac;\n.reg .b64 bd;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p0, %4, 0;\nsetp.eq.b32 p1, 0, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p0;\n"
        "add.u32 ac, %1, 8;\nadd.u64 bd, %2, 128;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ac], bd, %3, p1;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc0)
        : "memory");
  }
}
// Column of S where the second half of a tile's weights begins: 128 tokens' sit over
// columns 0-31 and 64-95, 64 tokens' over 0-15 and 16-31.
__device__ __forceinline__ constexpr int half_col(int kv) { return kv == 128 ? 64 : 16; }
__device__ __forceinline__ void commit_all(uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar)
      : "memory");
}

// Stage and phase of a ring position.
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// What a CTA works through of a pair (packed_plan.cuh).
struct PackedItem {
  int b, kvh;        // sequence, KV head
  int row0, ntok;    // first packed row and tokens of the unit
  int pos0;          // position of its first token
  int first;         // position of the sequence's first query
  int lo, hi;        // positions that its rows may attend to
  int tile0, nt;     // K/V tiles of it; nt -1: no more items
  int slot;          // partial result, -1: the unit is whole
  int pad;
};

// Split mode: a whole pair that begins at place f0 becomes what CTA `me` has of it.
// Returns its CTAs (their partial results).
__device__ __forceinline__ int cut(int f0, int tpg, int wsz, int me, PackedItem* it) {
  const int per = tile_places(it->ntok > tpg), nt = max(it->nt, 1), g0 = f0 + kOutPlaces;
  const int from = tiles_before(me * wsz - g0, nt, per), to = tiles_before((me + 1) * wsz - g0, nt, per);
  it->slot = from > 0 || to < nt ? 2 * me + (from == 0 ? 1 : 0) : -1;
  it->tile0 = from;
  if (it->nt > 0 || to <= from) it->nt = to - from;
  return (g0 + (nt - 1) * per) / wsz - g0 / wsz + 1;
}

// The plan of a small step (at most 32 sequences), which every CTA's K warp works out by
// itself, lane b with sequence b: split mode or, where no pair can have more than a few
// tiles, whole pairs in turn, which need no join. It saves the plan kernel in front, 4 us of
// a step of 11, and the join's launch behind.
template <bool WHOLE>
struct SmallPlan {
  int n, q0, len;  // of this lane's sequence: new tokens, first row, length
  int wsz;
  // the next pair: sequence, unit of it, KV head, places before it
  int b, u, h, f0;
  // (WHOLE: f0 is the next pair's number, u and h the units of this lane's sequence and those
  // up to its end)

  __device__ __forceinline__ PackedUnit unit(const PackedArgs& a, int b, int u) const {
    const int n_b = __shfl_sync(kFull, n, b), len_b = __shfl_sync(kFull, len, b), q_b = __shfl_sync(kFull, q0, b);
    return packed_unit(b, u, q_b, n_b, len_b, a.tpu, a.kv, a.window, a.tree != nullptr);
  }
  __device__ __forceinline__ int places(const PackedArgs& a, const PackedUnit& x) const {
    return pair_places(x.nt, x.ntok > a.tpg);
  }
  // The first pair of CTA `me`.
  __device__ __forceinline__ void begin(const PackedArgs& a, int lane, int me) {
    const bool in = lane < a.B;
    const int cap = a.MB * a.bs;
    const int s0 = in ? a.query_start[lane] : 0, s1 = in ? a.query_start[lane + 1] : 0;
    const int l0 = in ? a.seq_lens[lane] : 0;
    int start = min(max(s0, 0), a.T), end = in ? min(max(s1, 0), a.T) : 0;
    bool bad = start != s0 || end != s1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {  // starts made non-decreasing
      const int x = __shfl_up_sync(kFull, start, o);
      if (lane >= o) start = max(start, x);
    }
    bad = bad || (in && (start > max(s0, 0) || end < start));
    end = max(end, start);
    len = min(max(l0, 0), cap);
    n = in ? end - start : 0;
    q0 = start;
    if (me == 0) {
      if (bad || (a.tree && n > 64)) atomicOr(a.err, PA_DEVERR_QUERY);
      if (len != l0) atomicOr(a.err, PA_DEVERR_SEQ_LEN);
    }
    if constexpr (WHOLE) {
      f0 = me;
      u = h = (n + a.tpu - 1) / a.tpu;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, h, o);
        if (lane >= o) h += x;
      }
      return;
    }
    // places of this lane's sequence, one KV head
    int mine = 0;
    for (int t0 = 0, i = 0; t0 < n; t0 += a.tpu, ++i)
      mine += places(a, packed_unit(lane, i, q0, n, len, a.tpu, a.kv, a.window, a.tree != nullptr));
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += x;
    }
    const int all = __shfl_sync(kFull, upto, 31) * a.Hkv;
    wsz = max((all + a.ctas - 1) / a.ctas, a.min_places);
    const int at = me * wsz;
    const unsigned here = __ballot_sync(kFull, mine > 0 && at < upto * a.Hkv);
    b = here == 0 ? 32 : __ffs(here) - 1;
    u = h = 0;
    if (b == 32) return;
    f0 = (__shfl_sync(kFull, upto, b) - __shfl_sync(kFull, mine, b)) * a.Hkv;
    while (true) {
      const int c = places(a, unit(a, b, u));
      if (at < f0 + c * a.Hkv) {
        h = max(at - f0, 0) / c;
        f0 += h * c;
        return;
      }
      f0 += c * a.Hkv;
      ++u;
    }
  }
  // CTA `me`'s part of the next pair that it has one of, and its join's note for the merge
  // where the pair begins here and goes on in the next CTA.
  __device__ __forceinline__ void next(const PackedArgs& a, int lane, int me, PackedItem* it) {
    if constexpr (WHOLE) {  // every a.ctas'th pair
      const int un = f0 / a.Hkv, kvh = f0 - un * a.Hkv;
      const unsigned behind = __ballot_sync(kFull, h > un);
      if (behind == 0) return;
      const int at = __ffs(behind) - 1;
      const PackedUnit x = unit(a, at, un - __shfl_sync(kFull, h - u, at));
      *it = PackedItem{x.b, kvh, x.row0, x.ntok, x.pos0, x.first, x.lo, x.hi, 0, x.nt, -1, 0};
      f0 += a.ctas;
      return;
    }
    while (b < 32) {
      const PackedUnit x = unit(a, b, u);
      const int c = places(a, x), whole_nt = max(x.nt, 1);
      PackedItem y = PackedItem{x.b, h, x.row0, x.ntok, x.pos0, x.first, x.lo, x.hi, 0, x.nt, -1, 0};
      const int ctas = cut(f0, a.tpg, wsz, me, &y);
      const bool some = tiles_before((me + 1) * wsz - f0 - kOutPlaces, whole_nt, tile_places(x.ntok > a.tpg)) > y.tile0;
      const bool behind = y.tile0 >= whole_nt;  // all of it is the CTA's before
      if (!some && !behind) {
        b = 32;
        return;
      }
      f0 += c;
      if (++h == a.Hkv) {
        h = 0;
        if (++u * a.tpu >= __shfl_sync(kFull, n, b)) {
          u = 0;
          const unsigned live = __ballot_sync(kFull, n > 0), more = b < 31 ? live >> (b + 1) : 0u;
          b = more == 0 ? 32 : b + __ffs(more);
        }
      }
      if (behind) continue;
      *it = y;
      if (y.slot == 2 * me + 1 && lane == 0) {
        PackedJoin j = {};
        j.row0 = y.row0;
        j.ntok = y.ntok;
        j.kvh = y.kvh;
        j.n = ctas;
        reinterpret_cast<PackedJoin*>(a.plan + packed_joins_at(a.ctas))[me] = j;
      }
      return;
    }
  }
};

template <int QT>
__device__ __forceinline__ float f32_of(uint32_t w, int hi) {
  const uint16_t v = static_cast<uint16_t>(hi ? w >> 16 : w & 0xffffu);
  return QT == kBF16 ? __uint_as_float(static_cast<uint32_t>(v) << 16)
                     : __half2float(__ushort_as_half(v));
}
// Element `hi` of a pair of 16-bit values of the products' type.
template <bool BF16>
__device__ __forceinline__ float op_f32(uint32_t w, int hi) {
  return f32_of<BF16 ? kBF16 : kF16>(w, hi);
}
// Whether one of a pair's exponents is all ones (an infinity or NaN), in bits 15, 31 (the
// others are of no meaning).
template <bool BF16>
__device__ __forceinline__ uint32_t nonfinite(uint32_t w) {
  constexpr uint32_t m = BF16 ? 0x7f807f80u : 0x7c007c00u, one = BF16 ? 0x00800080u : 0x04000400u;
  return (w & m) + one;
}
// Two e4m3 values, nearest.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}
__device__ __forceinline__ void lds_f32x2(uint32_t addr, float& a, float& b) {
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(a), "=f"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ void sts_f32x2(uint32_t addr, float a, float b) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ void sts_b32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts_s8(uint32_t addr, int v) {
  asm volatile("st.shared.s8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ int lds_s8(uint32_t addr) {
  int v;
  asm volatile("ld.shared.s8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// 32 bytes, aligned to them.
__device__ __forceinline__ void stg_b32x8(void* to, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// Low k bits (none for k <= 0, all for k >= 32).
__device__ __forceinline__ uint32_t below(int k) {
  return k <= 0 ? 0u : (k >= 32 ? 0xffffffffu : (1u << k) - 1u);
}

template <int QT, int D, bool FP8, int PLAN>
__global__ void __launch_bounds__(Cfg<QT, D, FP8>::kThreads, 1)
    packed_attn_tc_kernel(const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ CUtensorMap tmQ, const PackedArgs a) {
  using C = Cfg<QT, D, FP8>;
  constexpr bool SMALL = PLAN != kPlanned;
  constexpr bool kBf16 = !FP8 && QT == kBF16;  // operand type of the products
  constexpr float kLift = kBf16 ? 0.f : kF16Lift;
  constexpr int NX = C::kGroups, KV = C::kKv;
  constexpr int kBarS = C::kBarS, kBarP = C::kBarP, kBarP2 = C::kBarP2, kBarO = C::kBarO, kBarQRaw = C::kBarQRaw,
                kBarQFull = C::kBarQFull, kBarQFree = C::kBarQFree, kBarOFull = C::kBarOFull,
                kBarOFree = C::kBarOFree, kBarStat = C::kBarStat, kBarLook = C::kBarLook, kBarItem = C::kBarItem,
                kBarItemFree = C::kBarItemFree;
  // Positions of the V tiles in use, and the barriers that say they are ready: the ring's,
  // or the two converted buffers'.
  constexpr int KB = C::kKStages, VB = FP8 ? 2 : C::kVStages;
  constexpr int kKReady = C::kBarKFull, kKFree = C::kBarKEmpty;
  constexpr int kVReady = FP8 ? C::kBarCVFull : C::kBarVFull, kVFree = FP8 ? C::kBarCVFree : C::kBarVEmpty;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = smem_addr(smem_raw);
  const uint32_t sQ = base + C::kQ, sK = base + C::kK, sV = base + C::kV;
  const uint32_t sVc = base + C::kVc;
  const uint32_t sVt = FP8 ? sVc : sV;  // 16-bit V tiles
  auto bar = [&](int i) -> uint32_t { return base + C::kBar + 8u * i; };
  const uint32_t* tslot = reinterpret_cast<const uint32_t*>(smem_raw + C::kSlot);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (base & 1023u) {  // the tiles would be misplaced (not so without static shared memory)
    if (tid == 0) atomicOr(a.err, PA_DEVERR_TIMEOUT);
    return;
  }
  if (tid == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmQ);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(bar(C::kBarKFull + i), 1);
      mbar_init(bar(C::kBarKEmpty + i), 1);
      mbar_init(bar(C::kBarVFull + i), 1);
      mbar_init(bar(C::kBarVEmpty + i), FP8 ? 128 : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarS + i), 1);
      mbar_init(bar(kBarP + i), kGroupThreads);
      mbar_init(bar(kBarP2 + i), kGroupThreads);
      mbar_init(bar(kBarO + i), 1);
      mbar_init(bar(kBarQFull + i), FP8 ? 128 : 1);
      mbar_init(bar(kBarOFull + i), 1);
      mbar_init(bar(kBarOFree + i), 128);
      mbar_init(bar(kBarStat + i), kGroupThreads);
      mbar_init(bar(kBarLook + i), 4);
      mbar_init(bar(C::kBarCVFull + i), 128);
      mbar_init(bar(C::kBarCVFree + i), 1);
      mbar_init(bar(C::kBarDrain + i), 1);
    }
    for (int i = 0; i < kItemRing; ++i) {
      mbar_init(bar(kBarItem + i), 1);
      mbar_init(bar(kBarItemFree + i), C::kThreads / 32);
    }
    mbar_init(bar(kBarQRaw), 1);
    mbar_init(bar(kBarQFree), 1);
    sts_b32(base + C::kSkip, 0);
    sts_b32(base + C::kSkip + 4, 0);
    fence_mbar_init();
  }
  if (warp == 0) tc::tmem_alloc(base + C::kSlot, kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tslot;
  griddep_wait();  // the plan, and behind it the caches and queries, are written
  griddep_launch_dependents();
  if constexpr (SMALL) {
    if (tid == 0 && PLAN == kSmallCut) reinterpret_cast<PackedJoin*>(a.plan + packed_joins_at(a.ctas))[blockIdx.x].n = 0;
    __syncthreads();  // (before the K warp may note a join)
  }

  // Item k from the ring, and done with it (every warp says so, of every item).
  auto item_at = [&](int k, PackedItem* it) -> bool {
    const int at = k % kItemRing;
    if (!wait_all(bar(kBarItem + at), k / kItemRing)) return false;
    uint32_t w[12];
#pragma unroll
    for (int i = 0; i < 3; ++i)
      lds_v4(base + C::kItem + 48 * at + 16 * i, w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    *it = PackedItem{static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]),  static_cast<int>(w[3]),
                     static_cast<int>(w[4]), static_cast<int>(w[5]), static_cast<int>(w[6]),  static_cast<int>(w[7]),
                     static_cast<int>(w[8]), static_cast<int>(w[9]), static_cast<int>(w[10]), 0};
    return true;
  };
  auto item_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarItemFree + k % kItemRing));
  };

  if (warp >= C::kMmaS) {
    if constexpr (C::kSplitRegs)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (warp == C::kLoadK || warp == C::kLoadV) {
      // ------------------------------------------------------------ producers
      // Lanes 0..kSlices-1 each look up one 16-token slice of a tile in the block
      // table and copy its 128-byte boxes; slices behind the range are not loaded.
      const bool is_v = warp == C::kLoadV;
      const CUtensorMap* map = is_v ? &tmV : &tmK;
      const int stages = is_v ? C::kVStages : C::kKStages;
      const uint32_t dst0 = (is_v ? sV : sK) + lane * 2048;
      const int full0 = is_v ? C::kBarVFull : C::kBarKFull, empty0 = is_v ? C::kBarVEmpty : C::kBarKEmpty;
      bool ok = true;
      Ring r;
      int c = 0;  // tiles so far
      // first row of this lane's slice of tile n, -1 behind the range
      auto row_of = [&](int b, int kvh, int start, int hi, int n, int nt) -> int {
        const int pos0 = start + n * KV + 16 * lane;
        if (lane >= C::kSlices || pos0 > hi || n >= nt) return -1;
        const int lb = pos0 / a.bs;
        int blk = a.block_tables[static_cast<size_t>(b) * a.MB + lb];
        if (static_cast<unsigned>(blk) >= static_cast<unsigned>(a.NB)) {
          atomicOr(a.err, PA_DEVERR_BLOCK_ID);
          blk = 0;
        }
        return (blk * a.Hkv + kvh) * a.bs + (pos0 - lb * a.bs);
      };
      // Works out item k and puts it into the ring (the K warp); returns its first row.
      const int me = blockIdx.x;
      int whole = 0, pairs = 0, wsz = 0;
      int2 share = make_int2(0, 0);
      if constexpr (!SMALL) {
        whole = a.plan[kPkWhole], pairs = a.plan[kPkPairs], wsz = a.plan[kPkWsz];
        share = reinterpret_cast<const int2*>(a.plan + packed_ctas_at())[me];
      }
      SmallPlan<PLAN == kSmallWhole> sp;
      if constexpr (SMALL) {
        if (!is_v) sp.begin(a, lane, me);
      }
      auto publish = [&](int k) -> int {
        PackedItem it = {};
        it.nt = -1;
        if constexpr (SMALL) {
          sp.next(a, lane, me, &it);
        } else {
          int p = whole ? me : share.x + k;
          if (whole && k > 0) {
            int taken = 0;
            if (lane == 0) taken = atomicAdd(a.plan + kPkNext, 1);
            p = a.ctas + __shfl_sync(kFull, taken, 0);
          }
          if (p < (whole ? pairs : share.y)) {
            const int u = p / a.Hkv;
            const int4* rec = reinterpret_cast<const int4*>(a.plan + packed_units_at(a.ctas)) + 3 * static_cast<size_t>(u);
            const int4 x = rec[0], y = rec[1];
            it = PackedItem{x.x, p - u * a.Hkv, x.y, x.z, x.w, y.x, y.y, y.z, 0, y.w, -1, 0};
            if (!whole) cut(rec[2].x + it.kvh * pair_places(it.nt, it.ntok > a.tpg), a.tpg, wsz, me, &it);
          }
        }
        const int at = k % kItemRing;
        if (k >= kItemRing) ok = wait_all(bar(kBarItemFree + at), k / kItemRing - 1) && ok;
        if (lane == 0 && ok) {
          const uint32_t to = base + C::kItem + 48 * at;
          sts_v4(to, make_uint4(it.b, it.kvh, it.row0, it.ntok));
          sts_v4(to + 16, make_uint4(it.pos0, it.first, it.lo, it.hi));
          sts_v4(to + 32, make_uint4(it.tile0, it.nt, it.slot, 0));
          mbar_arrive(bar(kBarItem + at));
        }
        __syncwarp();
        return row_of(it.b, it.kvh, (it.lo & ~15) + it.tile0 * KV, it.hi, 0, it.nt);
      };
      // Item -1 stands for the start: nothing but the first item to be worked out. (One copy
      // of each piece of code: what the warps of a CTA run in turn has to share the
      // instruction cache, whose misses show in every kernel time here. A small step is
      // over too soon for that, and 0.3 us faster with the first item by itself.)
      int row = -1, later = -1;
      if (SMALL && !is_v) row = publish(0);
      for (int k = SMALL ? 0 : -1; ok; ++k) {
        int b = 0, kvh = 0, start = 0, hi = 0, nt = 0;  // (in uniform registers)
        if (k >= 0) {
          PackedItem it;
          if (!(ok = item_at(k, &it))) break;
          b = __shfl_sync(kFull, it.b, 0);
          kvh = __shfl_sync(kFull, it.kvh, 0);
          start = __shfl_sync(kFull, (it.lo & ~15) + it.tile0 * KV, 0);
          hi = __shfl_sync(kFull, it.hi, 0);
          nt = __shfl_sync(kFull, it.nt, 0);
          item_done(k);
          if (nt < 0) break;
        }
#pragma unroll 1
        for (int n = is_v ? -1 : 0; n < max(nt, 1); ++n) {
          const int next = row_of(b, kvh, start, hi, n + 1, nt);  // looked up while the wait below runs
          if (n >= 0 && n < nt) {
            if (c >= stages && !(ok = wait_all(bar(empty0 + r.stage), r.phase ^ 1))) break;
            const uint32_t full = bar(full0 + r.stage);
            const int nslices = __popc(__ballot_sync(kFull, row >= 0));
            if (lane == 0) mbar_arrive_expect_tx(full, nslices * C::kRawBoxes * 2048);
            __syncwarp();
            if (row >= 0) {
              const uint32_t dst = dst0 + r.stage * C::kRing;
#pragma unroll
              for (int box = 0; box < static_cast<int>(C::kRawBoxes); ++box)
                tma_load_2d(dst + box * C::kBox, map, box * (FP8 ? 128 : 64), row, full);
            }
            __syncwarp();
            r.next(stages);
            ++c;
          }
          row = next;
          // the next item, once this one's first copies are on their way
          if (!is_v && n == max(min(nt, 2), 1) - 1) {
            later = publish(k + 1);
            if (!ok) break;
          }
        }
        if (!is_v) row = later;
      }
      if (!ok) {
        if (lane == 0) atomicOr(a.err, PA_DEVERR_TIMEOUT);
        for (int i = max(c - stages, 0); i < c; ++i)  // no copy outlives the CTA
          (void)mbar_wait_bounded(bar(full0 + i % stages), (i / stages) & 1, kDrainNs);
      }
    } else {
      // ------------------------------------------------------------ products
      // The warps stay together, so that what they issue with is uniform; their own
      // instructions are on the critical path.
      const uint32_t tm = __shfl_sync(kFull, tmem, 0);
      bool ok = true;
      Ring ring;
      uint32_t jobs = 0, live = 0;
      int done = 0;  // releases of K or V committed
      if (warp == C::kMmaS) {
        // (a negative scale flips the sign of A, Q)
        const uint32_t idS = tc::idesc_f16(kRows, KV, kBf16, false) | (a.score_scale < 0.f ? 1u << 13 : 0u);
        const uint64_t dQ = tc::sdesc_sw128(sQ, 16, 1024);
        const uint64_t dK = tc::sdesc_sw128(sK, 16, 1024);
        auto job = [&](bool own_rows) {
          const int x = jobs & 1;
          // the buffer's last P has been used
          if (jobs >= 2 && !(ok = wait_all(bar(kBarO + x), (jobs - 2) >> 1))) return;
          tc::fence_after_sync();
          const uint64_t q = dQ + (own_rows && x ? C::kQBytes >> 4 : 0);
          // FP8: the terms of Q's e4m3 sum, box by box of 128 head dims
          constexpr int kParts = FP8 ? C::kTerms * static_cast<int>(C::kRawBoxes) : C::kBoxes;
          constexpr int kAtOnce = NX == 2 ? 1 : kParts;
#pragma unroll kAtOnce
          for (int i = 0; i < kParts; ++i) {
            const int box = FP8 ? i / C::kTerms : i;
            mma4_ss_all<FP8>(tm + C::kColS + KV * x, q + (((FP8 ? C::q_region(i % C::kTerms, box) : i) * C::kQBox) >> 4),
                             dK + ((ring.stage * C::kRing + box * C::kBox) >> 4), idS, i > 0);
          }
          commit_all(bar(kBarS + x));
          ++jobs;
        };
        for (int k = 0; ok; ++k) {
          PackedItem it;
          if (!(ok = item_at(k, &it))) break;
          const int nt = __shfl_sync(kFull, it.nt, 0), row0 = __shfl_sync(kFull, it.row0, 0);
          const int head = __shfl_sync(kFull, it.kvh, 0) * a.G;
          const bool dual = NX == 2 && __shfl_sync(kFull, it.ntok, 0) > a.tpg;
          item_done(k);
          if (nt < 0) break;
          if (nt == 0) continue;
          {
            // Q, once the last item's products are done with it: a row tile's tokens times
            // the group's heads are one box a 64 head dims. (Rows behind the unit's are
            // other sequences', or zeros behind the last: not used.)
            if (live > 0 && !(ok = wait_all(bar(kBarQFree), live - 1))) break;
            if (lane == 0) {
              const int row_tiles = dual ? 2 : 1;
              const uint32_t full = bar(FP8 ? kBarQRaw : kBarQFull + (live & 1));
              mbar_arrive_expect_tx(full, row_tiles * C::kBoxes * a.tpg * a.G * 128);
              for (int xt = 0; xt < row_tiles; ++xt)
#pragma unroll
                for (int box = 0; box < C::kBoxes; ++box)
                  tma_load_3d(sQ + xt * C::kQBytes + box * C::kQBox, &tmQ, box * 64, head, row0 + xt * a.tpg, full);
            }
            __syncwarp();
          }
          if (!(ok = wait_all(bar(kBarQFull + (live & 1)), live >> 1))) {
            if (FP8) (void)mbar_wait_bounded(bar(kBarQRaw), live & 1, kDrainNs);
            else (void)mbar_wait_bounded(bar(kBarQFull + (live & 1)), (live >> 1) & 1, kDrainNs);
            break;  // (no copy outlives the CTA)
          }
          ++live;
#pragma unroll 1
          for (int n = 0; n < nt; ++n) {
            if (!(ok = wait_all(bar(kKReady + ring.stage), ring.phase))) break;
#pragma unroll 1
            for (int i = dual ? 2 : 1; i > 0 && ok; --i) job(dual);
            if (!ok) break;
            commit_all(bar(kKFree + ring.stage));
            ring.next(KB);
            ++done;
          }
          commit_all(bar(kBarQFree));
        }
      } else {
        constexpr uint32_t idO = tc::idesc_f16(kRows, D, kBf16, true);
        const uint64_t dV = tc::sdesc_sw128(sVt, C::kBox, 1024);
        int left = 0;  // jobs of this item
        // of each group: items begun in its O (the parity is all that counts, a bit each),
        // whether there was one, whether O holds something of this item
        uint32_t o_items = 0, o_any = 0, begun = 0;
        auto job = [&](bool masked) {
          const int x = jobs & 1, g = NX == 2 ? x : 0;
          if (!(begun >> g & 1)) {  // the last item's result has been read
            if ((o_any >> g & 1) && !(ok = wait_all(bar(kBarOFree + g), (o_items >> g) ^ 1))) return;
            o_items ^= 1u << g;
            o_any |= 1u << g;
          }
          if (!(ok = wait_all(bar(kBarP + x), jobs >> 1))) return;
          tc::fence_after_sync();
          volatile uint32_t* skip = reinterpret_cast<volatile uint32_t*>(smem_raw + C::kSkip) + x;
          if (masked && __any_sync(kFull, *skip != 0)) {  // the group has added this tile itself
            if (lane == 0) *skip = 0;
            __syncwarp();
          } else {
            // the half of the weights that is written first, then the other
            constexpr int kSteps = KV / 32;  // of 16 tokens a half
            const uint32_t o = tm + C::kColO + D * g, p = tm + C::kColS + KV * x;
            const uint64_t v = dV + ((ring.stage * C::kTile) >> 4);
            mma_ts_all<kSteps>(o, p, v, idO, begun >> g & 1);
            if (!(ok = wait_all(bar(kBarP2 + x), jobs >> 1))) return;
            tc::fence_after_sync();
            mma_ts_all<kSteps>(o, p + half_col(KV), v + 128 * kSteps, idO, 1u);
          }
          commit_all(bar(kBarO + x));
          begun |= 1u << g;
          ++jobs;
          // the group's last of this item: with two groups one of the last two
          if (--left < NX) {
            commit_all(bar(kBarOFull + g));
            begun &= ~(1u << g);
          }
        };
        for (int k = 0; ok; ++k) {
          PackedItem it;
          if (!(ok = item_at(k, &it))) break;
          const int nt = __shfl_sync(kFull, it.nt, 0);
          const int ntok = __shfl_sync(kFull, it.ntok, 0), start = __shfl_sync(kFull, (it.lo & ~15) + it.tile0 * KV, 0);
          const bool dual = NX == 2 && ntok > a.tpg;
          // tiles that all rows attend to in full lie between (the groups look through the others)
          const int sure_hi = (a.tree ? __shfl_sync(kFull, it.first, 0) : __shfl_sync(kFull, it.pos0, 0) + 1) - start;
          const int end = a.tree ? __shfl_sync(kFull, it.hi, 0) + 1 : __shfl_sync(kFull, it.pos0, 0) + ntok;
          const int sure_lo = (a.window > 0 ? end - a.window : 0) - start;
          item_done(k);
          if (nt < 0) break;
          if (nt == 0) continue;
          left = dual ? 2 * nt : nt;
#pragma unroll 1
          for (int n = 0; n < nt; ++n) {
            if (!(ok = wait_all(bar(kVReady + ring.stage), ring.phase))) break;
#pragma unroll 1
            for (int i = dual ? 2 : 1; i > 0 && ok; --i) job(n * KV < sure_lo || (n + 1) * KV > sure_hi);
            if (!ok) break;
            commit_all(bar(kVFree + ring.stage));
            ring.next(VB);
            ++done;
          }
        }
      }
      // no product and no arrival outlives the CTA
      if (!ok && lane == 0) atomicOr(a.err, PA_DEVERR_TIMEOUT);
      const uint64_t limit = ok ? kWaitNs : kDrainNs;
      const int drain = warp == C::kMmaS ? C::kBarDrain : C::kBarDrain + 1;
      const int free0 = warp == C::kMmaS ? kKFree : kVFree, bufs = warp == C::kMmaS ? KB : VB;
      commit_all(bar(drain));
      (void)mbar_wait_bounded(bar(drain), 0, limit);
      for (int i = 0; i < bufs && i < done; ++i)
        (void)mbar_wait_bounded(bar(free0 + i), ((done - 1 - i) / bufs) & 1, limit);
      __syncwarp();
    }
  } else if (warp >= C::kStoreWarp) {
    if constexpr (C::kSplitRegs)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kStoreRegs));
    // ---------------------------------------------------- queries in, results out
    const int wr0 = (warp - C::kStoreWarp) * 32;  // first row of this warp
    const int r = wr0 + lane;                   // row = tensor-memory lane
    const uint32_t trow = tmem + (static_cast<uint32_t>(wr0) << 16);
    const uint32_t mul = (65536u + a.G - 1) / a.G;  // row / G = row * mul >> 16, rows < 256
    // rows of out start on 32 bytes
    const bool wide = ((reinterpret_cast<uintptr_t>(a.out) | (static_cast<uintptr_t>(a.out_stride) << 1)) & 31) == 0;
    bool ok = true;
    uint32_t o_items = 0;  // items of each group so far (the parity, a bit each)
    uint32_t jobs = 0;
    // the results of an item, items in order
    auto store = [&](int k) {
      PackedItem item;  // (into uniform registers)
      if (!(ok = item_at(k, &item))) return;
      const int ntok = __shfl_sync(kFull, item.ntok, 0), nt = __shfl_sync(kFull, item.nt, 0);
      const int row0 = __shfl_sync(kFull, item.row0, 0), kvh = __shfl_sync(kFull, item.kvh, 0);
      const int slot = __shfl_sync(kFull, item.slot, 0);
      item_done(k);
      const bool dual = NX == 2 && ntok > a.tpg;
      const int nj = dual ? 2 * nt : nt;
      const uint32_t s = jobs & 1;  // group of the item's first job
      jobs += nj;
      const int g0 = NX == 2 ? static_cast<int>(s) : 0;  // the group with the first job
      const bool both = NX == 2 && nj > 1;
      // a group's result of this item is complete
      auto complete = [&](int g) {
        ok = ok && wait_all(bar(kBarOFull + g), o_items >> g) && wait_all(bar(kBarStat + g), o_items >> g);
        o_items ^= 1u << g;
        tc::fence_after_sync();
        return ok;
      };
      const bool join = both && !dual;  // both groups' O are the same rows'
#pragma unroll 1
      for (int q = 0; q < (dual ? 2 : 1); ++q) {
        const int xt = dual ? g0 ^ q : 0;  // row tile (the group of the first job first)
        const int ga = dual ? xt : g0;     // the group whose O holds its rows
        const int rows = min(ntok - xt * a.tpg, a.tpg) * a.G;
        if (nj > 0 && (!complete(ga) || (join && !complete(ga ^ 1)))) return;
        auto release = [&]() {  // the groups may go on in O
          if (nj > 0) {
            tc::fence_before_sync();
            mbar_arrive(bar(kBarOFree + ga));
            if (join) mbar_arrive(bar(kBarOFree + (ga ^ 1)));
          }
        };
        if (wr0 >= rows) {
          release();
        } else {
          float m = kFloor, l = 0.f, f_own = 0.f, f_other = 0.f;
          if (nj > 0) {
            lds_f32x2(base + C::kStat + (ga * kRows + r) * 8, m, l);
            f_own = 1.f;
            if (join) {
              float m1, l1;
              lds_f32x2(base + C::kStat + ((ga ^ 1) * kRows + r) * 8, m1, l1);
              const float top = fmaxf(m, m1);
              f_own = ex2(m - top);
              f_other = ex2(m1 - top);
              l = l * f_own + l1 * f_other;
              m = top;
            }
          }
          // O by 32 columns, the next ones on their way while these are stored. A lane has a
          // row: it stores whole 32-byte sectors of it. (Rows turned around between four
          // lanes first, for 64-byte pieces, held O 3,000 cycles longer.)
          const uint32_t t_own = trow + C::kColO + D * ga, t_other = trow + C::kColO + D * (ga ^ 1);
          char* to;  // this row's
          if (slot < 0) {
            // an empty row is zeros (its O is, as its weights were); a NaN in the sum stays one
            const float inv = l == 0.f ? 0.f : a.v_scale / l;
            f_own *= inv;
            f_other *= inv;
            const int t = static_cast<int>((r * mul) >> 16), h = r - t * a.G;
            to = static_cast<char*>(a.out) + 2 * (static_cast<size_t>(row0 + xt * a.tpg + t) * a.out_stride +
                                                  static_cast<size_t>(kvh * a.G + h) * D);
          } else {
            f_own *= a.v_scale;
            f_other *= a.v_scale;
            to = reinterpret_cast<char*>(a.part + static_cast<size_t>(slot) * packed_slot_floats(a.slot_rows, D) +
                                         static_cast<size_t>(xt * kRows + r) * D);
          }
          // columns d0 .. d0 + 15, taken and scaled
          auto put = [&](int d0, uint32_t (&v)[16]) {
            if (slot >= 0) {
              if (r < rows) stg_b32x8(to + 4 * d0, v), stg_b32x8(to + 4 * d0 + 32, v + 8);
            } else {
              uint32_t p[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                p[i] = pack16x2<QT == kBF16>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
              if (r < rows) {
                if (wide) {
                  stg_b32x8(to + 2 * d0, p);
                } else {
                  reinterpret_cast<uint4*>(to + 2 * d0)[0] = make_uint4(p[0], p[1], p[2], p[3]);
                  reinterpret_cast<uint4*>(to + 2 * d0)[1] = make_uint4(p[4], p[5], p[6], p[7]);
                }
              }
            }
            __syncwarp();
          };
          uint32_t v[16], w[16];
          if (nj == 0 || join) {
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 16) {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = w[i] = 0u;
              if (join) tc::ld16(t_own + d0, v), tc::ld16(t_other + d0, w);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                v[i] = __float_as_uint(fmaf(__uint_as_float(w[i]), f_other, __uint_as_float(v[i]) * f_own));
              if (d0 + 16 == D) release();  // before the last stores
              put(d0, v);
            }
          } else {
            tc::ld16_async(t_own, v);
            tc::ld16_async(t_own + 16, w);
#pragma unroll 1
            for (int d0 = 32;; d0 += 32) {
              tc::wait_ld();
              tc::pin(v);
              tc::pin(w);
              if (d0 == D) release();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f_own);
              put(d0 - 32, v);
              if (d0 < D) tc::ld16_async(t_own + d0, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f_own);
              put(d0 - 16, w);
              if (d0 == D) break;
              tc::ld16_async(t_own + d0 + 16, w);
            }
          }
          if (slot >= 0 && r < rows) {
            float* stat = a.part + static_cast<size_t>(slot) * packed_slot_floats(a.slot_rows, D) +
                          static_cast<size_t>(a.slot_rows) * D + xt * kRows + r;
            stat[0] = m - kLift;
            stat[a.slot_rows] = l;
          }
        }
      }
    };
    if constexpr (FP8) {
      // A warp takes every fourth octet of rows, a lane a row of it and every fourth
      // 16-byte chunk: the eight lanes of an access then have eight rows, whose chunks the
      // swizzle puts into different banks, in the raw tile as in the f16 one. One chunk at a
      // time: with 2, 4 at once 1,024 rows on 16,384 tokens take 229, 242 us instead of 216 (more
      // are faster by themselves, but their instructions displace the other warps'). With
      // one softmax group there is room for 8: 411 us at head_dim 256, with 4 417.
      constexpr int kOctets = KV / 32, kParts = D / 64;
      const int o0 = warp - C::kStoreWarp, sub = lane & 7, ch = lane >> 3;
      const uint32_t from0 = (8 * o0 + sub) * 128 + ((ch ^ sub) << 4);
      const uint32_t to_lo = (8 * o0 + sub) * 128 + (((2 * ch) ^ sub) << 4), to_hi = to_lo ^ 16;
      // Rows [r_lo, r_hi) are converted, the others become zeros.
      auto convert = [&](uint32_t src, uint32_t dst, int r_lo, int r_hi) {
        constexpr int N = NX == 2 ? 1 : 8;  // chunks of a lane at once
        static_assert(kOctets * kParts == 8, "chunks a lane");
        const bool part = r_lo > 0 || r_hi < KV;
#pragma unroll 1
        for (int g = 0; g < 8; g += N) {
          uint32_t w[N][4];
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const int p = (g + j) / kOctets, k = (g + j) % kOctets;
            lds_v4(src + (from0 ^ ((p & 1) << 6)) + (p >> 1) * C::kBox + 4096 * k, w[j][0], w[j][1], w[j][2], w[j][3]);
          }
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const int p = (g + j) / kOctets, k = (g + j) % kOctets, row = 8 * (o0 + 4 * k) + sub;
            uint32_t (&x)[4] = w[j];
            if (part && (row < r_lo || row >= r_hi)) x[0] = x[1] = x[2] = x[3] = 0u;
            uint32_t h[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              h[2 * i] = e4m3x2_to_f16x2(static_cast<uint16_t>(x[i] & 0xffffu));
              h[2 * i + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(x[i] >> 16));
            }
            sts_v4(dst + to_lo + p * C::kBox + 4096 * k, make_uint4(h[0], h[1], h[2], h[3]));
            sts_v4(dst + to_hi + p * C::kBox + 4096 * k, make_uint4(h[4], h[5], h[6], h[7]));
          }
        }
      };
      // This warp's rows of Q as sums of e4m3 values, D / 16 lanes a row. A row is scaled by a
      // power of two to a largest magnitude in [2^7, 2^8), and each term is what the ones
      // before it leave: of 4 bits each, two hold a bf16 and three an f16 exactly, but
      // for what lies below 2^-10, 2^-17 of the row's largest. A row with an infinity or NaN
      // is NaN.
      auto convert_q = [&](int ntok, uint32_t which) {
        constexpr int kLanes = D / 16, kPass = 32 / kLanes;  // lanes a row, rows a pass
        const int l = lane % kLanes;
#pragma unroll 1
        for (int xt = 0; xt < (NX == 2 && ntok > a.tpg ? 2 : 1); ++xt) {
          const uint32_t tile = sQ + xt * C::kQBytes;
          const int rows = min(ntok - xt * a.tpg, a.tpg) * a.G;
#pragma unroll 1
          for (int r0 = wr0; r0 < min(rows, wr0 + 32); r0 += 2 * kPass) {
            float v[2][16];
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // two passes at once
              const int row = r0 + u * kPass + lane / kLanes;
              const uint32_t at = tile + row * 128 + (l >> 2) * C::kQBox;
              uint32_t w[8];
              lds_v4(at + (((2 * (l & 3)) ^ (row & 7)) << 4), w[0], w[1], w[2], w[3]);
              lds_v4(at + (((2 * (l & 3) + 1) ^ (row & 7)) << 4), w[4], w[5], w[6], w[7]);
              uint32_t top = 0;  // largest magnitudes of the even and the odd elements, as bits
#pragma unroll
              for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
#pragma unroll
              for (int o = kLanes / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(kFull, top, o));
              const int ex = __float_as_int(f32_of<QT>(max(top >> 16, top & 0xffffu), 0)) >> 23;  // 255: not finite
              // (a row below 2^-119 has scores of zero for any weight)
              const int sh = ex == 255 ? 0 : max(ex - 134, -126);
              const float m = __int_as_float(ex == 255 ? 0x7fc00000 : (127 - sh) << 23);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[u][i] = f32_of<QT>(w[i >> 1], i & 1) * m;
              if (l == 0 && row < rows) sts_s8(base + C::kShift + (which & 1) * NX * kRows + xt * kRows + row, sh);
            }
            __syncwarp();  // (all of the rows has been read)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int row = r0 + u * kPass + lane / kLanes;
#pragma unroll
              for (int t = 0; t < C::kTerms; ++t) {
                uint32_t e[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                  const uint32_t pair = e4m3x2_of(v[u][i], v[u][i + 1]);
                  e[i >> 2] |= pair << (8 * (i & 2));
                  const uint32_t back = e4m3x2_to_f16x2(static_cast<uint16_t>(pair));
                  v[u][i] -= f32_of<kF16>(back, 0);
                  v[u][i + 1] -= f32_of<kF16>(back, 1);
                }
                if (row < rows)
                  sts_v4(tile + row * 128 + C::q_region(t, l >> 3) * C::kQBox + (((l & 7) ^ (row & 7)) << 4),
                         make_uint4(e[0], e[1], e[2], e[3]));
              }
            }
            __syncwarp();
          }
        }
        fence_proxy_async();
        mbar_arrive(bar(kBarQFull + (which & 1)));
      };
      int c = 0;                  // tiles so far
      uint32_t live = 0;          // items with tiles so far
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        int nt, ntok, v_lo, v_hi;  // tiles, tokens, range of V rows from the first tile on
        {
          PackedItem it;
          if (!(ok = item_at(k, &it))) break;
          const int start = (it.lo & ~15) + it.tile0 * KV;
          nt = it.nt;
          ntok = it.ntok;
          v_lo = it.lo - start;
          v_hi = it.hi + 1 - start;
        }
        int n = 0;
        do {
          if (n < nt) {
            if (n == 0) {
              if (!(ok = wait_all(bar(kBarQRaw), live))) break;
              convert_q(ntok, live);
              ++live;
            }
            const int stage = c % C::kVStages;
            if (!(ok = wait_all(bar(C::kBarVFull + stage), c / C::kVStages))) break;
            if (c > 1 && !(ok = wait_all(bar(C::kBarCVFree + (c & 1)), (c - 2) >> 1))) break;
            convert(sV + stage * C::kRing, sVc + (c & 1) * C::kTile, v_lo - n * KV, v_hi - n * KV);
            fence_proxy_async();  // the f16 tile, visible to the tensor core
            mbar_arrive(bar(C::kBarCVFull + (c & 1)));
            mbar_arrive(bar(C::kBarVEmpty + stage));  // reload the stage
            ++c;
          }
          if (n == 0 && k > 0) store(k - 1);
        } while (++n < nt && ok);
        if (nt < 0) break;
      }
    } else {
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        PackedItem it;
        if (!(ok = item_at(k, &it)) || it.nt < 0) break;
        store(k);
      }
    }
    if (!ok && lane == 0) atomicOr(a.err, PA_DEVERR_TIMEOUT);
  } else {
    // ---------------------------------------------------------------- softmax
    if constexpr (C::kSplitRegs)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    const int x = warp >> 2;        // group
    const int r = tid - x * kRows;  // row of the tile = tensor-memory lane
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tO = trow + C::kColO + D * x;
    const int tok_r = r / a.G;
    bool ok = true;
    uint32_t jobs = 0;   // of all items before
    uint32_t mine = 0;   // of this group
    uint32_t done = 0;   // items of this group
    uint32_t live = 0;   // items with tiles
    uint32_t tiles = 0;  // K/V tiles of the items before
    uint32_t looks = 0;  // tiles whose V was looked through
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      // What is the same for the whole group, in uniform registers; positions from the
      // first tile's first token on.
      int nt, row0, ntok, first, u_lo, u_hi, pos0, start;
      {
        PackedItem it;
        if (!(ok = item_at(k, &it))) break;
        start = __shfl_sync(kFull, (it.lo & ~15) + it.tile0 * KV, 0);
        nt = __shfl_sync(kFull, it.nt, 0);
        row0 = __shfl_sync(kFull, it.row0, 0);
        ntok = __shfl_sync(kFull, it.ntok, 0);
        first = __shfl_sync(kFull, it.first, 0) - start;
        u_lo = __shfl_sync(kFull, it.lo, 0) - start;      // the unit's range
        u_hi = __shfl_sync(kFull, it.hi, 0) + 1 - start;  // (its end)
        pos0 = __shfl_sync(kFull, it.pos0, 0) - start;
      }
      item_done(k);
      if (nt < 0) break;
      const bool dual = NX == 2 && ntok > a.tpg;
      const int nj = dual ? 2 * nt : nt;
      if (nj == 0) continue;
      const int s = jobs & 1;  // S buffer (and group) of the item's first job
      jobs += nj;
      // this group's jobs: every one (one group), or those of its parity
      const int j0 = NX == 2 ? (s ^ x) : 0, step = NX == 2 ? 2 : 1;
      const uint32_t which = live++;
      if (j0 >= nj) {
        tiles += nt;
        continue;
      }
      // this row: the range that it attends to (a tree: before the drafted tokens)
      const int xt = dual ? x : 0;
      const int tok = xt * a.tpg + tok_r;
      const bool valid = tok_r < a.tpg && tok < ntok;
      const bool alive = __any_sync(kFull, valid);
      uint64_t bits = 0;
      int r_lo, r_hi;
      if (a.tree) {
        const int nb = u_hi - first;  // drafted tokens that have a bit
        if (valid) bits = static_cast<uint64_t>(a.tree[row0 + tok]) & (nb >= 64 ? ~0ull : (1ull << nb) - 1);
        r_hi = first;
        r_lo = r_hi + __popcll(bits);  // its place + 1
      } else {
        r_hi = r_lo = pos0 + tok + 1;
      }
      r_lo = a.window > 0 ? max(r_lo - a.window, -start) : -start;
      if (!valid) bits = 0, r_hi = -start, r_lo = 0x40000000;
      // What all rows of the group attend to for sure: a tile inside takes no look
      // through V.
      const int sure_hi = a.tree ? first : pos0 + xt * a.tpg + 1;
      const int last = a.tree ? u_hi : pos0 + min(ntok, (xt + 1) * a.tpg);
      const int sure_lo = a.window > 0 ? last - a.window : -start;
      // (never zero, so that a masked score stays -inf)
      float sc = fmaxf(fabsf(a.score_scale), FLT_MIN);
      if constexpr (FP8) {
        if (!(ok = wait_all(bar(kBarQFull + (which & 1)), which >> 1))) break;
        if (valid) sc = fmaxf(FLT_MIN, ldexpf(sc, lds_s8(base + C::kShift + (which & 1) * NX * kRows + xt * kRows + r)));
      }
      float ms = kFloor, l = 0.f;  // reference max (scaled, log2 units) and running sum
#pragma unroll 1
      for (int j = j0; j < nj; j += step, ++mine) {
        const int n = dual ? j >> 1 : j, t0 = n * KV;
        const int buf = NX == 2 ? x : ((s + j) & 1);
        const uint32_t phase = NX == 2 ? mine : mine >> 1;
        const uint32_t tS = trow + C::kColS + KV * buf;
        const bool all_in = __all_sync(kFull, !valid || (t0 >= r_lo && t0 + KV <= r_hi));
        uint32_t mask[KV / 32];
#pragma unroll
        for (int w = 0; w < KV / 32; ++w) mask[w] = 0xffffffffu;
        if (!all_in) {
#pragma unroll
          for (int w = 0; w < KV / 32; ++w) {
            mask[w] = below(r_hi - t0 - 32 * w) & ~below(r_lo - t0 - 32 * w);
            const int sh = 32 * w + t0 - first;  // bit of this word's first token
            if (sh > -32 && sh < 64)
              mask[w] |= sh >= 0 ? static_cast<uint32_t>(bits >> sh) : static_cast<uint32_t>(bits << -sh);
          }
        }
        bool skip = false;
        // A tile that some row does not attend to in full.
        if (t0 < sure_lo || t0 + KV > sure_hi) {
          const uint32_t c = tiles + n, stage = c % VB;
          // S before V, but for a first look at a first tile: this S follows earlier products of
          // the group, so that the phase of V's barrier before the one that is waited for is
          // complete, and all warps have read what the last look found (one group: the last but one).
          if ((c >= VB || looks > 0) && !(ok = wait_all(bar(kBarS + buf), phase))) break;
          if (!(ok = wait_all(bar(kVReady + stage), c / VB))) break;
          const uint32_t vt = sVt + stage * C::kTile;
          uint32_t bad = 0;
          if (r < KV) {
            const int pos = t0 + r;
            const uint32_t at = vt + r * 128;
            if (pos >= u_lo && pos < u_hi) {
#pragma unroll 1
              for (int i = 0; i < 8 * C::kBoxes; i += 4) {
                uint32_t w[4][4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  lds_v4(at + (i >> 3) * C::kBox + ((((i & 4) + e) ^ (r & 7)) << 4), w[e][0], w[e][1], w[e][2], w[e][3]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  bad |= nonfinite<kBf16>(w[e][0]) | nonfinite<kBf16>(w[e][1]) | nonfinite<kBf16>(w[e][2]) |
                         nonfinite<kBf16>(w[e][3]);
              }
              bad &= 0x80008000u;
            } else if (!FP8 && (!dual || !(j & 1))) {
              // outside of the range: zeros, before the tile's first product
#pragma unroll 1
              for (int i = 0; i < 8 * C::kBoxes; ++i)
                sts_v4(at + (i >> 3) * C::kBox + (i & 7) * 16, make_uint4(0u, 0u, 0u, 0u));
            }
          }
          fence_proxy_async();
          // what any warp of the group has found
          const uint32_t look = base + C::kLook + 16 * (NX == 2 ? x : looks & 1);
          const bool any_bad = __any_sync(kFull, bad != 0);
          if (lane == 0) {
            sts_b32(look + 4 * (warp & 3), any_bad ? 1u : 0u);
            mbar_arrive(bar(kBarLook + x));
          }
          if (!(ok = wait_all(bar(kBarLook + x), looks++))) break;
          uint32_t w[4];
          lds_v4(look, w[0], w[1], w[2], w[3]);
          skip = (w[0] | w[1] | w[2] | w[3]) != 0;
        }
        if (!(ok = wait_all(bar(kBarS + buf), phase))) break;
        tc::fence_after_sync();
        if (alive) {
          uint32_t sv[KV / 32][32];
          const bool old = j != j0;  // O holds something
          tc::ld32_async(tS, sv[0]);
          tc::ld32_async(tS + 32, sv[1]);
          tc::wait_ld(sv[0], sv[1]);
          if constexpr (KV == 128) {  // the second half on its way during the first's maximum
            tc::ld32_async(tS + 64, sv[2]);
            tc::ld32_async(tS + 96, sv[3]);
          }
          // masked scores of two rows of sv as -inf
          auto mask_out = [&](int c) {
            if (!all_in) {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                if (__all_sync(kFull, !valid || mask[c + q] == 0xffffffffu)) continue;
#pragma unroll
                for (int i = 0; i < 32; ++i) sv[c + q][i] = (mask[c + q] >> i) & 1 ? sv[c + q][i] : 0xff800000u;
              }
            }
          };
          mask_out(0);
          float mxp[8];  // eight independent partial maxima (raw scores)
#pragma unroll
          for (int i = 0; i < 8; ++i) mxp[i] = -INFINITY;
          auto add_max = [&](int c) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int i = 0; i < 32; i += 2)
                mxp[(i >> 1) & 7] = fmax3(mxp[(i >> 1) & 7], __uint_as_float(sv[c + q][i]),
                                          __uint_as_float(sv[c + q][i + 1]));
          };
          add_max(0);
          if constexpr (KV == 128) {
            tc::wait_ld(sv[2], sv[3]);
            mask_out(2);
            add_max(2);
          }
          const float mxr = fmaxf(fmaxf(fmaxf(mxp[0], mxp[1]), fmaxf(mxp[2], mxp[3])),
                                  fmaxf(fmaxf(mxp[4], mxp[5]), fmaxf(mxp[6], mxp[7])));
          const float mx = fmaxf(mxr * sc, kFloor);
          const bool grow = mx > ms + kRescaleAbove;
          if (!old) {
            ms = mx;  // nothing accumulated yet
          } else if (__any_sync(kFull, grow)) {
            // O is complete up to the group's last job: with two groups S was issued after
            // its product; one group has to wait for it
            if (NX == 1) ok = wait_all(bar(kBarO + (buf ^ 1)), (mine - 1) >> 1);
            tc::fence_after_sync();
            const float alpha = grow ? ex2(ms - mx) : 1.f;
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 16) {
              uint32_t ov[16];
              tc::ld16(tO + d0, ov);
              const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const float2 o = __fmul2_rn(score_pair(ov, i), a2);
                ov[i] = __float_as_uint(o.x);
                ov[i + 1] = __float_as_uint(o.y);
              }
              tc::st16(tO + d0, ov);
            }
            l *= alpha;
            if (grow) ms = mx;
          }
          // P = 2^(s * sc - ms + kLift), packed in pairs over the scores' columns. It is
          // rounded to the products' 16-bit type, which the tensor core needs beside V's,
          // against sums in fp32 of the unrounded ones: at most 2^-8 of each weight for
          // bf16, for f16 2^-11 of it and, where it is subnormal, 2^-32 of the reference's
          // weight.
          const float2 sc2 = make_float2(sc, sc);
          float2 sp[4];
          // half of the tile's weights, from score `first` of sv rows c ..., to column col
          auto weigh = [&](int c, int first, int col) {
            const float2 nms2 = make_float2(kLift - ms, kLift - ms);
#pragma unroll
            for (int q = 0; q < KV / 64; ++q) {
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int e = first + 32 * q + 2 * i;
                const float2 t = __ffma2_rn(score_pair(sv[c + (e >> 5)], e & 31), sc2, nms2);
                const float p0 = ex2(t.x), p1 = ex2(t.y);
                sp[i & 3] = __fadd2_rn(sp[i & 3], make_float2(p0, p1));
                pk[i] = pack16x2<kBf16>(p0, p1);
              }
              tc::st16(tS + col + 16 * q, pk);
            }
          };
          if (skip) {
            // Infinities or NaN in V: weights times rows on the CUDA cores, attended
            // positions only.
            const uint32_t vt = sVt + ((tiles + n) % VB) * C::kTile;
            if (NX == 1 && old) ok = wait_all(bar(kBarO + (buf ^ 1)), (mine - 1) >> 1);
            // (the item's first job: the storing warps have read the last item's O)
            if (!old && done > 0) ok = wait_all(bar(kBarOFree + x), done - 1) && ok;
            tc::fence_after_sync();
#pragma unroll 1
            for (int e0 = 0; e0 < KV; e0 += 32) {
              tc::ld32_async(tS + e0, sv[0]);
              tc::wait_ld(sv[0]);
              uint32_t w = 0;
#pragma unroll
              for (int i = 0; i < KV / 32; ++i) w = e0 == 32 * i ? mask[i] : w;
              float sum = 0.f;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float p = (w >> i) & 1 ? ex2(fmaf(__uint_as_float(sv[0][i]), sc, kLift - ms)) : 0.f;
                sv[0][i] = __float_as_uint(p);
                sum += p;
              }
              l += sum;
#pragma unroll 1
              for (int d0 = 0; d0 < D; d0 += 16) {
                uint32_t ov[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) ov[i] = 0u;
                if (old || e0 > 0) tc::ld16(tO + d0, ov);
#pragma unroll 4
                for (int e = 0; e < 32; ++e) {
                  const bool on = (w >> e) & 1;
                  if (!__any_sync(kFull, on)) continue;
                  // (the weights sit in registers: a chain of selects picks one)
                  float p = 0.f;
#pragma unroll
                  for (int i = 0; i < 32; ++i) p = i == e ? __uint_as_float(sv[0][i]) : p;
                  const int row = e0 + e;
#pragma unroll
                  for (int q = 0; q < 2; ++q) {
                    uint32_t v[4];
                    const int c = (d0 & 63) / 8 + q;
                    lds_v4(vt + (d0 >> 6) * C::kBox + row * 128 + ((c ^ (row & 7)) << 4), v[0], v[1], v[2], v[3]);
                    if (on) {
#pragma unroll
                      for (int i = 0; i < 8; ++i)
                        ov[8 * q + i] = __float_as_uint(fmaf(p, op_f32<kBf16>(v[i >> 1], i & 1),
                                                             __uint_as_float(ov[8 * q + i])));
                    }
                  }
                }
                tc::st16(tO + d0, ov);
                tc::wait_st();
              }
            }
            if (r == 0) sts_b32(base + C::kSkip + 4 * buf, 1u);
            tc::fence_before_sync();
            mbar_arrive(bar(kBarP + buf));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) sp[i] = make_float2(0.f, 0.f);
            // half of the weights, which the products start on, then the other half
            weigh(0, 0, 0);
            tc::wait_st();
            tc::fence_before_sync();
            mbar_arrive(bar(kBarP + buf));
            weigh(KV == 128 ? 2 : 0, KV == 128 ? 0 : 32, half_col(KV));
            const float2 s01 = __fadd2_rn(sp[0], sp[1]), s23 = __fadd2_rn(sp[2], sp[3]);
            const float2 st = __fadd2_rn(s01, s23);
            l += st.x + st.y;
          }
        } else {
          mbar_arrive(bar(kBarP + buf));
        }
        if (!ok) break;
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(bar(kBarP2 + buf));
      }
      tiles += nt;
      if (!ok) break;
      // the statistics, once the last ones have been read
      if (done > 0 && !(ok = wait_all(bar(kBarOFree + x), done - 1))) break;
      sts_f32x2(base + C::kStat + (x * kRows + r) * 8, ms, l);
      mbar_arrive(bar(kBarStat + x));
      ++done;
    }
    if (!ok && lane == 0) atomicOr(a.err, PA_DEVERR_TIMEOUT);
  }

  // every product has completed (the issuing warps waited for them)
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int QT, int D, bool FP8, int PLAN>
cudaError_t launch_typed(const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tq,
                         const PackedArgs& a, cudaStream_t s, bool pdl) {
  using C = Cfg<QT, D, FP8>;
  // a function attribute of the current device's context: set every time, a host-side
  // store
  cudaError_t e = cudaFuncSetAttribute(packed_attn_tc_kernel<QT, D, FP8, PLAN>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  if constexpr (C::kSplitRegs) {
    // the softmax warps wait for registers that the block must have been given
    static const int regs = [] {
      cudaFuncAttributes f;
      return cudaFuncGetAttributes(&f, packed_attn_tc_kernel<QT, D, FP8, PLAN>) == cudaSuccess ? f.numRegs : 0;
    }();
    if (regs < C::kLaunchRegs) return cudaErrorLaunchOutOfResources;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, packed_attn_tc_kernel<QT, D, FP8, PLAN>, tk, tv, tq, a);
}

template <int QT, int PLAN>
cudaError_t launch_dim(bool fp8, int D, const CUtensorMap& tk, const CUtensorMap& tv,
                       const CUtensorMap& tq, const PackedArgs& a, cudaStream_t s, bool pdl) {
  if (fp8) {
    if (D == 128) return launch_typed<QT, 128, true, PLAN>(tk, tv, tq, a, s, pdl);
    if (D == 256) return launch_typed<QT, 256, true, PLAN>(tk, tv, tq, a, s, pdl);
    return cudaErrorInvalidValue;
  }
  if (D == 64) return launch_typed<QT, 64, false, PLAN>(tk, tv, tq, a, s, pdl);
  if (D == 128) return launch_typed<QT, 128, false, PLAN>(tk, tv, tq, a, s, pdl);
  if (D == 256) return launch_typed<QT, 256, false, PLAN>(tk, tv, tq, a, s, pdl);
  return cudaErrorInvalidValue;
}

template <int PLAN>
cudaError_t launch_packed(int qt, bool fp8, int D, const CUtensorMap& tk, const CUtensorMap& tv,
                          const CUtensorMap& tq, const PackedArgs& a, cudaStream_t s, bool pdl) {
  return qt == kBF16 ? launch_dim<kBF16, PLAN>(fp8, D, tk, tv, tq, a, s, pdl)
                     : launch_dim<kF16, PLAN>(fp8, D, tk, tv, tq, a, s, pdl);
}

}  // namespace
}  // namespace pa
