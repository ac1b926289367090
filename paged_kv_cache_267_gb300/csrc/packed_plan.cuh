// Layout of the plan of a ragged step (packed prompts or drafted trees), written
// by the plan kernel (packed_plan.cu) and read by the attention (packed_tc.cu)
// and the join (packed_merge.cu).
//
// Sequence b's queries are the packed rows [query_start[b], query_start[b + 1]).
// They are cut into units of tpu tokens; the (token, head) rows of a unit and a KV
// head, at most 256 (128 with head_dim 256), are one matrix Q, and the unit's
// K/V range is walked in tiles of kv tokens. Pair p = unit * Hkv + KV head. An item is
// what a CTA works through of a pair:
//   - whole mode: every pair is one item. Units are sorted by their cost, most first; CTA
//     w begins with pair w and then takes the next one that is left (a counter).
//   - split mode: the costs of all pairs form one space of places, in which a pair has
//     kOutPlaces for its way in and out and then tile_places() a tile, and CTA w has the
//     tiles that begin in [w * wsz, (w + 1) * wsz). A pair cut between CTAs leaves a
//     partial result with each, in slot 2 w + 1 with the one that has its first tile and
//     2 w with the others (each CTA has one of either kind at most); the merge joins
//     them.
// A unit that attends to nothing counts as one tile (its rows are zeros).
// Steps of few sequences and pairs have no plan kernel: every CTA works out its own part of
// split mode, and leaves the merge its note, or takes whole pairs in turn.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace pa {

struct PackedUnit {  // 12 words a unit
  int b;             // sequence
  int row0, ntok;    // first packed row and tokens of the unit
  int pos0;          // position of its first token
  int first;         // position of the sequence's first query
  int lo, hi;        // positions that its rows may attend to
  int nt;            // K/V tiles of it, from lo rounded down to 16 tokens
  int place;         // split mode: places before it
  int pad[3];
};
struct PackedJoin {  // 8 words a CTA: the pair that begins in it and goes on in the next
  int row0, ntok, kvh;
  int n;             // partial results, 0: none
  int pad[4];
};
// Header words: mode, pairs, places a CTA, counter of the pairs taken behind the first.
constexpr int kPackedHead = 8;
enum { kPkWhole = 0, kPkPairs = 1, kPkWsz = 2, kPkNext = 3 };

// Costs, in quarters of a tile of two row tiles: a pair's way in and out, a tile. (Of a
// 16-prompt batch a tile takes 2,650 cycles and a pair 7,000 besides; one row tile takes
// as long where an e4m3 cache is converted. The exact weight matters little: with 2 for one row
// tile, 64 trees on an e4m3 cache take 228 us instead of 233, 32 on a bf16 one 58.4 instead of
// 59.0.)
constexpr int kOutPlaces = 8;
__host__ __device__ constexpr inline int tile_places(bool dual) { return dual ? 4 : 3; }

struct PackedShape {
  int kv;    // tokens a K/V tile
  int rows;  // row tiles a unit: 2, or 1 with head_dim 256
};
__host__ __device__ constexpr inline PackedShape packed_shape(int D) {
  return D == 256 ? PackedShape{64, 1} : PackedShape{128, 2};
}

// Sections of the plan, in words from its start.
__host__ __device__ constexpr inline size_t packed_ctas_at() { return kPackedHead; }  // int2 a CTA
__host__ __device__ constexpr inline size_t packed_joins_at(int ctas) {
  return packed_ctas_at() + 2 * static_cast<size_t>((ctas + 1) & ~1);
}
__host__ __device__ constexpr inline size_t packed_units_at(int ctas) {
  return packed_joins_at(ctas) + 8 * static_cast<size_t>(ctas);
}
__host__ __device__ constexpr inline size_t packed_plan_words(int ctas, size_t units) {
  return packed_units_at(ctas) + 12 * units;
}
// Floats of a partial result: `rows` rows of D, their maxima and their sums.
__host__ __device__ constexpr inline size_t packed_slot_floats(int rows, int D) {
  return static_cast<size_t>(rows) * (D + 2);
}

__host__ __device__ constexpr inline int pair_places(int nt, bool dual) {
  return kOutPlaces + (nt > 1 ? nt : 1) * tile_places(dual);
}

// Unit u of sequence b, whose n new tokens begin at row q0 and end at position len.
__host__ __device__ __forceinline__ PackedUnit packed_unit(int b, int u, int q0, int n, int len, int tpu, int kv,
                                                           int window, bool tree) {
  PackedUnit it;
  const int t0 = u * tpu;
  it.b = b;
  it.row0 = q0 + t0;
  it.ntok = n - t0 < tpu ? n - t0 : tpu;
  it.first = len - n;
  it.pos0 = it.first + t0;
  // causal: from the first token's window to the last token; tree: from the window of a
  // row with no ancestor to the last drafted token that a bit can name
  it.hi = tree ? it.first + (n < 64 ? n : 64) - 1 : it.pos0 + it.ntok - 1;
  const int from = tree ? it.first : it.pos0 + 1;
  it.lo = window > 0 && from > window ? from - window : 0;
  it.nt = it.hi >= it.lo ? (it.hi + 1 - (it.lo & ~15) + kv - 1) / kv : 0;
  it.place = 0;
  it.pad[0] = it.pad[1] = it.pad[2] = 0;
  return it;
}

// Tiles of a pair that begin before place x, counted from its first tile's.
__host__ __device__ constexpr inline int tiles_before(int x, int nt, int per) {
  const int t = x <= 0 ? 0 : (x + per - 1) / per;
  return t < nt ? t : nt;
}

}  // namespace pa
