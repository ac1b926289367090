// Layout of the plan of a ragged step (packed prompts or drafted trees), written
// by the plan kernel (packed_plan.cu) and read by the attention (packed_tc.cu)
// and the join (packed_merge.cu).
//
// Sequence b's queries are the packed rows [query_start[b], query_start[b + 1]).
// They are cut into units of tpu tokens; the (token, head) rows of a unit and a KV
// head, at most 256 (128 with head_dim 256), are one matrix Q, and the unit's
// K/V range is walked in tiles of kv tokens. An item is a run of a unit's tiles
// that one CTA works through.
//   - whole mode: every unit is one item; items are sorted by their tiles, most
//     first, and dealt out to the CTAs there and back (0 .. C-1, C-1 .. 0, ...).
//   - split mode: the tiles of all units form one flat index space, unit- then KV
//     head-major, with a few places before each unit's for its way in and out, and
//     CTA w takes [w * wsz, (w + 1) * wsz) of it. Item u + w is what CTA w has of the
//     tiles of unit u (counted over KV heads): unique, because the walk through the
//     (unit, CTA) grid is a monotone staircase. A unit cut between CTAs
//     leaves a partial result with each, in slot 2 w if it is CTA w's first item,
//     else 2 w + 1 (its last); the merge joins them.
// A unit that attends to nothing counts as one tile (its rows are zeros).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace pa {

struct PackedItem {  // 12 words an item
  int b, kvh;        // sequence, KV head
  int row0, ntok;    // first packed row and tokens of the unit
  int pos0;          // position of its first token
  int first;         // position of the sequence's first query
  int lo, hi;        // positions that its rows may attend to
  int tile0, nt;     // K/V tiles of it, from lo rounded down to 16 tokens
  int slot;          // partial result, -1: the unit is whole
  int pad;
};
struct PackedJoin {  // 8 words a CTA: the unit cut at the CTA's end that starts in it
  int row0, ntok, kvh;
  int n;             // partials, 0: none
  int slot0, slot1;  // the first and the second; each other one is 2 behind the last
  int pad[2];
};
constexpr int kPackedHead = 8;
enum { kPkWhole = 0, kPkItems = 1 };  // header words: mode, items in whole mode

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
__host__ __device__ constexpr inline size_t packed_items_at(int ctas) {
  return packed_joins_at(ctas) + 8 * static_cast<size_t>(ctas);
}
__host__ __device__ constexpr inline size_t packed_plan_words(int ctas, size_t items) {
  return packed_items_at(ctas) + 12 * items;
}
// Floats of a partial result: `rows` rows of D, their maxima and their sums.
__host__ __device__ constexpr inline size_t packed_slot_floats(int rows, int D) {
  return static_cast<size_t>(rows) * (D + 2);
}

}  // namespace pa
