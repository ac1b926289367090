// Layout of the plan of a shared-prefix decode step, written by the plan
// kernel (shared_plan.cu) and read by the prefix, decode and merge kernels.
//
// Sequences of group g share their first P tokens (P a multiple of the block
// size, so of 16). A row takes part when it is at least that long and no window
// cuts it, or one that reaches back over at least half of its length into them;
// rows [r0, r0 + n) are those from the first that does to the last. With S the
// largest window start of those that take part, rounded up to 16 (0 without
// windows), the prefix kernel computes the partial softmax of all of them over
// [S, P); the decode kernel covers the rest of their ranges, [start, S) and
// [P, L), and the whole range of every other row.
//
// The (query, head) rows of one KV head of a group, n * G of them, are cut into
// nut units of up pairs (sequences) each, at most 256 rows; a unit of at most
// 128 rows is computed by both softmax groups of its CTA, each on every other
// K/V tile, a larger one (dual) by one group per 128 rows.
// All K/V tiles of all units form one flat index space, group- then KV head-
// then unit-major; CTA w of the prefix kernel takes tiles [w * wsz, (w + 1) *
// wsz). A run of one CTA's tiles inside one unit is a segment; its partials go
// to slots
//   base_g + lid * up + i,  lid = unit + (w - wfirst),
// for the unit's index among the group's (KV head, unit) list, the first CTA
// that meets the group and pair i: unique because the
// walk through the (unit, CTA) grid is a monotone staircase. Slots have the
// decode partials' layout (one KV head's G columns of one sequence).
#pragma once

#include "pa_internal.h"

namespace pa {

constexpr int kSharedHead = 8;      // header words
// tiles a CTA of the prefix kernel; units of the decode kernel of one KV head; and
// units a warp of it. A (sequence, KV head) pair has a unit for each of the
// 16-token tiles that the decode kernel covers, and one before them for its way
// in and out (its queries, its partial: 0.8 us of a warp, where a tile takes 0.9;
// warps with a dozen pairs of a tile or two each otherwise end 8 us after the
// others' 24).
enum { kShWsz = 0, kShTails = 1, kShTailsWs = 2 };

struct SharedGroup {  // 12 words a group
  int r0, n;          // rows
  int table_row;      // r0, whose block table the prefix is read through
  int prefix;         // P - S, 0 when the group does not share
  int f0;             // first flat tile
  int nt;             // K/V tiles of the prefix
  int nut, up;        // units a KV head, pairs a unit
  int base;           // first partial slot (counted from the prefix region)
  int dual;           // its units have rows for both softmax groups
  int wfirst;         // first CTA that meets the group
  int first;          // S
};

struct SharedCta {  // 16 words a CTA of the prefix kernel
  int f0, f1;   // its flat tiles
  int group;    // the group of f0
  int pad;
  SharedGroup g;  // that group, so that a CTA starts on one load
};

struct SharedRow {  // 12 words a sequence
  int start;        // first position of its range
  int head;         // 16-token tiles of it before S
  int len;          // its length, inside the tables
  int pref;         // units of the decode kernel of the sequences before
  int tiles;        // 16-token tiles that it covers of this one
  int nt;           // K/V tiles of its prefix, 0: no part of it here
  int f0;           // first flat tile of its unit at KV head 0
  int kv_step;      // flat tiles between KV heads
  int slot0;        // slot of lid 0 for this sequence's pair
  int lid0;         // unit - wfirst at KV head 0 (added to the CTA)
  int up, nut;      // slots between lids, lids between KV heads
};

// Words of the plan: header, CTAs, groups, rows.
__host__ __device__ constexpr inline size_t shared_plan_words(int64_t B, int64_t NG, int ctas) {
  return kSharedHead + 16 * static_cast<size_t>(ctas) + 12 * static_cast<size_t>(NG) +
         12 * static_cast<size_t>(B);
}
__host__ __device__ __forceinline__ const SharedCta* shared_ctas(const int32_t* plan) {
  return reinterpret_cast<const SharedCta*>(plan + kSharedHead);
}
__host__ __device__ __forceinline__ const SharedGroup* shared_groups(const int32_t* plan, int ctas) {
  return reinterpret_cast<const SharedGroup*>(plan + kSharedHead + 16 * ctas);
}
__host__ __device__ __forceinline__ const SharedRow* shared_rows(const int32_t* plan, int ctas,
                                                                 int NG) {
  return reinterpret_cast<const SharedRow*>(plan + kSharedHead + 16 * ctas + 12 * NG);
}

}  // namespace pa
