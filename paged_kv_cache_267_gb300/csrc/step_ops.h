// Argument structs and launchers of the serving-step operators (pool_ops.cu,
// norm_cache.cu, shared_plan.cu, prefix_tc.cu). Host-only types.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// Division of 31-bit integers by a fixed d as a multiplication.
struct FastDiv {
  uint32_t mul, shift;
};
// (d = 1: mul 0, which stands for no division; d = 0 never divides)
inline FastDiv fast_div(uint32_t d) {
  if (d <= 1) return FastDiv{0, 0};
  uint32_t l = 1;
  while ((1ull << l) < d) ++l;
  return FastDiv{static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d), l - 1};
}
// The block pool (pool_ops.cu). in_place: lens_out is lens, or state_out is
// state; the last CTA to have read them then writes them.
struct PoolExtendArgs {
  int32_t* tables;               // [B, MB]
  const int32_t* lens;           // [B] before the step
  const int32_t* fresh;          // [B] new tokens
  const int32_t* free_list;      // [NF]
  int32_t* state;                // {free blocks, ticket}
  int32_t* lens_out;             // [B]
  int32_t* state_out;            // {free blocks, 0}
  int32_t* query_start;          // [B + 1]
  int64_t* slots;                // [T]
  int32_t* positions;            // [T]
  int32_t* err;                  // device error word
  int B, MB, bs, NF, T;
  FastDiv div;                   // by bs
  bool in_place;
  bool wide;                     // slots and positions are 16-byte aligned
};
struct PoolReleaseArgs {
  const int32_t* tables;         // [B, MB]
  const int32_t* lens;           // [B]
  const int32_t* released;       // [B], nonzero: give the blocks back
  const int32_t* shared;         // [B] tokens in blocks that stay, or null
  int32_t* free_list;            // [NF]
  int32_t* state;
  int32_t* lens_out;
  int32_t* state_out;
  int32_t* err;
  int B, MB, bs, NF;
  FastDiv div;                   // by bs
  bool in_place;
};
cudaError_t pool_extend_launch(const PoolExtendArgs& a, int num_sms, cudaStream_t s);
cudaError_t pool_release_launch(const PoolReleaseArgs& a, int num_sms, cudaStream_t s);

// Norm, rotation and cache write of a batch's projected rows (norm_cache.cu).
struct NormCacheArgs {
  const void* q;                 // [T, Hq, D], rows of q_stride elements
  const void* k;                 // [T, Hkv, D]
  const void* v;
  void* q_out;                   // [T, Hq, D]
  void* kc;                      // [NB, Hkv, bs, D]
  void* vc;
  const int64_t* slots;          // [T]
  const int32_t* positions;      // [T]
  const float* cos_sin;          // [NP, R]: R / 2 cosines, then R / 2 sines
  const void* q_weight;          // [D] or null (no norm)
  const void* k_weight;
  int32_t* err;
  int64_t q_stride, k_stride, v_stride, out_stride;  // elements a row
  int64_t NB;
  int T, Hq, Hkv, D, R, NP, bs;
  FastDiv per_row_div, bs_div;   // set by the launcher: by the units of a row, by bs
  float eps, k_scale, v_scale;
  bool interleaved;
};
cudaError_t norm_cache_launch(int type, bool fp8, const NormCacheArgs& a, int num_sms,
                              cudaStream_t s);

// Shared-prefix decode: the plan (shared_plan.cu) and the attention over the
// shared positions (prefix_tc.cu).
// Times that share the SMs between the prefix kernel and the decode kernel of a
// step, in nanoseconds of one SM while both run: a K/V tile of the prefix for
// two row tiles or one, a unit's way in and out (its queries and partials), a
// 16-token tile of a tail (one KV head), and what a CTA of each kernel costs
// besides.
struct SharedCost {
  float dual_ns, single_ns, unit_ns, tail_ns, prefix_ns, decode_ns;
};
struct SharedPlanArgs {
  const int32_t* group_starts;   // [NG + 1]
  const int32_t* prefix_lens;    // [NG]
  const int32_t* seq_lens;       // [B]
  int32_t* plan;                 // shared_plan_words(B, NG) words of workspace
  int32_t* err;
  int B, NG, MB, bs, Hkv, G, window;
  int kv, unit_rows;             // tokens a K/V tile, rows a unit
  bool halves;                   // small units are computed in two halves
  int ctas;                      // of the prefix kernel
  int whole;                     // more busy CTAs than this: take all SMs
  int decode_ctas, decode_per_sm;  // of the decode kernel
  int decode_warps, decode_min_tiles;  // a CTA; least tiles a warp
  bool wide_partials;            // a partial has 8 KB and more
  SharedCost cost;
  int min_tiles;                 // least K/V tiles a CTA
};
cudaError_t shared_plan_launch(const SharedPlanArgs& a, cudaStream_t s, bool pdl);

struct PrefixArgs {
  const void* q;                 // [B, Hq, D]
  const int32_t* block_tables;   // [B, MB]
  const int32_t* plan;           // written by the plan kernel
  float* part;                   // first prefix partial
  int32_t* err;
  int ctas;                      // the grid, which the plan's layout depends on
  int NG, Hq, Hkv, G, bs, MB, NB;
  float score_scale;             // scale * log2(e) (* k_scale for FP8)
  float v_scale;                 // FP8: applied to the partial outputs
};
// Tokens a K/V tile, rows a unit, and whether a unit of at most half of them
// is computed in two halves of the tiles.
struct PrefixShape {
  int kv, unit_rows;
  bool halves;
};
PrefixShape prefix_shape(int D);
cudaError_t prefix_launch(int qt, bool fp8, int D, const CUtensorMap& tk, const CUtensorMap& tv,
                          const PrefixArgs& a, int grid, cudaStream_t s, bool pdl);

// Joins the decode kernel's partials and the prefix kernel's (shared_merge.cu).
struct SharedMergeArgs {
  void* out;                     // [B, Hq, D]
  const float* part;             // all partials, the decode kernel's first
  const int32_t* plan;           // the step's
  int B, Hkv, G, D, NG, ctas;
  int part0;                     // first slot of the prefix partials
};
cudaError_t shared_merge_launch(int out_type, const SharedMergeArgs& a, cudaStream_t s, bool pdl);

}  // namespace pa
