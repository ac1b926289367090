// Argument structs and launchers of the ragged steps: packed prompts and drafted
// trees (packed_plan.cu, packed_tc.cu, packed_merge.cu), and the moves of cached
// rows (cache_moves.cu). Host-only types.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <vector_types.h>
#include <stdint.h>

#include "packed_plan.cuh"
#include "step_ops.h"

namespace pa {

struct PackedPlanArgs {
  const int32_t* query_start;   // [B + 1]
  const int32_t* seq_lens;      // [B]
  int32_t* plan;
  int32_t* err;
  int B, T, MB, bs, Hkv, window;
  int tpu;                      // tokens a unit
  int kv;                       // tokens a K/V tile
  int ctas;                     // of the attention
  int tpg;                      // tokens a row tile
  int min_places;               // least places a CTA in split mode
  int split_places;             // what a split costs a CTA
  bool tree;
};
cudaError_t packed_plan_launch(const PackedPlanArgs& a, cudaStream_t s, bool pdl);

struct PackedArgs {
  void* out;                    // [T, Hq, D], rows of out_stride elements
  const int32_t* block_tables;  // [B, MB]
  const int64_t* tree;          // [T] ancestor bits, or null: causal
  int32_t* plan;
  float* part;                  // partial results
  int32_t* err;
  const int32_t* query_start;   // [B + 1], small steps: each CTA plans by itself
  const int32_t* seq_lens;      // [B]
  int B, T, tpu, kv, min_places;  // as in PackedPlanArgs
  int64_t out_stride;
  int ctas, Hkv, G, bs, MB, NB, window;
  int tpg;                      // tokens a row tile: 128 / G
  int slot_rows;                // rows of a partial result
  float score_scale;            // scale * log2(e) (* k_scale for FP8)
  float v_scale;                // FP8: applied to the output
};
cudaError_t packed_launch(int qt, bool fp8, int D, const CUtensorMap& tk, const CUtensorMap& tv,
                          const CUtensorMap& tq, const PackedArgs& a, cudaStream_t s, bool pdl);
// Small steps, which have no plan kernel: pairs cut between CTAs, or whole pairs and no join.
cudaError_t packed_launch_small(int qt, bool fp8, int D, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CUtensorMap& tq, const PackedArgs& a, cudaStream_t s, bool pdl);
cudaError_t packed_launch_whole(int qt, bool fp8, int D, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CUtensorMap& tq, const PackedArgs& a, cudaStream_t s, bool pdl);

struct PackedMergeArgs {
  void* out;
  const float* part;
  const int32_t* plan;
  int64_t out_stride;
  int ctas, G, D, tpg, slot_rows;
  bool small;                   // the plan is complete only behind the attention
};
cudaError_t packed_merge_launch(int out_type, const PackedMergeArgs& a, cudaStream_t s, bool pdl);

struct CopyBlocksArgs {
  void* kc;                     // [layers, NB, Hkv, bs, D], layers k_layer bytes apart
  void* vc;
  const int2* block_pairs;      // [pairs] (source, target)
  int32_t* err;
  int64_t k_layer, v_layer;     // bytes
  int layers, NB, pairs;
  int units;                    // 16-byte units a block
  int chunks;                   // CTAs a block
};
int copy_blocks_chunk();        // 16-byte units a CTA moves
cudaError_t copy_blocks_launch(const CopyBlocksArgs& a, cudaStream_t s);

struct CompactArgs {
  void* kc;                     // [layers, NB, Hkv, bs, D], layers k_layer bytes apart
  void* vc;
  const int32_t* block_tables;  // [B, MB]
  const int32_t* seq_lens;      // [B]
  const int32_t* query_start;   // [B + 1]
  const int32_t* kept;          // [B, M]
  const int32_t* num_kept;      // [B]
  int32_t* lens_out;            // [B]
  int32_t* kept_tokens;         // [B] or null
  int32_t* err;
  int64_t k_layer, v_layer;     // bytes
  int layers, B, MB, NB, Hkv, bs, M;
  int row_units;                // 16-byte units a row
  int share;                    // planes (layer, K or V) a CTA, set by the launcher
  FastDiv unit_div, row_div;    // by a row of all heads, by a row; set by the launcher
};
cudaError_t compact_cache_launch(const CompactArgs& a, int num_sms, cudaStream_t s);

}  // namespace pa
