// The attention of small ragged steps, which every CTA plans by itself, pairs cut (packed_tc.cuh).
#include "packed_tc.cuh"

namespace pa {
cudaError_t packed_launch_small(int qt, bool fp8, int D, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CUtensorMap& tq, const PackedArgs& a, cudaStream_t s, bool pdl) {
  return launch_packed<kSmallCut>(qt, fp8, D, tk, tv, tq, a, s, pdl);
}
}  // namespace pa
