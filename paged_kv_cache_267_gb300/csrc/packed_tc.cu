// The attention of ragged steps whose plan is a kernel's (packed_tc.cuh).
#include "packed_tc.cuh"

namespace pa {
cudaError_t packed_launch(int qt, bool fp8, int D, const CUtensorMap& tk, const CUtensorMap& tv,
                          const CUtensorMap& tq, const PackedArgs& a, cudaStream_t s, bool pdl) {
  return launch_packed<kPlanned>(qt, fp8, D, tk, tv, tq, a, s, pdl);
}
}  // namespace pa
