// Decode kernel instantiations for the tails of shared-prefix steps, bf16 caches.
#include "decode.cuh"

namespace pa {

PA_DECODE_FAMILY(sh_bf16, kBF16, kBF16, false, true)

}  // namespace pa
