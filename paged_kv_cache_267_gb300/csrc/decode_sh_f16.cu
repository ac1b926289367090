// Decode kernel instantiations for the tails of shared-prefix steps, f16 caches.
#include "decode.cuh"

namespace pa {

PA_DECODE_FAMILY(sh_f16, kF16, kF16, false, true)

}  // namespace pa
