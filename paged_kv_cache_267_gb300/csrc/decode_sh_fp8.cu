// Decode kernel instantiations for the tails of shared-prefix steps, FP8 e4m3 caches.
#include "decode.cuh"

namespace pa {

PA_DECODE_FAMILY(sh_fp8_f16, kE4M3, kF16, false, true)
PA_DECODE_FAMILY(sh_fp8_bf16, kE4M3, kBF16, false, true)

}  // namespace pa
