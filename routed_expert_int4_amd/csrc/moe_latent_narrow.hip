// Attention over the latent cache in 8 bits.
//
// Codes stay codes in LDS, half the bytes of the bf16 tile on every way, and
// become bf16 where the matrix instructions take them: a key's codes with its
// row's power of two, which each lane has one of, a value's without, the power
// of two then being part of the weight (2^e p is exact).
#include "moe_latent_device.h"

namespace moe {

hipError_t launch_latent_narrow(const LatentArgs& a, hipStream_t s) {
    if (a.rank == 512)
        launch_rank<512, true>(a, s);
    else
        launch_rank<256, true>(a, s);
    return hipGetLastError();
}

}  // namespace moe
