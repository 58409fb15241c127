// Attention over the bf16 latent cache.
#include "moe_latent_device.h"

namespace moe {

bool latent_shape_supported(int rank, int rope) { return rope == kRopeWidth && (rank == 512 || rank == 256); }

size_t latent_workspace(int B, int max_q, int heads, int rank, int max_len) {
    const LatentCut c = latent_cut(B, max_q, heads, max_len, false);  // no fewer runs than for rows of 8 bits
    return (size_t)c.runs * c.group * 2 * c.rows * (rank + 2) * sizeof(float);
}

hipError_t launch_latent_attention(const LatentArgs& a, hipStream_t s) {
    if (a.cache_scale) return launch_latent_narrow(a, s);
    if (a.rank == 512)
        launch_rank<512, false>(a, s);
    else
        launch_rank<256, false>(a, s);
    return hipGetLastError();
}

}  // namespace moe
