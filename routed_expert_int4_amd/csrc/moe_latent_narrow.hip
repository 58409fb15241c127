// Attention over the latent cache in 8 bits.
//
// Codes stay codes in LDS, half the bytes of the bf16 tile on every way, and
// become bf16 where the matrix instructions take them: a key's codes with its
// row's power of two, which each lane has one of, a value's without, the power
// of two then being part of the weight (2^e p is exact).
//
// Half the bytes leave room for three tiles: loads are two ahead.  One token per
// sequence is bound by the cache's bytes, 640 + 4 per row, and by what a tile
// costs its workgroup, 2.47 us, about equally: 32 sequences of 16384 rows 111 us
// (3.1 TB/s; 103 without the loads), the bf16 cache 132 to 141.  Several tokens are
// bound by instructions: a wave has 34 matrix instructions to a tile, 128
// conversions and some 175 other vector instructions, which the matrix cores do
// not hide: 11 x 5 tokens (trees) over 9001 ragged rows 76 us (0.56 PFLOP/s), of
// which the join takes 9 and the runs' beginnings and ends some 12.  Loads moved
// between the scores, the exchange and the values: no difference; the two groups
// of four waves a step apart, three barriers to a tile: none.
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
