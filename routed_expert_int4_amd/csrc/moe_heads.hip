// One product per head: out[t][h][n] = sum_k x[t][h][k] w[h][n][k], bf16 in
// and out, fp32 sums.  The absorbed form of latent attention needs it on
// both sides: queries into the latent space (K = head width, N = rank) and
// attention outputs back out (K = rank, N = value width).
//
// Every shape it serves is memory bound (few operations per byte: at 1024
// tokens 8.6 GFLOP against 92 MB), so operands go from global memory straight
// to registers in matrix-core order, without LDS: the matrix instruction's
// rows are n and its columns are tokens, so that a lane holds four
// consecutive n of one token and stores eight bytes.
#include "moe_block.h"
#include "moe_block_device.h"

namespace moe {
namespace {

// 16 bytes at k of a row of K values; zero past its end.
__device__ __forceinline__ bf16x8 row_chunk(const uint16_t* row, int k, int K) {
    u32x4 u = *as_global<u32x4>(row + (k < K ? k : 0));
    if (k >= K) u = u32x4{0, 0, 0, 0};
    return __builtin_bit_cast(bf16x8, u);
}

// Few tokens: one token, 64 heads, 128 to 512 takes 3.6 us, of which reading
// 8.4 MB of weights is 1.8.  A wave owns NT x TT tiles of 16 n by 16 tokens; the four waves of a
// workgroup lie along n.
template <int NT, int TT>
__global__ void __launch_bounds__(256) head_linear_kernel(HeadArgs a) {
    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int h = blockIdx.z;
    const int n0 = (blockIdx.x * 4 + wave_in_block()) * NT * 16, t0 = blockIdx.y * TT * 16;
    if (n0 >= a.N) return;
    const uint16_t* w[NT];
    const uint16_t* x[TT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int n = n0 + i * 16 + col;
        w[i] = a.w + ((long)h * a.N + (n < a.N ? n : a.N - 1)) * a.K;
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        const int t = t0 + i * 16 + col;
        x[i] = a.x + (long)(t < a.T ? t : a.T - 1) * a.x_stride_t + h * a.x_stride_h;
    }
    f32x4 acc[NT][TT] = {};
    // 64 inner columns a step, the next step's loads in flight: a lane takes
    // 32 neighbouring bytes of each row, its part of two instructions (both
    // operands permute the inner columns alike)
    bf16x8 wf[2][NT][2], xf[2][TT][2];
    auto load = [&](int buf, int k0) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int k = k0 + quad * 16 + c * 8;
#pragma unroll
            for (int i = 0; i < NT; ++i) wf[buf][i][c] = row_chunk(w[i], k, a.K);
#pragma unroll
            for (int i = 0; i < TT; ++i) xf[buf][i][c] = row_chunk(x[i], k, a.K);
        }
    };
    auto multiply = [&](int buf) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < TT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[buf][i][c], xf[buf][j][c], acc[i][j], 0, 0, 0);
    };
    load(0, 0);
    for (int k0 = 0; k0 < a.K; k0 += 128) {
        if (k0 + 64 < a.K) load(1, k0 + 64);
        multiply(0);
        if (k0 + 64 >= a.K) break;
        if (k0 + 128 < a.K) load(0, k0 + 128);
        multiply(1);
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int t = t0 + j * 16 + col;
        if (t >= a.T) continue;
        uint16_t* o = a.out + (long)t * a.o_stride_t + h * a.o_stride_h;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int n = n0 + i * 16 + quad * 4;
            const u32x2 v = {pack_bf16(acc[i][j][0], acc[i][j][1]), pack_bf16(acc[i][j][2], acc[i][j][3])};
            if (n < a.N) *reinterpret_cast<u32x2*>(o + n) = v;  // N is a multiple of 4
        }
    }
}

// Many tokens: a wave keeps the weights of its NW x 16 rows and KC inner
// columns in registers and a workgroup of four passes over tiles
// of 64 tokens of one head, loaded asynchronously one ahead into the other of
// two LDS buffers: token rows lie heads * K apart in memory, and 64 KB in
// flight per CU are what reading them takes (1024 tokens x 64 heads, 512 to
// 128: through registers 50 us, 64 tokens per workgroup with the weights read
// again for each 38 us; so 20.5, 4.5 TB/s).  The 16-byte chunk c of row r sits at place
// c ^ (r & 15): the 16 rows of an operand read cover all banks.  Row m of
// instruction tile i is n = m / 4 * 4 NW + 4 i + m % 4, so that a lane holds
// 4 NW neighbouring outputs of one token.
template <int KC, int NW, int PER_CU>
__global__ void __launch_bounds__(256, PER_CU) head_linear_tile_kernel(HeadArgs a) {
    constexpr int TT = 4, kSteps = KC / 32, kChunks = KC / 8, kTileBytes = 64 * KC * 2;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kTileBytes];
    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4, wave = wave_in_block();
    // a head's workgroups lie on one die (they are dealt in turn)
    const int h = blockIdx.x, n0 = (blockIdx.y * 4 + wave) * NW * 16;
    const int tiles = (a.T + 63) / 64, turns = (a.K + KC - 1) / KC;
    const uint16_t* x = a.x + h * a.x_stride_h;
    const unsigned lds0 = lds_address(lds);
    auto issue = [&](int tile, int turn, int buf) {
#pragma unroll
        for (int i = 0; i < kTileBytes / 4096; ++i) {
            const int at = (i * 4 + wave) * 64 + lane, r = at / kChunks, k = turn * KC + ((at % kChunks) ^ (r & 15)) * 8;
            const int t = tile * 64 + r;
            const uint16_t* p = x + (long)t * a.x_stride_t + k;
            load_to_lds16(t < a.T && k < a.K ? static_cast<const void*>(p) : kZeros,
                          lds0 + buf * kTileBytes + (i * 4 + wave) * 1024);
        }
    };
    const uint16_t* w[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const int n = n0 + (col >> 2) * 4 * NW + i * 4 + (col & 3);
        w[i] = a.w + ((long)h * a.N + (n < a.N ? n : a.N - 1)) * a.K;
    }
    bf16x8 wf[NW][kSteps];
    // (complete on return: the compiler must not wait for weights inside the
    // loop, where the next tile is on its way)
    auto load_weights = [&](int turn) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int i = 0; i < NW; ++i) wf[i][s] = row_chunk(w[i], turn * KC + s * 32 + quad * 8, a.K);
        wait_vmem<0>();
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int i = 0; i < NW; ++i) asm volatile("" : "+v"(wf[i][s]));
    };
    int tile = blockIdx.z, buf = 0;
    issue(tile, 0, 0);
    load_weights(0);
    lds_barrier();
    for (; tile < tiles; tile += gridDim.z) {
        f32x4 acc[NW][TT] = {};
        for (int turn = 0; turn < turns; ++turn) {
            // what comes after this part: the next inner columns, or the next tile
            const bool last = turn + 1 == turns;
            const int next_tile = last ? tile + (int)gridDim.z : tile, next_turn = last ? 0 : turn + 1;
            const bool more = next_tile < tiles;
            if (more) issue(next_tile, next_turn, buf ^ 1);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                bf16x8 xf[TT];
#pragma unroll
                for (int j = 0; j < TT; ++j) {
                    const int r = j * 16 + col;
                    xf[j] = lds_chunk(lds0 + buf * kTileBytes + r * KC * 2 + ((s * 4 + quad) ^ (r & 15)) * 16);
                }
#pragma unroll
                for (int i = 0; i < NW; ++i)
#pragma unroll
                    for (int j = 0; j < TT; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[i][s], xf[j], acc[i][j], 0, 0, 0);
            }
            if (turns > 1 && more) load_weights(next_turn);  // more inner columns than the registers hold
            wait_vmem<0>();
            lds_barrier();  // the next part is in LDS, and every wave is done with this one
            buf ^= 1;
        }
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            const int t = tile * 64 + j * 16 + col;
            if (t >= a.T) continue;
            const int n = n0 + quad * 4 * NW;
            uint16_t* o = a.out + (long)t * a.o_stride_t + h * a.o_stride_h + n;
#pragma unroll
            for (int i = 0; i < NW; i += 2) {
                const u32x4 v = {pack_bf16(acc[i][j][0], acc[i][j][1]), pack_bf16(acc[i][j][2], acc[i][j][3]),
                                 pack_bf16(acc[i + 1][j][0], acc[i + 1][j][1]), pack_bf16(acc[i + 1][j][2], acc[i + 1][j][3])};
                if (n + i * 4 + 7 < a.N && a.out_vec) {
                    *reinterpret_cast<u32x4*>(o + i * 4) = v;
                } else {  // N is a multiple of 4
                    if (n + i * 4 < a.N) *reinterpret_cast<u32x2*>(o + i * 4) = u32x2{v[0], v[1]};
                    if (n + i * 4 + 4 < a.N) *reinterpret_cast<u32x2*>(o + i * 4 + 4) = u32x2{v[2], v[3]};
                }
            }
        }
    }
}

template <int NT, int TT>
void launch_rows(const HeadArgs& a, hipStream_t s) {
    const dim3 grid((a.N + 64 * NT - 1) / (64 * NT), (a.T + 16 * TT - 1) / (16 * TT), a.heads);
    hipLaunchKernelGGL((head_linear_kernel<NT, TT>), grid, dim3(256), 0, s, a);
}
template <int KC, int NW, int PER_CU>
void launch_tiles(const HeadArgs& a, hipStream_t s) {
    // workgroups that share a head's token tiles: enough of them to fill the chip
    const int blocks = (a.N + 64 * NW - 1) / (64 * NW), tiles = (a.T + 63) / 64;
    int share = (256 * PER_CU + a.heads * blocks - 1) / (a.heads * blocks);
    share = share < tiles ? share : tiles;
    hipLaunchKernelGGL((head_linear_tile_kernel<KC, NW, PER_CU>), dim3(a.heads, blocks, share), dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_head_linear(const HeadArgs& a, hipStream_t s) {
    // Few tokens: what counts is the weights' one reading (32 tokens, 64
    // heads, 128 to 512: 7.1 us, 8.9 in token tiles; 512 to 128: 8.4 and 8.0).
    if (a.T <= 16)
        launch_rows<1, 1>(a, s);
    else if (a.K <= 128 && a.T <= 64)
        launch_rows<1, 2>(a, s);
    else if (a.K <= 128)
        launch_tiles<128, 2, 4>(a, s);
    else
        launch_tiles<512, 2, 1>(a, s);
    return hipGetLastError();
}

}  // namespace moe
