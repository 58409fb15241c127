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

// A wave owns NT x TT tiles of 16 n by 16 tokens; the four waves of a
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

// Many tokens: a workgroup owns 64 tokens of one head and all n.  Their rows
// (KC inner columns at a time) are loaded asynchronously into LDS, all at
// once, so that a CU has 128 KB in flight (64-token rows lie heads * K apart
// in memory; through registers the same loads would be bound by latency at
// two waves per SIMD).  Weights come from the L2, which all token tiles of a
// head share.  The 16-byte chunk c of row r sits at place c ^ (r & 15): the
// 16 rows of an operand read cover all banks.
template <int KC>
__global__ void __launch_bounds__(256, 2) head_linear_tile_kernel(HeadArgs a) {
    constexpr int NT = 2, TT = 4, kSteps = KC / 32, kChunks = KC / 8;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[64 * KC * 2];
    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4, wave = wave_in_block();
    // all token tiles of a head on one die (they are dealt in turn)
    const int h = blockIdx.x, t0 = blockIdx.y * 64;
    const uint16_t* x = a.x + h * a.x_stride_h;
    const unsigned lds0 = lds_address(lds);
    auto issue = [&](int k0) {
#pragma unroll
        for (int i = 0; i < KC * 128 / 4096; ++i) {
            const int at = (i * 4 + wave) * 64 + lane, r = at / kChunks, k = k0 + ((at % kChunks) ^ (r & 15)) * 8;
            const int t = t0 + r;
            const uint16_t* p = x + (long)t * a.x_stride_t + k;
            load_to_lds16(t < a.T && k < a.K ? static_cast<const void*>(p) : kZeros, lds0 + (i * 4 + wave) * 1024);
        }
    };
    issue(0);
    // every wave takes every turn (the barriers need all four); one whose rows
    // lie past the end repeats the last row and stores nothing
    for (int block = 0; block < a.N; block += 4 * NT * 16) {
        const int n0 = block + wave * NT * 16;
        const uint16_t* w[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int n = n0 + i * 16 + col;
            w[i] = a.w + ((long)h * a.N + (n < a.N ? n : a.N - 1)) * a.K;
        }
        f32x4 acc[NT][TT] = {};
        for (int k0 = 0; k0 < a.K; k0 += KC) {
            bf16x8 wf[NT][kSteps];
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int i = 0; i < NT; ++i) wf[i][s] = row_chunk(w[i], k0 + s * 32 + quad * 8, a.K);
            if (k0 > 0 || (block > 0 && a.K > KC)) {  // more inner columns than a tile holds
                lds_barrier();
                issue(k0);
            }
            wait_vmem<0>();
            lds_barrier();
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                bf16x8 xf[TT];
#pragma unroll
                for (int j = 0; j < TT; ++j) {
                    const int r = j * 16 + col;
                    xf[j] = lds_chunk(lds0 + r * KC * 2 + ((s * 4 + quad) ^ (r & 15)) * 16);
                }
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < TT; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[i][s], xf[j], acc[i][j], 0, 0, 0);
            }
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
                if (n < a.N) *reinterpret_cast<u32x2*>(o + n) = v;
            }
        }
    }
}

template <int NT, int TT>
void launch_tiles(const HeadArgs& a, hipStream_t s) {
    const dim3 grid((a.N + 64 * NT - 1) / (64 * NT), (a.T + 16 * TT - 1) / (16 * TT), a.heads);
    hipLaunchKernelGGL((head_linear_kernel<NT, TT>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_head_linear(const HeadArgs& a, hipStream_t s) {
    if (a.T <= 16)
        launch_tiles<1, 1>(a, s);
    else if (a.K <= 128)
        hipLaunchKernelGGL(head_linear_tile_kernel<128>, dim3(a.heads, (a.T + 63) / 64), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL(head_linear_tile_kernel<512>, dim3(a.heads, (a.T + 63) / 64), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
