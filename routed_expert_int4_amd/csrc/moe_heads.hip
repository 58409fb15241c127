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
#pragma unroll 4
    for (int k0 = 0; k0 < a.K; k0 += 32) {
        const int k = k0 + quad * 8;
        bf16x8 wf[NT], xf[TT];
#pragma unroll
        for (int i = 0; i < NT; ++i) wf[i] = row_chunk(w[i], k, a.K);
#pragma unroll
        for (int i = 0; i < TT; ++i) xf[i] = row_chunk(x[i], k, a.K);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < TT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[i], xf[j], acc[i][j], 0, 0, 0);
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

template <int NT, int TT>
void launch_tiles(const HeadArgs& a, hipStream_t s) {
    const dim3 grid((a.N + 64 * NT - 1) / (64 * NT), (a.T + 16 * TT - 1) / (16 * TT), a.heads);
    hipLaunchKernelGGL((head_linear_kernel<NT, TT>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_head_linear(const HeadArgs& a, hipStream_t s) {
    if (a.T <= 16)
        launch_tiles<1, 1>(a, s);
    else if (a.T <= 64)
        launch_tiles<1, 2>(a, s);
    else
        launch_tiles<2, 4>(a, s);
    return hipGetLastError();
}

}  // namespace moe
