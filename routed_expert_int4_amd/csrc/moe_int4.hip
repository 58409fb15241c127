// Product of bf16 activations with 4-bit weights:
//
//   out[m][n] = sum_g s[n][g] sum_{k in g} q[n][k] x[m][k]
//
// with q two's complement nibbles (even column low), one fp16 scale per GROUP
// columns, fp32 sums.  A nibble becomes bf16 by placing it below the leading
// one of a value between 1 and 2: bits 3..6 of the mantissa, its top bit
// flipped, give 1 + (q + 8) / 16 = 1.5 + q / 16, one shift and one three-input
// operation for two weights.  The 1.5 leaves through the matrix cores too: the
// sums of a group start from its activations times -1.5 (one instruction for
// all weight rows of a wave), so that what a scale multiplies is
// sum q x / 16, with no rounding but fp32's.
//
// Activations are the matrix instruction's rows, weights its columns: a lane
// then holds one weight row's results and needs one scale per group.  A
// weight row's 16 bytes per lane hold four blocks of 8 columns of one group of
// 32; the swaps between the lane rows of a wave turn them into operands whose
// lanes share a group.
#include "moe_block.h"
#include "moe_block_device.h"

namespace moe {
namespace {

constexpr unsigned kNibbles = 0x00780078u, kOneAndHalf = 0x3FC03FC0u;
constexpr float kCodeUnit = 16.0f;  // sums are of q / 16

// Eight weights of a dword as bf16 1.5 + q / 16, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 widen(unsigned w) {
    const u32x4 u = {(w << 3 & kNibbles) ^ kOneAndHalf, (w >> 1 & kNibbles) ^ kOneAndHalf, (w >> 5 & kNibbles) ^ kOneAndHalf,
                     (w >> 9 & kNibbles) ^ kOneAndHalf};
    return __builtin_bit_cast(bf16x8, u);
}
// Eight activations in that order.
__device__ __forceinline__ bf16x8 in_order(u32x4 x) {
    const u32x4 u = {__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                     __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
    return __builtin_bit_cast(bf16x8, u);
}
__device__ __forceinline__ bf16x8 minus_one_and_half() {
    const u32x4 u = {0xBFC0BFC0u, 0xBFC0BFC0u, 0xBFC0BFC0u, 0xBFC0BFC0u};
    return __builtin_bit_cast(bf16x8, u);
}

__device__ __forceinline__ void swap32(unsigned& a, unsigned& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0], b = r[1];
}
__device__ __forceinline__ void swap16(unsigned& a, unsigned& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0], b = r[1];
}

__device__ __forceinline__ void store_out(const Int4Args& a, int t, int n, float v) {
    const long at = (long)t * a.ldo + n;
    if (a.out_f32)
        static_cast<float*>(a.out)[at] = v;
    else
        static_cast<uint16_t*>(a.out)[at] = round_bf16(v);
}

// Few tokens: the weights stream from memory once, straight into operand
// order.  A workgroup has NT x 16 weight rows and TT x 16 tokens; its waves
// share the inner columns, 128 (a segment) at a time in turn, U segments
// loaded one batch ahead, and join their sums through LDS in wave order.
template <int GROUP, int NT, int TT, int WAVES, int U>
__global__ void __launch_bounds__(WAVES * 64) int4_rows_kernel(Int4Args a) {
    constexpr int kPer = GROUP > 32 ? GROUP / 32 : 1, kGroups = 4 / kPer;  // blocks of 32 per group, groups per segment
    __shared__ float sums[WAVES][NT * TT * 4][64];
    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4, wave = wave_in_block();
    const int n0 = blockIdx.x * NT * 16, t0 = blockIdx.y * TT * 16;
    const int segs = (a.K + 127) / 128;
    const uint8_t* w_row[NT];
    const uint16_t* s_row[NT];
    const uint16_t* x_row[TT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int n = n0 + i * 16 + col;
        w_row[i] = a.w + (long)(n < a.N ? n : a.N - 1) * a.ldw;
        s_row[i] = a.scale + (long)(n < a.N ? n : a.N - 1) * a.lds;
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int t = t0 + j * 16 + col;
        x_row[j] = a.x + (long)(t < a.M ? t : a.M - 1) * a.ldx;
    }
    f32x4 acc[NT][TT] = {};
    struct Batch {
        u32x4 w[U][NT], x[U][TT][4];
        uint16_t s[U][NT][kGroups];
    } b[2];
    auto load = [&](Batch& v, int batch) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int seg = (batch * U + u) * WAVES + wave;
            if (seg >= segs) return;
            const int k0 = seg * 128;
            const bool whole = k0 + 128 <= a.K;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int k = k0 + quad * 32;
                v.w[u][i] = load_stream16(w_row[i] + (k < a.K ? k / 2 : 0));
                if (whole) {
                    // (a row of scales starts on two bytes)
                    typedef uint16_t scales __attribute__((ext_vector_type(kGroups), aligned(2)));
                    const scales s = *as_global<scales>(s_row[i] + seg * kGroups);
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) v.s[u][i][g] = s[g];
                } else {
#pragma unroll
                    for (int g = 0; g < kGroups; ++g)
                        v.s[u][i][g] = k0 + g * GROUP < a.K ? *as_global<uint16_t>(s_row[i] + seg * kGroups + g) : 0;
                }
            }
#pragma unroll
            for (int j = 0; j < TT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int k = k0 + c * 32 + quad * 8;
                    v.x[u][j][c] = *as_global<u32x4>(x_row[j] + (k < a.K ? k : 0));
                    if (!whole && k >= a.K) v.x[u][j][c] = u32x4{0, 0, 0, 0};
                }
        }
    };
    auto multiply = [&](Batch& v, int batch) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if ((batch * U + u) * WAVES + wave >= segs) return;
            bf16x8 x[TT][4];
            f32x4 start[TT][kGroups];
#pragma unroll
            for (int j = 0; j < TT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    x[j][c] = in_order(v.x[u][j][c]);
                    const f32x4 zero = {};
                    start[j][c / kPer] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        x[j][c], minus_one_and_half(), c % kPer ? start[j][c / kPer] : zero, 0, 0, 0);
                }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                // from four blocks of 8 columns of a lane row's own 32 to the same block of each lane row
                unsigned w[4] = {v.w[u][i][0], v.w[u][i][1], v.w[u][i][2], v.w[u][i][3]};
                swap32(w[0], w[2]);
                swap32(w[1], w[3]);
                swap16(w[0], w[1]);
                swap16(w[2], w[3]);
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const float s = half_bits_to_float(v.s[u][i][g]);
                    f32x4 d[TT];
#pragma unroll
                    for (int c = g * kPer; c < (g + 1) * kPer; ++c) {
                        const bf16x8 q = widen(w[c]);
#pragma unroll
                        for (int j = 0; j < TT; ++j)
                            d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[j][c], q, c % kPer ? d[j] : start[j][g], 0, 0, 0);
                    }
#pragma unroll
                    for (int j = 0; j < TT; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[j][e], s, acc[i][j][e]);
                }
            }
        }
    };
    const int batches = (segs + U * WAVES - 1) / (U * WAVES);
    load(b[0], 0);
    for (int k = 0; k < batches; k += 2) {
        if (k + 1 < batches) load(b[1], k + 1);
        multiply(b[0], k);
        if (k + 1 >= batches) break;
        if (k + 2 < batches) load(b[0], k + 2);
        multiply(b[1], k + 1);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sums[wave][(i * TT + j) * 4 + e][lane] = acc[i][j][e];
    __syncthreads();
    for (int at = threadIdx.x; at < NT * TT * 4 * 64; at += WAVES * 64) {
        const int v = at >> 6, l = at & 63;
        const int n = n0 + (v / (TT * 4)) * 16 + (l & 15), t = t0 + (v / 4 % TT) * 16 + (l >> 4) * 4 + (v & 3);
        if (n >= a.N || t >= a.M) continue;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) sum += sums[w][v][l];
        store_out(a, t, n, sum * kCodeUnit);
    }
}

// Many tokens: the activations of a tile pass through LDS, 64 WK inner
// columns (a stage) loaded asynchronously one stage ahead; weights go from
// memory into the registers of the waves that own their rows, one stage ahead
// too.  WT x WN waves lie along tokens and weight rows, TT x NT matrix tiles of
// 32 x 32 each; WK waves share the inner columns of a stage and join their
// sums at the end.
__device__ __forceinline__ constexpr int at_step(int e) { return e == 1 ? 2 : e == 2 ? 1 : e; }

template <int GROUP, int TT, int NT, int WT, int WN, int WK>
__global__ void __launch_bounds__(WT * WN * WK * 64, 1) int4_tile_kernel(Int4Args a) {
    constexpr int kWaves = WT * WN * WK, kTokens = WT * TT * 32, kChunks = 8 * WK;  // 16-byte chunks of a row of a stage
    constexpr int kStageBytes = kTokens * kChunks * 16, kLoads = kStageBytes / 1024 / kWaves;
    constexpr int kScales = GROUP == 32 ? 2 : 1, kSteps = 4 / kScales;  // scales of a wave's 64 columns, steps of 16 for each
    constexpr int kSumBytes = WK > 1 ? (WK - 1) * WT * WN * TT * NT * 16 * 64 * 4 : 0;
    constexpr int kLds = 2 * kStageBytes > kSumBytes ? 2 * kStageBytes : kSumBytes;
    static_assert(kLoads * kWaves * 1024 == kStageBytes && kLds <= 160 * 1024, "stage");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
    const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31, wave = wave_in_block();
    const int wk = wave % WK, wn = wave / WK % WN, wt = wave / (WK * WN);
    // workgroups of one die (they are dealt in turn) take neighbouring tiles
    // of the same weight rows
    const int n_tiles = (a.N + WN * NT * 32 - 1) / (WN * NT * 32), t_tiles = (a.M + kTokens - 1) / kTokens;
    const int per_die = (n_tiles * t_tiles + 7) / 8, tile = (blockIdx.x & 7) * per_die + (blockIdx.x >> 3);
    if (tile >= n_tiles * t_tiles) return;
    const int t0 = tile % t_tiles * kTokens, n0 = (tile / t_tiles * WN + wn) * NT * 32;
    const int stages = (a.K + 64 * WK - 1) / (64 * WK);
    const unsigned lds0 = lds_address(lds);
    // chunk c of row r lies at place c ^ (r & 7): the rows of an operand read cover all banks
    auto issue = [&](int stage, int buf) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = (i * kWaves + wave) * 64 + lane, r = at / kChunks, c = (at % kChunks) ^ (r & 7);
            const int t = t0 + r, k = (stage * kChunks + c) * 8;
            const uint16_t* p = a.x + (long)t * a.ldx + k;
            load_to_lds16(t < a.M && k < a.K ? static_cast<const void*>(p) : kZeros,
                          lds0 + buf * kStageBytes + (i * kWaves + wave) * 1024);
        }
    };
    const uint8_t* w_row[NT];
    const uint16_t* s_row[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int n = n0 + i * 32 + col;
        w_row[i] = a.w + (long)(n < a.N ? n : a.N - 1) * a.ldw;
        s_row[i] = a.scale + (long)(n < a.N ? n : a.N - 1) * a.lds;
    }
    u32x4 w_next[NT];
    uint16_t s_next[NT][kScales];
    auto load_weights = [&](int stage) {
        const int k0 = (stage * WK + wk) * 64, k = k0 + half * 32;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            w_next[i] = *as_global<u32x4>(w_row[i] + (k < a.K ? k / 2 : 0));
#pragma unroll
            for (int g = 0; g < kScales; ++g) {
                const int kg = k0 + g * 32;
                s_next[i][g] = *as_global<uint16_t>(s_row[i] + (kg < a.K ? kg / GROUP : 0));
            }
        }
    };
    f32x16 acc[NT][TT] = {};
    issue(0, 0);
    load_weights(0);
    for (int stage = 0; stage < stages; ++stage) {
        const int buf = stage & 1;
        wait_vmem<0>();
        unsigned w[NT][4];
        float s[NT][kScales];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            asm volatile("" : "+v"(w_next[i]));
#pragma unroll
            for (int d = 0; d < 4; ++d) w[i][d] = w_next[i][d];
            // lane halves hold 32 columns each: to halves of 8 columns of the
            // same 16, which leaves the four steps in dwords 0 2 1 3
            swap32(w[i][0], w[i][1]);
            swap32(w[i][2], w[i][3]);
#pragma unroll
            for (int g = 0; g < kScales; ++g) s[i][g] = half_bits_to_float(s_next[i][g]);
        }
        lds_barrier();  // the stage is in LDS, and every wave is done with the other buffer
        if (stage + 1 < stages) {
            issue(stage + 1, buf ^ 1);
            load_weights(stage + 1);
        }
#pragma unroll
        for (int g = 0; g < kScales; ++g) {
            f32x16 start[TT];
            bf16x8 x[TT][kSteps];
#pragma unroll
            for (int j = 0; j < TT; ++j)
#pragma unroll
                for (int e = 0; e < kSteps; ++e) {
                    const int r = (wt * TT + j) * 32 + col, c = wk * 8 + (g * kSteps + e) * 2 + half;
                    x[j][e] = in_order(__builtin_bit_cast(
                        u32x4, lds_chunk(lds0 + buf * kStageBytes + (r * kChunks + (c ^ (r & 7))) * 16)));
                    const f32x16 zero = {};
                    start[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[j][e], minus_one_and_half(), e ? start[j] : zero, 0, 0, 0);
                }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                bf16x8 q[kSteps];
#pragma unroll
                for (int e = 0; e < kSteps; ++e) q[e] = widen(w[i][at_step(g * kSteps + e)]);
#pragma unroll
                for (int j = 0; j < TT; ++j) {
                    f32x16 d = start[j];
#pragma unroll
                    for (int e = 0; e < kSteps; ++e) d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[j][e], q[e], d, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][j][e] = fmaf(d[e], s[i][g], acc[i][j][e]);
                }
            }
        }
    }
    if constexpr (WK > 1) {
        __syncthreads();
        float* const slot = reinterpret_cast<float*>(lds) + ((wt * WN + wn) * (WK - 1)) * (NT * TT * 16 * 64);
        if (wk > 0) {
            float* const mine = slot + (wk - 1) * (NT * TT * 16 * 64) + lane;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < TT; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) mine[((i * TT + j) * 16 + e) * 64] = acc[i][j][e];
        }
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int o = 0; o < WK - 1; ++o)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < TT; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        acc[i][j][e] += slot[o * (NT * TT * 16 * 64) + ((i * TT + j) * 16 + e) * 64 + lane];
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int n = n0 + i * 32 + col;
        if (n >= a.N) continue;
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int t = t0 + (wt * TT + j) * 32 + 8 * (e / 4) + 4 * half + e % 4;
                if (t < a.M) store_out(a, t, n, acc[i][j][e] * kCodeUnit);
            }
    }
}

template <int GROUP, int NT, int TT, int WAVES, int U>
void launch_few(const Int4Args& a, hipStream_t s) {
    const dim3 grid((a.N + 16 * NT - 1) / (16 * NT), (a.M + 16 * TT - 1) / (16 * TT));
    hipLaunchKernelGGL((int4_rows_kernel<GROUP, NT, TT, WAVES, U>), grid, dim3(WAVES * 64), 0, s, a);
}
template <int GROUP, int TT, int NT, int WT, int WN, int WK>
void launch_tiles(const Int4Args& a, hipStream_t s) {
    const long tiles = (long)((a.N + WN * NT * 32 - 1) / (WN * NT * 32)) * ((a.M + WT * TT * 32 - 1) / (WT * TT * 32));
    hipLaunchKernelGGL((int4_tile_kernel<GROUP, TT, NT, WT, WN, WK>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                       dim3(WT * WN * WK * 64), 0, s, a);
}

template <int GROUP>
void launch_group(const Int4Args& a, hipStream_t s) {
    if (a.M <= 16)
        launch_few<GROUP, 1, 1, 8, 2>(a, s);
    else if (a.M <= 32)
        launch_few<GROUP, 1, 2, 8, 1>(a, s);
    else if ((long)a.M * a.N < 128l * 256 * 128)
        launch_tiles<GROUP, 2, 2, 1, 1, 4>(a, s);
    else
        launch_tiles<GROUP, 2, 4, 2, 2, 1>(a, s);
}

}  // namespace

hipError_t launch_int4_linear(const Int4Args& a, hipStream_t s) {
    if (a.group == 32)
        launch_group<32>(a, s);
    else if (a.group == 64)
        launch_group<64>(a, s);
    else
        launch_group<128>(a, s);
    return hipGetLastError();
}

}  // namespace moe
