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
// then holds one weight row's results and needs one scale per group.
//
// Few tokens are bound by reading the weights, and a load by the lines that it
// touches, some two cycles each: 32 bytes of 32 rows cost four times what 128
// bytes of eight do.  Many are bound by no one thing: 64 columns of a wave's 64 x
// 96 results are 32 matrix instructions and 370 others, 192 of them the scaling
// of the groups' sums (for every result and group, whatever the tile).  Counted,
// the matrix cores are busy for 40 % of the time and the others take 59 % of the
// SIMDs' cycles; the two overlap in part, and the waves wait for a third of their
// time.  The scaling does not hold it: at group 128 there are 272 others, 43 % of
// the cycles, of which there are as many, and 4 to 8 % less time among other calls.
//
// Measured, 6144 x 8192, group 32 (25 MB of codes, 3 of scales): 1 token 9.6 us
// (3.0 TB/s, a quarter of it launch and first latency; 49152 rows 51 us, 4.4
// TB/s), 16 tokens 12.5, 32 17.6, 64 28, 128 45, 512 135, 2048 290 (0.71
// PFLOP/s; group 128 265, 0.78).
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

__device__ __forceinline__ void store_out(const Int4Args& a, int t, int n, float v) {
    const long at = (long)t * a.ldo + n;
    if (a.out_f32)
        static_cast<float*>(a.out)[at] = v;
    else
        static_cast<uint16_t*>(a.out)[at] = round_bf16(v);
}

// One or two tokens: a lane takes the 16 bytes, 32 columns, of a weight row
// that share a scale and multiplies them with two-element dot products: fewer
// instructions than operands of the matrix cores take for so few rows.  Eight
// lanes read 128 neighbouring bytes of a row.  The eight waves of a workgroup
// share the inner columns of 16 weight rows, 256 at a time in turn; all loads
// of a turn of 8192 columns are on their way before the activations, put in the
// weights' order, have come to LDS.  (1 x 6144 x 8192: 9.6 us; four lanes to a
// row 13.8, matrix instructions 22.9.)
constexpr int kTurnSegs = 4, kFewWaves = 8, kSeg = 256, kTurn = kTurnSegs * kFewWaves * kSeg;
template <int GROUP, int TOKENS>
__global__ void __launch_bounds__(kFewWaves * 64) int4_few_kernel(Int4Args a) {
    // (the 64 bytes that go with a lane's weights: their four chunks are turned
    // by the upper bit of the lane's place, so that eight lanes cover all banks)
    __shared__ __attribute__((aligned(16))) u32x4 xs[TOKENS][kTurn / 8];
    __shared__ float minus[TOKENS][kTurn / 32];  // -1.5 times the sum of 32 activations
    __shared__ float sums[kFewWaves][TOKENS][16];
    const int lane = threadIdx.x & 63, place = lane & 7, wave = wave_in_block(), n0 = blockIdx.x * 16;
    const uint8_t* w_row[2];
    const uint16_t* s_row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int n = n0 + h * 8 + (lane >> 3);
        w_row[h] = a.w + (long)(n < a.N ? n : a.N - 1) * a.ldw;
        s_row[h] = a.scale + (long)(n < a.N ? n : a.N - 1) * a.lds;
    }
    float acc[2][TOKENS] = {};
    for (int k_turn = 0; k_turn < a.K; k_turn += kTurn) {
        u32x4 w[kTurnSegs][2];
        uint16_t s[kTurnSegs][2];
#pragma unroll
        for (int i = 0; i < kTurnSegs; ++i) {
            const int k_seg = k_turn + (i * kFewWaves + wave) * kSeg, k = k_seg + place * 32;
            if (k_seg >= a.K) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[i][h] = load_stream16(w_row[h] + (k < a.K ? k / 2 : 0));
                s[i][h] = *as_global<uint16_t>(s_row[h] + (k < a.K ? k / GROUP : 0));
            }
        }
        if (k_turn > 0) __syncthreads();
        // (zero past the last column, which leaves any weight without effect)
        for (int i = threadIdx.x; i < TOKENS * (kTurn / 8); i += kFewWaves * 64) {
            const int t = i / (kTurn / 8), c = i % (kTurn / 8), k = k_turn + c * 8;
            if (k_turn + c / (kSeg / 8) * kSeg >= a.K) continue;  // (whole segments only)
            u32x4 x = {0, 0, 0, 0};
            if (k < a.K && t < a.M) x = *as_global<u32x4>(a.x + (long)t * a.ldx + k);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += bf16_lo(x[j]) + bf16_hi(x[j]);
            sum += dpp_f<kDppXor1>(sum);
            sum += dpp_f<kDppXor2>(sum);
            xs[t][c ^ ((c >> 4) & 1)] = __builtin_bit_cast(u32x4, in_order(x));
            if ((c & 3) == 0) minus[t][c / 4] = -1.5f * sum;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTurnSegs; ++i) {
            const int seg = i * kFewWaves + wave;
            if (k_turn + seg * kSeg >= a.K) break;
            float d[2][TOKENS];
#pragma unroll
            for (int t = 0; t < TOKENS; ++t) d[0][t] = d[1][t] = minus[t][seg * 8 + place];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                u32x4 q[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) q[h] = __builtin_bit_cast(u32x4, widen(w[i][h][c]));
#pragma unroll
                for (int t = 0; t < TOKENS; ++t) {
                    const u32x4 x = xs[t][(seg * 32 + place * 4 + c) ^ (place >> 2)];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const unsigned xj = x[j];  // (a bit cast of an element would take the first one's bits)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const unsigned qj = q[h][j];
                            d[h][t] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(i16x2, qj), __builtin_bit_cast(i16x2, xj), d[h][t], false);
                        }
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < TOKENS; ++t) acc[h][t] = fmaf(d[h][t], half_bits_to_float(s[i][h]), acc[h][t]);
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            float sum = acc[h][t];
            sum += dpp_f<kDppXor1>(sum);
            sum += dpp_f<kDppXor2>(sum);
            sum += dpp_f<kDppHalfMirror>(sum);
            if (place == 0) sums[wave][t][h * 8 + (lane >> 3)] = sum;
        }
    __syncthreads();
    if (threadIdx.x < TOKENS * 16) {
        const int t = threadIdx.x / 16, n = n0 + (threadIdx.x & 15);
        if (n >= a.N || t >= a.M) return;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) sum += sums[w][t][threadIdx.x & 15];
        store_out(a, t, n, sum * kCodeUnit);
    }
}

// Up to 32 tokens: one or two matrix tiles of them, and the weights streamed
// from memory once.  A workgroup has NT x 16 weight rows; its eight waves share
// the inner columns, 256 (a chunk) at a time in turn, and join their sums in
// wave order.  What bounds a load is the number of lines that it touches, so
// all go to LDS asynchronously, eight lanes to 128 bytes of a weight row and as
// many or twice as many to a row of activations, and are read from there in
// operand order; a wave waits for nothing but its own loads.  Activations come
// 128 columns (a stage; 64 of two tiles) at a time.  The scales of a turn of
// 4096 or 8192 columns lie in LDS too.  (16 x 6144 x 8192: 12.5 us; everything
// straight into registers in operand order, 64 bytes of 16 rows to a load, 21.4
// and, with more of it on its way, 24 and 27.)
constexpr int kChunk = 256;
template <int GROUP, int NT, int TT, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, 2) int4_rows_kernel(Int4Args a) {
    constexpr int kTurnColumns = WAVES * kChunk * 4;
    constexpr int kStage = 128 / TT, kStages = kChunk / kStage, kSteps = kStage / 32;  // columns, stages per chunk, steps per stage
    constexpr int kGroups = GROUP < kStage ? kStage / GROUP : 1, kPer = kSteps / kGroups;  // scales per stage, steps per scale
    constexpr int kRows = NT * 16, kTurnGroups = kTurnColumns / GROUP, kScaleRow = kTurnGroups * 2 + 8;  // bytes; rows apart by two banks
    constexpr int kWeights = kRows * kChunk / 2, kActs = TT * 16 * kStage * 2, kWave = 2 * (kWeights + kActs);
    constexpr int kWeightLoads = kWeights / 1024, kActLoads = kActs / 1024;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[WAVES * kWave];
    __shared__ __attribute__((aligned(16))) uint8_t scales[kRows * kScaleRow];
    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4, wave = wave_in_block();
    const int n0 = blockIdx.x * kRows;
    const unsigned weights_at = lds_address(lds) + wave * kWave, acts_at = weights_at + 2 * kWeights;
    // Piece p (16 bytes) of row r lies at place p ^ (r / 2 % 8) of 128 bytes,
    // or p ^ (r % 16) of 256: a step's operand reads cover all banks.
    constexpr int kActPieces = kStage / 8;
    auto act_place = [](int piece, int r) { return (kActPieces == 16 ? piece ^ r : piece ^ (r / 2)) & (kActPieces - 1); };
    const uint8_t* w_from[kWeightLoads];
    int w_piece[kWeightLoads];
#pragma unroll
    for (int j = 0; j < kWeightLoads; ++j) {
        const int r = j * 8 + (lane >> 3), n = n0 + r;
        w_from[j] = a.w + (long)(n < a.N ? n : a.N - 1) * a.ldw;
        w_piece[j] = (lane & 7) ^ (r / 2 & 7);
    }
    const uint16_t* x_from[kActLoads];
    int x_piece[kActLoads];
#pragma unroll
    for (int j = 0; j < kActLoads; ++j) {
        const int r = j * (64 / kActPieces) + lane / kActPieces;
        x_from[j] = a.x + (long)(r < a.M ? r : a.M - 1) * a.ldx;
        x_piece[j] = act_place(lane % kActPieces, r);
    }
    f32x4 acc[NT][TT] = {};
    for (int k_turn = 0; k_turn < a.K; k_turn += kTurnColumns) {
        const int columns = a.K - k_turn < kTurnColumns ? a.K - k_turn : kTurnColumns;
        const int chunks = (columns + WAVES * kChunk - 1) / (WAVES * kChunk), stages = chunks * kStages;
        auto first_column = [&](int chunk) { return k_turn + (chunk * WAVES + wave) * kChunk; };
        // (columns past the last one: weights read others, activations zeros)
        auto load_weights = [&](int chunk) {
            const int k0 = first_column(chunk);
#pragma unroll
            for (int j = 0; j < kWeightLoads; ++j) {
                const int k = k0 + w_piece[j] * 32;
                load_to_lds16(w_from[j] + (k < a.K ? k / 2 : 0), weights_at + (chunk & 1) * kWeights + j * 1024);
            }
        };
        auto load_acts = [&](int stage) {
            const int k0 = first_column(stage / kStages) + stage % kStages * kStage;
#pragma unroll
            for (int j = 0; j < kActLoads; ++j) {
                const int k = k0 + x_piece[j] * 8;
                load_to_lds16(k < a.K ? static_cast<const void*>(x_from[j] + k) : kZeros, acts_at + (stage & 1) * kActs + j * 1024);
            }
        };
        // a part of a row's scales per thread, zero past the last one
        constexpr int kThreads = WAVES * 64 / kRows, kEach = kTurnGroups / kThreads;  // threads per row, scales of a thread
        typedef uint16_t part __attribute__((ext_vector_type(kEach < 8 ? kEach : 8), aligned(2)));  // (a row of scales starts on two bytes)
        constexpr int kPart = kEach < 8 ? kEach : 8, kParts = kEach / kPart;
        part s_part[kParts];
        const int s_row = threadIdx.x / kThreads, s_first = threadIdx.x % kThreads * kEach, groups = columns / GROUP;
        {
            const uint16_t* p = a.scale + (long)(n0 + s_row < a.N ? n0 + s_row : a.N - 1) * a.lds + k_turn / GROUP;
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                const int g = s_first + i * kPart;
                if (g + kPart <= groups) {
                    s_part[i] = *as_global<part>(p + g);
                } else {
#pragma unroll
                    for (int j = 0; j < kPart; ++j) s_part[i][j] = g + j < groups ? *as_global<uint16_t>(p + g + j) : (uint16_t)0;
                }
            }
        }
        if (k_turn > 0) __syncthreads();  // the last turn's scales have served
        load_weights(0);
        load_acts(0);
        if (chunks > 1) load_weights(1);
        load_acts(1);
#pragma unroll
        for (int i = 0; i < kParts; ++i)
#pragma unroll
            for (int j = 0; j < kPart; ++j)
                *reinterpret_cast<uint16_t*>(scales + s_row * kScaleRow + (s_first + i * kPart + j) * 2) = s_part[i][j];
        lds_barrier();
        for (int stage = 0; stage < stages; ++stage) {
            const int chunk = stage / kStages, in_chunk = stage % kStages;
            // the loads behind this stage's: the next stage's activations, if
            // any, and before them the next chunk's weights, if any
            if (stage + 1 == stages)
                wait_vmem<0>();
            else if (in_chunk == 0 && chunk + 1 < chunks)
                wait_vmem<kWeightLoads + kActLoads>();
            else
                wait_vmem<kActLoads>();
            const unsigned w_at = weights_at + (chunk & 1) * kWeights, x_at = acts_at + (stage & 1) * kActs;
            bf16x8 x[TT][kSteps];
            unsigned w[NT][kSteps];
            typedef uint16_t stage_scales __attribute__((ext_vector_type(kGroups)));
            stage_scales s[NT];
#pragma unroll
            for (int j = 0; j < TT; ++j)
#pragma unroll
                for (int e = 0; e < kSteps; ++e) {
                    const int r = j * 16 + col;
                    x[j][e] = lds_chunk(x_at + r * (kStage * 2) + act_place(e * 4 + quad, r) * 16);
                }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int r = i * 16 + col;
#pragma unroll
                for (int e = 0; e < kSteps; ++e)
                    w[i][e] = lds_dword(w_at + r * (kChunk / 2) + (((in_chunk * kSteps + e) ^ (r / 2)) & 7) * 16 + quad * 4);
                s[i] = *reinterpret_cast<const stage_scales*>(scales + r * kScaleRow +
                                                              (first_column(chunk) - k_turn + in_chunk * kStage) / GROUP * 2);
            }
            f32x4 start[TT][kGroups];
#pragma unroll
            for (int j = 0; j < TT; ++j)
#pragma unroll
                for (int e = 0; e < kSteps; ++e) {
                    x[j][e] = in_order(__builtin_bit_cast(u32x4, x[j][e]));
                    const f32x4 zero = {};
                    start[j][e / kPer] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        x[j][e], minus_one_and_half(), e % kPer ? start[j][e / kPer] : zero, 0, 0, 0);
                }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    f32x4 d[TT];
#pragma unroll
                    for (int e = g * kPer; e < (g + 1) * kPer; ++e) {
                        const bf16x8 q = widen(w[i][e]);
#pragma unroll
                        for (int j = 0; j < TT; ++j)
                            d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[j][e], q, e % kPer ? d[j] : start[j][g], 0, 0, 0);
                    }
                    const uint16_t bits = s[i][g];
                    const float f = half_bits_to_float(bits);
#pragma unroll
                    for (int j = 0; j < TT; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[j][e], f, acc[i][j][e]);
                }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this stage's reads, before what is loaded over it
            if (in_chunk + 1 == kStages && chunk + 2 < chunks) load_weights(chunk + 2);
            if (stage + 2 < stages) load_acts(stage + 2);
        }
    }
    __syncthreads();
    float* const sums = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sums[((wave * NT * TT + i * TT + j) * 4 + e) * 64 + lane] = acc[i][j][e];
    __syncthreads();
    for (int at = threadIdx.x; at < NT * TT * 4 * 64; at += WAVES * 64) {
        const int v = at >> 6, l = at & 63;
        const int n = n0 + v / (TT * 4) * 16 + (l & 15), t = v / 4 % TT * 16 + (l >> 4) * 4 + (v & 3);
        if (n >= a.N || t >= a.M) continue;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) sum += sums[(w * NT * TT * 4 + v) * 64 + l];
        store_out(a, t, n, sum * kCodeUnit);
    }
}

// More tokens: tiles on the matrix cores.  WT x WN waves lie along tokens and
// weight rows, TT x NT matrix tiles of 32 x 32 each; WK waves share the inner
// columns of a stage, 64 each, and join their sums at the end.  Everything goes
// to LDS asynchronously, RING - 1 stages ahead, as it lies in memory (what
// bounds a load is the number of lines that it touches), the scales of a turn
// of 8192 columns at its beginning.  (64 x 6144 x 8192: 28 us; weights and
// scales straight into registers 34.)
// A weight row's 16 bytes of a lane half hold four dwords of 8 columns; swapped
// with the other half's they are the four steps of 16, in dwords 0 2 1 3.
__device__ __forceinline__ constexpr int at_step(int e) { return e == 1 ? 2 : e == 2 ? 1 : e; }

template <int GROUP, int TT, int NT, int WT, int WN, int WK, int RING>
__global__ void __launch_bounds__(WT * WN * WK * 64, 2) int4_tile_kernel(Int4Args a) {
    constexpr int kWaves = WT * WN * WK, kTokens = WT * TT * 32, kRows = WN * NT * 32, kColumns = 64 * WK, kTurnColumns = 8192;
    constexpr int kActRow = kColumns * 2, kWeightRow = kColumns / 2, kActs = kTokens * kActRow, kWeights = kRows * kWeightRow;
    constexpr int kActLoads = kActs / 1024 / kWaves, kWeightLoads = kWeights / 1024 / kWaves, kLoads = kActLoads + kWeightLoads;
    constexpr int kScales = GROUP == 32 ? 2 : 1, kSteps = 4 / kScales;  // scales of a wave's 64 columns, steps of 16 for each
    constexpr int kSumBytes = WK > 1 ? (WK - 1) * WT * WN * TT * NT * 16 * 64 * 4 : 0, kRing = RING * (kActs + kWeights);
    constexpr int kTurnGroups = kTurnColumns / GROUP, kScaleRow = kTurnGroups * 2 + 8;  // bytes; rows apart by two banks
    static_assert(kActLoads * kWaves * 1024 == kActs && kWeightLoads * kWaves * 1024 == kWeights && kSumBytes <= kRing, "stage");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing];
    __shared__ __attribute__((aligned(16))) uint8_t scales[kRows * kScaleRow];
    const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31, wave = wave_in_block();
    const int wk = wave % WK, wn = wave / WK % WN, wt = wave / (WK * WN);
    // workgroups of one die (they are dealt in turn) take neighbouring tiles
    // of the same weight rows
    const int n_tiles = (a.N + kRows - 1) / kRows, t_tiles = (a.M + kTokens - 1) / kTokens;
    const int per_die = (n_tiles * t_tiles + 7) / 8, tile = (blockIdx.x & 7) * per_die + (blockIdx.x >> 3);
    if (tile >= n_tiles * t_tiles) return;
    const int t0 = tile % t_tiles * kTokens, n_tile = tile / t_tiles * kRows, n0 = n_tile + wn * NT * 32;
    const unsigned lds0 = lds_address(lds);
    // Piece c (16 bytes) of row r lies at place c mixed with the row so that
    // the rows of an operand read cover all banks.
    auto act_place = [](int r, int c) { return c ^ (r & 15); };
    auto weight_place = [](int r, int c) { return c ^ (r / (8 / WK) & (2 * WK - 1)); };
    const uint16_t* x_from[kActLoads];
    int x_column[kActLoads];
#pragma unroll
    for (int i = 0; i < kActLoads; ++i) {
        const int at = ((i * kWaves + wave) * 64 + lane) * 16, r = at / kActRow, t = t0 + r;
        x_from[i] = a.x + (long)(t < a.M ? t : a.M - 1) * a.ldx;
        x_column[i] = act_place(r, at % kActRow / 16) * 8;
    }
    const uint8_t* w_from[kWeightLoads];
    int w_column[kWeightLoads];
#pragma unroll
    for (int i = 0; i < kWeightLoads; ++i) {
        const int at = ((i * kWaves + wave) * 64 + lane) * 16, r = at / kWeightRow, n = n_tile + r;
        w_from[i] = a.w + (long)(n < a.N ? n : a.N - 1) * a.ldw;
        w_column[i] = weight_place(r, at % kWeightRow / 16) * 32;
    }
    f32x16 acc[NT][TT] = {};
    for (int k_turn = 0; k_turn < a.K; k_turn += kTurnColumns) {
        const int columns = a.K - k_turn < kTurnColumns ? a.K - k_turn : kTurnColumns, stages = (columns + kColumns - 1) / kColumns;
        // (columns past the last one: weights read others, activations zeros)
        auto issue = [&](int stage, int buf) {
            const int k0 = k_turn + stage * kColumns;
            const unsigned dst = lds0 + buf * (kActs + kWeights) + wave * 1024;
#pragma unroll
            for (int i = 0; i < kActLoads; ++i) {
                const int k = k0 + x_column[i];
                load_to_lds16(k < a.K ? static_cast<const void*>(x_from[i] + k) : kZeros, dst + i * kWaves * 1024);
            }
#pragma unroll
            for (int i = 0; i < kWeightLoads; ++i) {
                const int k = k0 + w_column[i];
                load_to_lds16(w_from[i] + (k < a.K ? k / 2 : 0), dst + kActs + i * kWaves * 1024);
            }
        };
        // a part of a row's scales per thread, zero past the last one
        constexpr int kThreads = kWaves * 64 / kRows, kEach = kTurnGroups / kThreads, kPart = kEach < 8 ? kEach : 8, kParts = kEach / kPart;
        typedef uint16_t part __attribute__((ext_vector_type(kPart), aligned(2)));  // (a row of scales starts on two bytes)
        part s_part[kParts];
        const int s_row = threadIdx.x / kThreads, s_first = threadIdx.x % kThreads * kEach, groups = columns / GROUP;
        const uint16_t* p = a.scale + (long)(n_tile + s_row < a.N ? n_tile + s_row : a.N - 1) * a.lds + k_turn / GROUP;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int g = s_first + i * kPart;
            if (g + kPart <= groups) {
                s_part[i] = *as_global<part>(p + g);
            } else {
#pragma unroll
                for (int j = 0; j < kPart; ++j) s_part[i][j] = g + j < groups ? *as_global<uint16_t>(p + g + j) : (uint16_t)0;
            }
        }
        if (k_turn > 0) __syncthreads();  // the last turn's scales and stages have served
#pragma unroll
        for (int i = 0; i < RING - 1; ++i)
            if (i < stages) issue(i, i);
#pragma unroll
        for (int i = 0; i < kParts; ++i)
#pragma unroll
            for (int j = 0; j < kPart; ++j)
                *reinterpret_cast<uint16_t*>(scales + s_row * kScaleRow + (s_first + i * kPart + j) * 2) = s_part[i][j];
        int buf = 0;
        for (int stage = 0; stage < stages; ++stage) {
            if (stage + RING - 2 < stages)
                wait_vmem<(RING - 2) * kLoads>();
            else
                wait_vmem<0>();
            lds_barrier();  // the stage is in LDS, and every wave is done with the one before
            if (stage + RING - 1 < stages) issue(stage + RING - 1, buf == 0 ? RING - 1 : buf - 1);
            const unsigned from = lds0 + buf * (kActs + kWeights);
            buf = buf == RING - 1 ? 0 : buf + 1;
            unsigned w[NT][4];
            float s[NT][kScales];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int r = (wn * NT + i) * 32 + col;
                const u32x4 v = __builtin_bit_cast(u32x4, lds_chunk(from + kActs + r * kWeightRow + weight_place(r, wk * 2 + half) * 16));
#pragma unroll
                for (int d = 0; d < 4; ++d) w[i][d] = v[d];
                swap32(w[i][0], w[i][1]);
                swap32(w[i][2], w[i][3]);
#pragma unroll
                for (int g = 0; g < kScales; ++g) {
                    const uint16_t bits = *reinterpret_cast<const uint16_t*>(scales + r * kScaleRow + (stage * kColumns + wk * 64 + g * 32) / GROUP * 2);
                    s[i][g] = half_bits_to_float(bits);
                }
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
                        x[j][e] = in_order(__builtin_bit_cast(u32x4, lds_chunk(from + r * kActRow + act_place(r, c) * 16)));
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

// Many tokens: one wave to the whole inner dimension of its TT x NT matrix
// tiles, WT x WN waves along tokens and weight rows.  Of a stage of 64 columns
// the activations come to LDS asynchronously, a stage ahead, and are put in
// order as they are read; weights come two stages at a time, scales four.  Two
// waves of two workgroups fit a SIMD, and what counts is what instructions cost.
// (2048 x 6144 x 8192: 128 x 192 tiles 290 us, 128 x 128 350; weights and scales
// straight into registers 325; one wave per SIMD 732.)
template <int GROUP, int TT, int NT, int WT, int WN, int PER_SIMD>
__global__ void __launch_bounds__(WT * WN * 64, PER_SIMD) int4_many_kernel(Int4Args a) {
    constexpr int kWaves = WT * WN, kTokens = WT * TT * 32, kChunks = 8;  // 16-byte chunks of a row of a stage
    constexpr int kStageBytes = kTokens * kChunks * 16, kLoads = kStageBytes / 1024 / kWaves;
    constexpr int kScales = GROUP == 32 ? 2 : 1, kSteps = 4 / kScales;  // scales of a wave's 64 columns, steps of 16 for each
    static_assert(kLoads * kWaves * 1024 == kStageBytes, "stage");
    // Weights come 128 columns (a chunk, two stages) at a time, scales 256.
    constexpr int kRows = WN * NT * 32, kChunkBytes = kRows * 64, kChunkLoads = kChunkBytes / 1024 / kWaves, kPart = 256 / GROUP;
    static_assert(kChunkLoads * kWaves * 1024 == kChunkBytes && kRows <= kWaves * 64, "chunk");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * (kStageBytes + kChunkBytes)];
    typedef uint16_t part __attribute__((ext_vector_type(kPart), aligned(2)));  // (a row of scales starts on two bytes)
    __shared__ __attribute__((aligned(16))) uint16_t scales[2][kRows][kPart];
    const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31, wave = wave_in_block();
    const int wn = wave % WN, wt = wave / WN;
    // workgroups of one die (they are dealt in turn) take neighbouring tiles
    // of the same weight rows
    const int n_tiles = (a.N + WN * NT * 32 - 1) / (WN * NT * 32), t_tiles = (a.M + kTokens - 1) / kTokens;
    const int per_die = (n_tiles * t_tiles + 7) / 8, tile = (blockIdx.x & 7) * per_die + (blockIdx.x >> 3);
    if (tile >= n_tiles * t_tiles) return;
    const int t0 = tile % t_tiles * kTokens, n_tile = tile / t_tiles * WN * NT * 32, n0 = n_tile + wn * NT * 32;
    const int stages = (a.K + 63) / 64;
    const unsigned lds0 = lds_address(lds);
    // Addresses are a base for the tile and the stage and an offset that a lane
    // keeps; rows past the last one repeat it.  Chunk c of row r of the
    // activations lies at place c ^ (r & 7), of the weights at c ^ (r / 4 & 3).
    // The weights' operand reads cover all banks; rows of activations that are
    // eight apart share theirs, and at group 32 scales of rows sixteen apart
    // (conflicts are counted for 11 % of a compute unit's cycles at group 32, 5 %
    // at 128).  (What bounds loads is the number of lines that they touch: weights
    // straight into operand order would be 32 lines to a load of 1 KB.)
    unsigned x_off[kLoads], w_off[kChunkLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int at = (i * kWaves + wave) * 64 + lane, r = at / kChunks, c = (at % kChunks) ^ (r & 7);
        const int last = a.M - 1 - t0;
        x_off[i] = (unsigned)(r < last ? r : last) * (unsigned)(a.ldx * 2) + c * 16;
    }
    const int last_row = a.N - 1 - n_tile;
    auto weight_place = [](int r, int c) { return c ^ (r >> 2 & 3); };
#pragma unroll
    for (int i = 0; i < kChunkLoads; ++i) {
        const int r = (i * kWaves + wave) * 16 + (lane >> 2);
        w_off[i] = (unsigned)(r < last_row ? r : last_row) * (unsigned)a.ldw + weight_place(r, lane & 3) * 16;
    }
    const uint8_t* const x_base = reinterpret_cast<const uint8_t*>(a.x + (long)t0 * a.ldx);
    const uint8_t* const w_base = a.w + (long)n_tile * a.ldw;
    const int s_row = threadIdx.x < last_row ? threadIdx.x : last_row;
    const uint16_t* const s_base = a.scale + (long)(n_tile + s_row) * a.lds;
    const int groups = a.K / GROUP;
    part s_next;
    auto issue_acts = [&](int stage, int buf) {
        const bool whole = stage * 64 + 64 <= a.K;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const unsigned dst = lds0 + buf * kStageBytes + (i * kWaves + wave) * 1024;
            if (whole) {
                load_to_lds16(x_base + (long)stage * 128, x_off[i], dst);
            } else {  // columns past the last one count as zero
                const int at = (i * kWaves + wave) * 64 + lane, c = (at % kChunks) ^ ((at / kChunks) & 7);
                const uint8_t* p = x_base + (long)stage * 128 + x_off[i];
                load_to_lds16(stage * 64 + c * 8 < a.K ? p : kZeros, dst);
            }
        }
    };
    auto issue_weights = [&](int chunk) {
        const bool whole = chunk * 128 + 128 <= a.K;
#pragma unroll
        for (int i = 0; i < kChunkLoads; ++i) {
            const unsigned dst = lds0 + 2 * kStageBytes + (chunk & 1) * kChunkBytes + (i * kWaves + wave) * 1024;
            if (whole) {
                load_to_lds16(w_base + (long)chunk * 64, w_off[i], dst);
            } else {  // (the product with zero)
                const int c = weight_place((i * kWaves + wave) * 16 + (lane >> 2), lane & 3);
                load_to_lds16(w_base + w_off[i] + (chunk * 128 + c * 32 < a.K ? (long)chunk * 64 : -(long)c * 16), dst);
            }
        }
    };
    auto load_scales = [&](int turn) {  // of 256 columns, a row per thread; zero past the last one
        const int first = turn * kPart;
        if (first + kPart <= groups) {
            s_next = *as_global<part>(s_base + first);
        } else {
#pragma unroll
            for (int i = 0; i < kPart; ++i) s_next[i] = first + i < groups ? *as_global<uint16_t>(s_base + first + i) : (uint16_t)0;
        }
    };
    f32x16 acc[NT][TT] = {};
    load_scales(0);
    issue_acts(0, 0);
    issue_weights(0);
    for (int stage = 0; stage < stages; ++stage) {
        const int buf = stage & 1;
        wait_vmem<0>();
        if (stage % 4 == 0 && (int)threadIdx.x < kRows) {
#pragma unroll
            for (int i = 0; i < kPart; ++i) scales[stage >> 2 & 1][threadIdx.x][i] = s_next[i];
        }
        lds_barrier();  // the stage is in LDS, and every wave is done with the other buffer
        if (stage + 1 < stages) {
            if (stage % 4 == 3) load_scales((stage + 1) / 4);
            issue_acts(stage + 1, buf ^ 1);
            if (stage & 1) issue_weights((stage + 1) / 2);
        }
        unsigned w[NT][4];
        float s[NT][kScales];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int r = (wn * NT + i) * 32 + col;
            const u32x4 v = __builtin_bit_cast(u32x4, lds_chunk(lds0 + 2 * kStageBytes + (stage >> 1 & 1) * kChunkBytes + r * 64 +
                                                                weight_place(r, (stage & 1) * 2 + half) * 16));
#pragma unroll
            for (int d = 0; d < 4; ++d) w[i][d] = v[d];
            // lane halves hold 32 columns each: to halves of 8 columns of the
            // same 16, which leaves the four steps in dwords 0 2 1 3
            swap32(w[i][0], w[i][1]);
            swap32(w[i][2], w[i][3]);
#pragma unroll
            for (int g = 0; g < kScales; ++g) {
                const uint16_t bits = scales[stage >> 2 & 1][r][(stage % 4 * 64 + g * 32) / GROUP];
                s[i][g] = half_bits_to_float(bits);
                asm("" : "+v"(s[i][g]));  // (or every product would convert it again)
            }
        }
#pragma unroll
        for (int g = 0; g < kScales; ++g) {
            f32x16 start[TT];
            bf16x8 x[TT][kSteps];
#pragma unroll
            for (int j = 0; j < TT; ++j)
#pragma unroll
                for (int e = 0; e < kSteps; ++e) {
                    const int r = (wt * TT + j) * 32 + col, c = (g * kSteps + e) * 2 + half;
                    x[j][e] = in_order(__builtin_bit_cast(
                        u32x4, lds_chunk(lds0 + buf * kStageBytes + (r * kChunks + (c ^ (r & 7))) * 16)));
                    const f32x16 zero = {};
                    start[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[j][e], minus_one_and_half(), e ? start[j] : zero, 0, 0, 0);
                }
            // a tile's sums are scaled while the next one's are computed: the
            // barriers keep the compiler from waiting for each in turn
            f32x16 d[2];
            auto scale = [&](int p) {
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[p / TT][p % TT][e] = fmaf(d[p & 1][e], s[p / TT][g], acc[p / TT][p % TT][e]);
            };
            bf16x8 q[kSteps];
#pragma unroll
            for (int p = 0; p < NT * TT; ++p) {
                if (p % TT == 0) {
#pragma unroll
                    for (int e = 0; e < kSteps; ++e) q[e] = widen(w[p / TT][at_step(g * kSteps + e)]);
                }
                d[p & 1] = start[p % TT];
#pragma unroll
                for (int e = 0; e < kSteps; ++e)
                    d[p & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[p % TT][e], q[e], d[p & 1], 0, 0, 0);
                if (p > 0) scale(p - 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            scale(NT * TT - 1);
        }
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

template <int GROUP, int TOKENS>
void launch_few(const Int4Args& a, hipStream_t s) {
    hipLaunchKernelGGL((int4_few_kernel<GROUP, TOKENS>), dim3((a.N + 15) / 16), dim3(kFewWaves * 64), 0, s, a);
}
template <int GROUP, int NT, int TT, int WAVES>
void launch_rows(const Int4Args& a, hipStream_t s) {
    hipLaunchKernelGGL((int4_rows_kernel<GROUP, NT, TT, WAVES>), dim3((a.N + 16 * NT - 1) / (16 * NT)), dim3(WAVES * 64), 0, s, a);
}
// A compute unit holds one workgroup of eight waves, or three of four with 16
// weight rows: the shortest form that takes one round over the chip, and where
// there are more, 32 rows to four waves (16 tokens; us; 8 and 4 waves with 16
// rows, 8 and 4 with 32):
//   2048 x 6144    7.2   9.3   9.1  11.7      12288 x 2048  11.7   7.9  10.8   8.9
//   6144 x 8192   17.7  15.8  12.6  16.2      49152 x 8192   108    85    80    72
template <int GROUP, int TT>
void launch_rows_of(const Int4Args& a, hipStream_t s) {
    const int rows = (a.N + 15) / 16;
    if (rows <= 256 && a.K > 2048) return launch_rows<GROUP, 1, TT, 8>(a, s);
    if (rows <= 512 && a.K > 2048) return launch_rows<GROUP, 2, TT, 8>(a, s);
    if (rows <= 768) return launch_rows<GROUP, 1, TT, 4>(a, s);
    launch_rows<GROUP, 2, TT, 4>(a, s);
}
template <int GROUP, int TT, int NT, int WT, int WN, int WK, int RING>
void launch_tiles(const Int4Args& a, hipStream_t s) {
    const long tiles = (long)((a.N + WN * NT * 32 - 1) / (WN * NT * 32)) * ((a.M + WT * TT * 32 - 1) / (WT * TT * 32));
    hipLaunchKernelGGL((int4_tile_kernel<GROUP, TT, NT, WT, WN, WK, RING>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                       dim3(WT * WN * WK * 64), 0, s, a);
}
template <int GROUP, int TT, int NT, int WT, int WN, int PER_SIMD>
void launch_many(const Int4Args& a, hipStream_t s) {
    const long tiles = (long)((a.N + WN * NT * 32 - 1) / (WN * NT * 32)) * ((a.M + WT * TT * 32 - 1) / (WT * TT * 32));
    hipLaunchKernelGGL((int4_many_kernel<GROUP, TT, NT, WT, WN, PER_SIMD>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                       dim3(WT * WN * 64), 0, s, a);
}

// Shapes of tiles and what a stage of inner columns takes them, in
// nanoseconds: alone on a compute unit, and with as many as fit (measured; the
// large ones are bound by instructions, the small ones by one step after the
// other), with kBegin for a tile's beginning and end.
struct Shape {
    int tokens, rows, columns, alone, together, fit;
};
constexpr Shape kShapes[] = {{32, 32, 512, 900, 900, 1},    {32, 64, 256, 770, 770, 1},    {64, 64, 256, 1250, 1250, 1},
                             {64, 128, 128, 1050, 1050, 1}, {128, 128, 64, 1200, 1750, 2}, {128, 192, 64, 1560, 2330, 2}};
constexpr double kBegin = 3000.0;
// The shape that takes least time over the rounds it needs on the chip (us at
// K = 8192; 64 x 6144: 35, 29, 44, 72 in the first four; 512 x 6144: 198, 155,
// 131, 144, 159, 200; 1024 x 6144: 442, 313, 260, 232, 207, 203).
int best_shape(const Int4Args& a) {
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < (int)(sizeof(kShapes) / sizeof(kShapes[0])); ++i) {
        const Shape& s = kShapes[i];
        auto up = [](long n, long d) { return (n + d - 1) / d; };
        const long per_cu = up(up(a.M, s.tokens) * up(a.N, s.rows), 256), full = per_cu / s.fit, rest = per_cu % s.fit;
        const double stages = (double)up(a.K, s.columns);
        const double time = (double)full * (stages * s.together + kBegin) + (rest ? stages * s.alone + kBegin : 0.0);
        if (i == 0 || time < least) least = time, best = i;
    }
    return best;
}

// Dot products or a matrix tile, us on one card: one token 2048 x 6144 7.0 and
// 7.1, 6144 x 8192 10.2 and 12.3 (group 128 9.7 and 11.3), 12288 x 2048 7.1 and 7.4,
// 49152 x 8192 49.5 and 61.1; two tokens 6.5 and 7.0, 12.4 and 12.3 (11.8 and 11.3),
// 7.4 and 7.3, 61.0 and 61.3.
template <int GROUP>
void launch_group(const Int4Args& a, hipStream_t s) {
    if (a.M == 1) return launch_few<GROUP, 1>(a, s);
    if (a.M == 2) return launch_few<GROUP, 2>(a, s);
    if (a.M <= 16) return launch_rows_of<GROUP, 1>(a, s);
    if (a.M <= 32) return launch_rows_of<GROUP, 2>(a, s);
    switch (best_shape(a)) {
        case 0: return launch_tiles<GROUP, 1, 1, 1, 1, 8, 3>(a, s);
        case 1: return launch_tiles<GROUP, 1, 1, 1, 2, 4, 4>(a, s);
        case 2: return launch_tiles<GROUP, 2, 1, 1, 2, 4, 3>(a, s);
        case 3: return launch_tiles<GROUP, 2, 1, 1, 4, 2, 3>(a, s);
        case 4: return launch_many<GROUP, 2, 2, 2, 2, 2>(a, s);
        default:
            launch_many<GROUP, 2, 3, 2, 2, 2>(a, s);
    }
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
