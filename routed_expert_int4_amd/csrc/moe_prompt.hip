// Causal attention over keys and values expanded per head (the expanded form
// of latent attention): ragged sequences packed one after another, the
// position part of the keys shared by all heads.
//
// One pass over the keys with the running maximum and sum of the softmax.  A
// workgroup owns 128 queries of one head, 32 per wave; tiles of KT keys go
// through LDS, loaded asynchronously one tile ahead into the other of two
// buffers.  Bound by the matrix cores: per 64 keys a wave issues 40 matrix
// instructions of 32 x 32 x 16 (widths 192 and 128), 1280 cycles, and some
// 900 cycles of exponentials and statistics, which the second workgroup on
// the same CU fills in (half of LDS each).
//
// 64 heads of widths 192 and 128, causal: 8192 tokens 1.22 to 1.32 ms from one
// card and run to the next, 1.05 to 1.13 PFLOP/s (a large bf16 matrix product
// reaches 1.50); three sequences of 257 tokens 17 us, where launch and the
// longest run of tiles count.
// 4096 tokens, 32 heads: 108 us (64, 64), 166 us (128, 128), 387 us (192, 256:
// 512 registers, of which 10 spill; tiles of 64 keys spill more: 729).
//
// A weight of zero times a value that is not finite would still make NaN, so
// tiles that some query of the wave does not see whole are searched for such
// values first; where there are any, they count as zero in the products and
// the scores of their keys, where seen, turn NaN.
#include <type_traits>

#include "moe_block.h"
#include "moe_block_device.h"

namespace moe {
namespace {

// Key rows are cut into parts of 64 columns, each part of a tile an array of
// 128-byte rows in LDS.  The chunk c (16 bytes) of row r sits at place
// c ^ ((r / 2) & 7), so that the 16 rows of an operand read (same chunk)
// cover all banks; value rows are mixed so that the four rows by 64 bytes of
// a transposed read do.
__device__ __forceinline__ int key_place(int c, int r) { return c ^ ((r >> 1) & 7); }
template <int ROW_BYTES>
__device__ __forceinline__ int value_place(int c, int r) {
    return ROW_BYTES % 256 ? c ^ (((r >> 1) & 1) << 2) : c ^ ((r & 3) << 2);
}

template <int NOPE, int ROPE, int VD, int KT, int PER_CU>
__global__ void __launch_bounds__(256, PER_CU) prompt_attention_kernel(PromptArgs a) {
    static_assert(ROPE == 64 && NOPE % 64 == 0, "the position part is one part of 64 columns");
    constexpr int kSub = KT / 32, kParts = NOPE / 64 + 1, kPartBytes = KT * 128, kOut = VD / 32;
    constexpr int kTileBytes = kParts * kPartBytes + KT * VD * 2;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2][kTileBytes];
    const int lane = threadIdx.x & 63, wave = wave_in_block(), half = lane >> 5, col = lane & 31;
    const int h = blockIdx.x, b = blockIdx.z;
    // bounds come from device memory: kept inside the tensors whatever they say
    auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    auto inside = [&](int v, int n) {
        v = uniform(v);
        return v < 0 ? 0 : (v > n ? n : v);
    };
    const int q_first = inside(a.cu_q[b], a.Tq), q_count = inside(a.cu_q[b + 1], a.Tq) - q_first;
    const int k_first = inside(a.cu_k[b], a.Tk), k_count_all = inside(a.cu_k[b + 1], a.Tk) - k_first;
    const int k_count = k_count_all > 0 ? k_count_all : 0;
    // the last tiles see the most keys: they go first
    const int tile = gridDim.y - 1 - blockIdx.y, q0 = tile * 128;
    if (q0 >= q_count) return;
    const int past = k_count - q_count;  // keys before the first query's own
    const int my_q = q0 + wave * 32 + col;
    const bool row_ok = my_q < q_count;
    const long q_row = q_first + (row_ok ? my_q : q_count - 1);

    bf16x8 qf[kParts * 4];
    {
        const uint16_t* p = a.q + q_row * a.q_stride_t + h * a.q_stride_h + half * 8;
#pragma unroll
        for (int k = 0; k < kParts * 4; ++k) qf[k] = __builtin_bit_cast(bf16x8, *as_global<u32x4>(p + k * 16));
    }
    // visible keys of this lane's query, and of the workgroup's and wave's last one
    auto visible = [&](int q) {
        const int n = a.causal ? past + q + 1 : k_count;
        return n < 0 ? 0 : (n > k_count ? k_count : n);
    };
    const int last_q = q0 + 127 < q_count ? q0 + 127 : q_count - 1;
    const int wave_last = q0 + wave * 32 + 31 < q_count ? q0 + wave * 32 + 31 : q_count - 1;
    const int limit = row_ok ? visible(my_q) : 0;
    const int wave_limit = uniform(q0 + wave * 32 < q_count ? visible(wave_last) : 0);
    // tiles that all of the wave's rows see whole
    const int wave_full = uniform((q0 + wave * 32 < q_count ? visible(q0 + wave * 32) : 0) / KT);
    const int tiles = uniform((visible(last_q) + KT - 1) / KT);

    // Loads of one tile: an instruction covers whole rows, and the place of a
    // lane's chunk is the same in all of a kind.
    constexpr int kValueRows = 1024 / (VD * 2);
    const int kr = wave * 8 + lane / 8, vr = wave * kValueRows + lane / (VD / 8);
    const int k_chunk = key_place(lane % 8, kr), v_chunk = value_place<VD * 2>(lane % (VD / 8), vr);
    const uint16_t* k_base = a.k + (long)k_first * a.k_stride_t + h * a.k_stride_h;
    const uint16_t* r_base = a.k_rope + (long)k_first * a.kr_stride_t;
    const uint16_t* v_base = a.v + (long)k_first * a.v_stride_t + h * a.v_stride_h;
    const unsigned lds0 = lds_address(&lds[0][0]);
    auto issue_part = [&](const uint16_t* base, long stride, int key0, int row, int chunk, unsigned dst) {
        // row: this lane's row in the tile
        if (key0 + KT <= k_count) {
            load_to_lds16(base + (long)key0 * stride + 0, (unsigned)(row * stride * 2 + chunk * 16), dst);
        } else {
            const int key = key0 + row;
            const uint16_t* p = base + (long)key * stride + chunk * 8;
            load_to_lds16(key < k_count ? static_cast<const void*>(p) : kZeros, dst);
        }
    };
    auto issue = [&](int t) {
        const int key0 = t * KT;
        const unsigned dst = lds0 + (t & 1) * kTileBytes + wave * 1024;
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int i = 0; i < KT / 32; ++i)
                issue_part(p < kParts - 1 ? k_base + p * 64 : r_base, p < kParts - 1 ? a.k_stride_t : a.kr_stride_t, key0,
                           kr + i * 32, k_chunk, dst + p * kPartBytes + i * 4096);
#pragma unroll
        for (int i = 0; i < KT / (4 * kValueRows); ++i)
            issue_part(v_base, a.v_stride_t, key0, vr + i * 4 * kValueRows, v_chunk, dst + kParts * kPartBytes + i * 4096);
    };

    // This lane's places in a tile: keys (row reads of 16 bytes) and values
    // (transposed reads of four keys); an exclusive or with the low part of a
    // chunk and an immediate offset reach every operand.
    const unsigned key_at = lds0 + col * 128 + key_place(half, col) * 16;
    const int vrow = half * 4 + ((lane & 15) >> 2), vchunk = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
    const unsigned value_at =
        lds0 + kParts * kPartBytes + vrow * VD * 2 + value_place<VD * 2>(vchunk, vrow) * 16 + (lane & 1) * 8;
    const float c = a.scale * 1.44269504088896340736f;
    float m = kNoMax, l = 0.0f;
    f32x16 o[kOut] = {};
    // the queries have landed: the compiler must not wait for them inside the
    // loop, where the next tile is on its way
#pragma unroll
    for (int k = 0; k < kParts * 4; ++k) asm volatile("" : "+v"(qf[k]));
    auto next_tile = [&](int t) {
        wait_vmem<0>();
        lds_barrier();  // tile t is in LDS, and every wave is done with the other buffer
        if (t + 1 < tiles) issue(t + 1);
    };
    auto one_tile = [&](int t, auto masked) __attribute__((always_inline)) {
        const int key0 = t * KT;
        const unsigned buf = (t & 1) * kTileBytes;
        f32x16 s[kSub] = {};
        unsigned key_base[4];  // the rest of an address is an immediate offset
#pragma unroll
        for (int k = 0; k < 4; ++k) key_base[k] = (key_at + buf) ^ k * 32;
        // operands are read kAhead instructions before their use (the
        // scheduling barriers keep that order); tiles of 32 keys alternate
        constexpr int kAhead = 3;
        bf16x8 x[kAhead];
        auto key_chunk = [&](int i) {
            const int k = i / kSub, u = i % kSub;
            return lds_chunk(key_base[k % 4] + (k / 4) * kPartBytes + u * 32 * 128);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) x[i] = key_chunk(i);
#pragma unroll
        for (int i = 0; i < kParts * 4 * kSub; ++i) {
            s[i % kSub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[i % kAhead], qf[i / kSub], s[i % kSub], 0, 0, 0);
            if (i + kAhead < kParts * 4 * kSub) x[i % kAhead] = key_chunk(i + kAhead);
            __builtin_amdgcn_sched_barrier(0);
        }
        bool guarded = false;  // a value of this tile is not finite, and some query does not see all of it
        if constexpr (masked.value) {
            const int left = limit - key0 - 4 * half;  // keys of this tile that this lane's query sees
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (u * 32 + 8 * (i / 4) + i % 4 >= left) s[u][i] = -__builtin_inff();
            constexpr int kReads = KT * VD * 2 / 1024, kRowLanes = VD / 8;
            const unsigned at = lds0 + buf + kParts * kPartBytes + lane * 16;
            u16x2 most = {0, 0};
#pragma unroll
            for (int i = 0; i < kReads; ++i)
                most = __builtin_elementwise_max(most, magnitudes(__builtin_bit_cast(u32x4, lds_chunk(at + i * 1024))));
            guarded = __any(not_finite(most));
            if (guarded) {
                unsigned long long keys = 0;
#pragma unroll 1
                for (int i = 0; i < kReads; ++i) {
                    const unsigned long long bad =
                        __ballot(not_finite(magnitudes(__builtin_bit_cast(u32x4, lds_chunk(at + i * 1024)))));
                    for (int r = 0; r < 64 / kRowLanes; ++r)
                        if (bad >> (r * kRowLanes) & ((1ull << kRowLanes) - 1)) keys |= 1ull << (i * (64 / kRowLanes) + r);
                }
                // the scores of these keys turn NaN where they are seen
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    const unsigned word = (unsigned)(keys >> (u * 32)) >> (4 * half);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int key = 8 * (i / 4) + i % 4;
                        if ((word >> key & 1) && u * 32 + key < left) s[u][i] = __builtin_nanf("");
                    }
                }
            }
        }
        unsigned value_base[4];
#pragma unroll
        for (int k = 0; k < (kOut < 4 ? kOut : 4); ++k) value_base[k] = (value_at + buf) ^ k * 64;
        auto value_chunk = [&](int i) {
            const int k = i / (kSub * 2), u = i % (kSub * 2);
            const unsigned lo = value_base[k % 4] + (k / 4) * 256 + u * 16 * VD * 2;
            return values_transposed(lo, lo + 8 * VD * 2);
        };
        // the first values are read before the exponentials
#pragma unroll
        for (int i = 0; i < kAhead; ++i) x[i] = value_chunk(i);
        // Exponentials against the running maximum as it is.  It only has to
        // move when they grow large: their sum says so (and, at the first
        // tile, infinitely so), without a maximum over every tile.
        bf16x8 p[kSub * 2];
        auto all_exponentials = [&]() {
            float sum = 0.0f;
            const float mc = m * c;
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = s[u][i];
                p[u * 2] = exponentials(v, c, mc, sum);
                p[u * 2 + 1] = exponentials(v + 8, c, mc, sum);
            }
            return sum;
        };
        float sum = all_exponentials();
        if (__any(sum > kMaxSum)) {
            float top = s[0][0];
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
            const float nm = fmaxf(m, half_max(top)), f = __builtin_amdgcn_exp2f((m - nm) * c);
            m = nm;
            l *= f;
#pragma unroll
            for (int k = 0; k < kOut; ++k)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[k][i] *= f;
            sum = all_exponentials();
        }
        l += sum;
        if (masked.value && guarded) {
#pragma unroll
            for (int i = 0; i < kOut * kSub * 2; ++i) {
                const int k = i / (kSub * 2), u = i % (kSub * 2);
                const bf16x8 v = __builtin_bit_cast(bf16x8, finite_only(__builtin_bit_cast(u32x4, value_chunk(i))));
                o[k] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, p[u], o[k], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            return;
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kOut * kSub * 2; ++i) {
            const int k = i / (kSub * 2), u = i % (kSub * 2);
            o[k] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[i % kAhead], p[u], o[k], 0, 0, 0);
            if (i + kAhead < kOut * kSub * 2) x[i % kAhead] = value_chunk(i + kAhead);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Two loops, so that the one over whole tiles carries nothing of the
    // masks; every wave passes one barrier per tile in either.
    if (tiles > 0) issue(0);
    int t = 0;
    for (; t < wave_full; ++t) {
        next_tile(t);
        one_tile(t, std::false_type{});
    }
    for (; t < tiles; ++t) {
        next_tile(t);
        if (t * KT < wave_limit) one_tile(t, std::true_type{});
    }
    if (!row_ok) return;
    l = half_sum(l);
    // a row that sees no key gives zero
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    uint16_t* out = a.out + q_row * a.o_stride_t + h * a.o_stride_h + half * 4;
#pragma unroll
    for (int k = 0; k < kOut; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<u32x2*>(out + k * 32 + i * 8) =
                u32x2{pack_bf16(o[k][i * 4] * inv, o[k][i * 4 + 1] * inv), pack_bf16(o[k][i * 4 + 2] * inv, o[k][i * 4 + 3] * inv)};
}

template <int NOPE, int ROPE, int VD, int KT, int PER_CU>
void launch_shape(const PromptArgs& a, hipStream_t s) {
    const dim3 grid(a.heads, (a.max_q + 127) / 128, a.B);
    hipLaunchKernelGGL((prompt_attention_kernel<NOPE, ROPE, VD, KT, PER_CU>), grid, dim3(256), 0, s, a);
}

}  // namespace

bool prompt_shape_supported(int nope, int rope, int vdim) {
    return rope == 64 && ((nope == 64 && vdim == 64) || (nope == 128 && vdim == 128) || (nope == 192 && vdim == 256));
}

hipError_t launch_prompt_attention(const PromptArgs& a, hipStream_t s) {
    if (a.nope == 64)
        launch_shape<64, 64, 64, 64, 2>(a, s);
    else if (a.nope == 128)
        launch_shape<128, 64, 128, 64, 2>(a, s);
    else  // 230 registers of queries and sums: one wave per SIMD
        launch_shape<192, 64, 256, 32, 1>(a, s);
    return hipGetLastError();
}

}  // namespace moe
