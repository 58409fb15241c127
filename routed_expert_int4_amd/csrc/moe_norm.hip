// Residual addition with root-mean-square norm (bf16 and 8-bit outputs), and
// the write side of the latent cache (norm of the latent, rotation of the
// position part, scatter to slots).
//
// Both are memory bound: each value is read once, kept in registers between
// the sum of squares and the scaling, and written once.  8192 rows of 6144
// (fp32 and bf16 in, bf16 and 8-bit out) 85 us, 5.3 TB/s; 8192 new cache rows
// with 64 heads' queries 27 us, 5.7 TB/s (a large copy reaches 4.75, with as
// much written as read).  One row takes 3 us either way, three latencies.
#include "moe_block.h"
#include "moe_block_device.h"

namespace moe {
namespace {

// Eight values from column c of a row; columns at or past H read as zero.
template <bool VEC>
__device__ __forceinline__ void load8(float (&v)[8], const void* row, int c, int H, bool f32) {
    if constexpr (VEC) {
        if (f32) {
            const f32x4 a = as_global<f32x4>(row)[c / 4], b = as_global<f32x4>(row)[c / 4 + 1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = a[j];
                v[4 + j] = b[j];
            }
        } else {
            const u32x4 a = as_global<u32x4>(row)[c / 8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = bf16_lo(a[j]);
                v[2 * j + 1] = bf16_hi(a[j]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = 0.0f;
            if (c + j < H)
                v[j] = f32 ? as_global<float>(row)[c + j] : bf16_to_f32(as_global<uint16_t>(row)[c + j]);
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(const float (&v)[8], void* row, int c, int H, bool f32) {
    if constexpr (VEC) {
        if (f32) {
            f32x4* p = static_cast<f32x4*>(row) + c / 4;
            p[0] = f32x4{v[0], v[1], v[2], v[3]};
            p[1] = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            static_cast<u32x4*>(row)[c / 8] = u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                    pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < H) {
                if (f32)
                    static_cast<float*>(row)[c + j] = v[j];
                else
                    static_cast<uint16_t*>(row)[c + j] = round_bf16(v[j]);
            }
    }
}

__device__ __forceinline__ const void* row_of(const void* p, long stride, long t, bool f32) {
    return static_cast<const uint8_t*>(p) + t * stride * (f32 ? 4 : 2);
}

// Sum over the block's waves (at most 16), the same in every lane.
__device__ __forceinline__ float block_sum(float v, float* part) {
    v = wave_sum(v);
    const int n = blockDim.x >> 6;
    if (n == 1) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.0f;
    for (int i = 0; i < n; ++i) t += part[i];
    return t;
}

// The group of 128 columns that this lane's eight belong to lies in 16
// neighbouring lanes: its largest magnitude, scale and codes.
template <bool VEC>
__device__ __forceinline__ void store_fp8(const float (&y)[8], int c, int H, uint8_t* q_row, float* scale_row,
                                          long scale_stride_g) {
    unsigned top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = umax(top, __builtin_bit_cast(unsigned, y[j]) & 0x7FFFFFFFu);
    const float s = group_scale(row_max_u32(top));
    if (c >= H) return;
    if ((threadIdx.x & 15) == 0) scale_row[(long)(c >> 7) * scale_stride_g] = s;
    const float inv = 1.0f / s;
    const unsigned lo = pack_fp8x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    const unsigned hi = pack_fp8x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
    if constexpr (VEC) {
        reinterpret_cast<u32x2*>(q_row)[c >> 3] = u32x2{lo, hi};
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < H) q_row[c + j] = (uint8_t)((j < 4 ? lo >> (8 * j) : hi >> (8 * (j - 4))) & 255u);
    }
}

// One row per workgroup, eight columns per lane and round, I rounds: the row
// stays in registers.  TYPES fixes the operand types of the 16-byte path (a
// branch on them between the loads would wait for each in turn): residual 0
// none, 1 bf16, 2 fp32, + 3 for fp32 x, + 6 for fp32 weights, + 12 for none (no
// norm: the addition and the 8-bit output alone); -1 leaves all to the
// arguments and moves single elements.
template <int I, int TYPES>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(NormArgs a) {
    constexpr bool VEC = TYPES >= 0;
    __shared__ float part[16];
    const long t = blockIdx.x;
    if constexpr (VEC) {
        a.x_f32 = TYPES / 3 % 2, a.weight_f32 = TYPES / 6 == 1;
        if (TYPES >= 12) a.weight = nullptr;
        a.residual_f32 = TYPES % 3 == 2;
        if (TYPES % 3 == 0) a.residual = nullptr;
        a.sum_f32 = TYPES % 3 ? a.residual_f32 : a.x_f32;
    }
    const void* x = row_of(a.x, a.x_stride, t, a.x_f32);
    const void* r = a.residual ? row_of(a.residual, a.residual_stride, t, a.residual_f32) : nullptr;
    void* sum = a.sum ? const_cast<void*>(row_of(a.sum, a.sum_stride, t, a.sum_f32)) : nullptr;
    float v[I][8], w[I][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        if (c < a.H) {
            load8<VEC>(v[i], x, c, a.H, a.x_f32);
            if (a.weight) load8<VEC>(w[i], a.weight, c, a.H, a.weight_f32);
            if (r) {
                float u[8];
                load8<VEC>(u, r, c, a.H, a.residual_f32);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += u[j];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    const float rms = a.weight ? 1.0f / sqrtf(block_sum(ss, part) / (float)a.H + a.eps) : 1.0f;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c < a.H && sum) store8<VEC>(v[i], sum, c, a.H, a.sum_f32);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = c + j < a.H ? (a.weight ? v[i][j] * rms * w[i][j] : v[i][j]) : 0.0f;
        if (c < a.H && a.y) store8<VEC>(y, a.y + t * a.y_stride, c, a.H, false);
        if (a.q) store_fp8<VEC>(y, c, a.H, a.q + t * a.q_stride, a.scale + t * a.scale_stride_t, a.scale_stride_g);
    }
}

// Rotates the pair (even, odd) columns 2i, 2i + 1 by the angle of pair i:
// eight columns from an even column c.
__device__ __forceinline__ u32x4 rotate8(u32x4 u, const float* cos_row, int c, int rope) {
    const int i = c / 2;
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float co = as_global<float>(cos_row)[i + j], si = as_global<float>(cos_row)[rope / 2 + i + j];
        const float e = bf16_lo(u[j]), d = bf16_hi(u[j]);
        o[j] = pack_bf16(e * co - d * si, e * si + d * co);
    }
    return o;
}

// One workgroup per token.  Wave 0 (lanes of eight columns, up to four
// rounds) norms the latent; all lanes rotate: the key's position part first,
// then the queries', eight columns each.
__global__ void __launch_bounds__(256) latent_append_kernel(AppendArgs a) {
    const long t = blockIdx.x;
    const int rope8 = a.rope / 8;
    const int pos = a.positions[t];
    const int64_t slot = a.slots ? a.slots[t] : -1;
    const uint16_t* kv = a.kv + t * a.kv_stride;
    // a slot outside the pool writes no row; a position outside the table
    // has no angle and rotates to NaN
    uint16_t* row = a.cache && slot >= 0 && slot < a.n_slots ? a.cache + slot * (a.rank + a.rope) : nullptr;
    const bool known = pos >= 0 && pos < a.n_positions;
    const float* angle = a.table + (known ? (long)pos * a.rope : 0);
    const u32x4 nan = {0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
    if (threadIdx.x < 64) {
        constexpr int I = kAppendMaxRank / 512;
        float v[I][8];
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int c = (threadIdx.x + i * 64) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
            if (c < a.rank) load8<true>(v[i], kv, c, a.rank, false);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
        }
        const float rms = 1.0f / sqrtf(wave_sum(ss) / (float)a.rank + a.eps);
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int c = (threadIdx.x + i * 64) * 8;
            if (i * 512 >= a.rank) break;
            float y[8], w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 0.0f;
            if (c < a.rank) load8<true>(w, a.weight, c, a.rank, a.weight_f32);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = v[i][j] * rms * w[j];
            if (c < a.rank && row) store8<true>(y, row, c, a.rank, false);
            if (c < a.rank && a.rows) store8<true>(y, a.rows + t * a.rows_stride, c, a.rank, false);
            if (a.lat_q)
                store_fp8<true>(y, c, a.rank, a.lat_q + t * a.lat_stride, a.lat_scale + t * a.ls_stride_t,
                                a.ls_stride_g);
        }
    }
    const int jobs = rope8 * (1 + (a.q ? a.heads : 0));
    // the key's jobs go to the last lanes, which have no latent to norm
    for (int k = blockDim.x - 1 - threadIdx.x; k < jobs; k += blockDim.x) {
        const int h = k / rope8 - 1, c = (k % rope8) * 8;
        if (h < 0) {
            if (!row && !a.rows) continue;
            const u32x4 o = known ? rotate8(as_global<u32x4>(kv + a.rank)[c / 8], angle, c, a.rope) : nan;
            if (row) *reinterpret_cast<u32x4*>(row + a.rank + c) = o;
            if (a.rows) *reinterpret_cast<u32x4*>(a.rows + t * a.rows_stride + a.rank + c) = o;
        } else {
            const u32x4 u = *as_global<u32x4>(a.q + t * a.q_stride_t + h * a.q_stride_h + c);
            *reinterpret_cast<u32x4*>(a.q_out + t * a.qo_stride_t + h * a.qo_stride_h + c) =
                known ? rotate8(u, angle, c, a.rope) : nan;
        }
    }
}

template <int I, int TYPES>
void launch_norm_types(const NormArgs& a, int types, int threads, hipStream_t s) {
    if constexpr (TYPES < 18) {
        if (types == TYPES)
            hipLaunchKernelGGL((add_rmsnorm_kernel<I, TYPES>), dim3(a.T), dim3(threads), 0, s, a);
        else
            launch_norm_types<I, TYPES + 1>(a, types, threads, s);
    }
}
template <int I>
void launch_norm_rounds(const NormArgs& a, int threads, bool vec, hipStream_t s) {
    const int types = vec ? (a.residual ? 1 + a.residual_f32 : 0) + 3 * a.x_f32 +
                                (a.weight ? 6 * a.weight_f32 : 12)
                          : -1;
    launch_norm_types<I, -1>(a, types, threads, s);
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s) {
    // 16-byte accesses where every row of every tensor starts on 16 bytes
    // (8 for the codes)
    const bool vec = a.H % 8 == 0 && aligned(a.x, 16) && a.x_stride % 8 == 0 && (!a.weight || aligned(a.weight, 16)) &&
                     (!a.residual || (aligned(a.residual, 16) && a.residual_stride % 8 == 0)) &&
                     (!a.sum || (aligned(a.sum, 16) && a.sum_stride % 8 == 0)) &&
                     (!a.y || (aligned(a.y, 16) && a.y_stride % 8 == 0)) &&
                     (!a.q || (aligned(a.q, 8) && a.q_stride % 8 == 0));
    const int lanes = ((a.H + 7) / 8 + 63) / 64 * 64;
    // Few rows: one round over as many lanes as the row needs (the shortest
    // path for one token).  Many rows: up to three rounds per lane, so that
    // each lane has several loads in flight.
    int rounds = (lanes + 1023) / 1024;
    if (a.T >= 512 && lanes >= 256) rounds = lanes >= 4 * rounds * 192 ? (rounds > 3 ? rounds : 3) : (rounds > 2 ? rounds : 2);
    const int threads = ((lanes + rounds - 1) / rounds + 63) / 64 * 64;
    switch (rounds) {
        case 1: launch_norm_rounds<1>(a, threads, vec, s); break;
        case 2: launch_norm_rounds<2>(a, threads, vec, s); break;
        case 3: launch_norm_rounds<3>(a, threads, vec, s); break;
        default: launch_norm_rounds<4>(a, threads, vec, s); break;
    }
    return hipGetLastError();
}

hipError_t launch_latent_append(const AppendArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(latent_append_kernel, dim3(a.T), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
