// Device helpers of the attention-half kernels: bf16 and E4M3 conversion,
// asynchronous loads into LDS, and the matrix-core wrappers they share.
#pragma once

#include "moe_device.h"

namespace moe {
namespace {

// One load from every 64 bytes of a kernel's arguments, so that those that are
// first used late are in the scalar cache by then (each line is a trip to
// memory, one after the other where they are used).
template <int BYTES>
__device__ __forceinline__ void touch_arguments() {
    const auto* p = (const __attribute__((address_space(4))) int*)__builtin_amdgcn_kernarg_segment_ptr();
    int all = 0;
#pragma unroll
    for (int i = 0; i < BYTES; i += 64) all ^= p[i / 4];
    asm volatile("" ::"s"(all));
}


typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float kFp8Max = 448.0f;  // largest E4M3 value

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __builtin_bit_cast(float, (unsigned)b << 16); }
__device__ __forceinline__ float bf16_lo(unsigned u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float bf16_hi(unsigned u) { return __builtin_bit_cast(float, u & 0xFFFF0000u); }

// Two fp32 values rounded to nearest even bf16, packed (first in the low half).
__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
    bf16x2 v;
    v[0] = (__bf16)a;
    v[1] = (__bf16)b;
    return __builtin_bit_cast(unsigned, v);
}
__device__ __forceinline__ uint16_t round_bf16(float a) { return __builtin_bit_cast(uint16_t, (__bf16)a); }

// Clamp to the E4M3 range that leaves NaN as it is (the conversion then
// writes the NaN code; a min/max pair would turn it into 448).
__device__ __forceinline__ float clamp_fp8(float v) {
    return __builtin_fabsf(v) > kFp8Max ? __builtin_copysignf(kFp8Max, v) : v;
}
__device__ __forceinline__ unsigned pack_fp8x4(float a, float b, float c, float d) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_fp8(a), clamp_fp8(b), 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(clamp_fp8(c), clamp_fp8(d), r, true);
}

// Maximum over the 16 lanes of a row, in all of them.
__device__ __forceinline__ unsigned row_max_u32(unsigned v) {
    v = umax(v, dpp_u<kDppXor1>(v));
    v = umax(v, dpp_u<kDppXor2>(v));
    v = umax(v, dpp_u<kDppHalfMirror>(v));
    return umax(v, dpp_u<kDppMirror>(v));
}

// Scale of one group of 128 values whose largest magnitude has the bits
// `top` (the integer order of magnitudes puts NaN above infinity, so a NaN
// in the group makes its scale NaN).
__device__ __forceinline__ float group_scale(unsigned top) {
    const float s = __builtin_bit_cast(float, top) * (1.0f / kFp8Max);
    return s < 1e-12f ? 1e-12f : s;
}

// 8-bit cache rows: E4M3 codes times a power of two.  A code has 4 bits of
// significand, so a row's values are exact in bf16.
// The least power of two that brings magnitudes up to the one with the bits
// `top` (finite) into the codes' range; 1 for zero.
__device__ __forceinline__ float row_power(unsigned top) {
    const int e = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u);  // 448 = 1.75 * 2^8
    return top == 0 ? 1.0f : __builtin_bit_cast(float, (unsigned)(e < 27 ? 27 : e) << 23);  // 2^-100 and up
}
// Eight codes as bf16.
__device__ __forceinline__ u32x4 codes_to_bf16(unsigned lo, unsigned hi, float scale) {
    return u32x4{__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false)),
                 __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true)),
                 __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false)),
                 __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true))};
}

// 16 bytes per lane from global memory straight into LDS: lane l's bytes land
// at dst + 16 l.  dst is wave-uniform.  Written in assembly because the
// compiler drains every outstanding one before the next LDS read of any
// kind; the kernels wait with wait_vmem<n>() where a tile is needed.  It has
// no register output.  The compiler's own waits stay safe: a counter that
// holds more operations than it knows of only makes them wait longer.  m0 is
// set in the same block; nothing else in these kernels uses it.
__device__ __forceinline__ unsigned lds_address(const void* p) {
    return (unsigned)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
__device__ __forceinline__ void load_to_lds16(const void* src, unsigned dst) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src),
                 "s"(__builtin_amdgcn_readfirstlane(dst))
                 : "memory");
}
// The same from a base in scalar registers plus a byte offset per lane.  A lane
// read may just have made the base, here or in the caller, and a vector memory
// instruction may read such a register five wait states later: s_mov and s_nop
// are those, since the compiler adds none in front of inline assembly.
__device__ __forceinline__ void load_to_lds16_lane(unsigned long long base, unsigned offset, unsigned dst) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base),
                 "s"(__builtin_amdgcn_readfirstlane(dst))
                 : "memory");
}
// The same from a wave-uniform base, wherever the compiler keeps it.
__device__ __forceinline__ void load_to_lds16(const void* base, unsigned offset, unsigned dst) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    const unsigned lo = __builtin_amdgcn_readfirstlane((unsigned)p), hi = __builtin_amdgcn_readfirstlane((unsigned)(p >> 32));
    load_to_lds16_lane((uint64_t)hi << 32 | lo, offset, dst);
}
// Four bytes per lane into LDS: lane l's bytes land at dst + 4 l.
__device__ __forceinline__ void load_to_lds4(const void* src, unsigned dst) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src),
                 "s"(__builtin_amdgcn_readfirstlane(dst))
                 : "memory");
}
// Waits until at most N of the wave's vector memory operations are
// outstanding.
template <int N>
__device__ __forceinline__ void wait_vmem() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
}
// Barrier without the drain of outstanding loads that __syncthreads adds;
// LDS operations of the wave are complete before it.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Source of rows that lie outside a tensor or are masked away: as long as the
// longest row loaded at once.
__device__ __attribute__((aligned(16))) const uint8_t kZeros[2048] = {};

// ------------------------------------------------- attention, one wave's part
// Scores are computed transposed: a 32 x 32 matrix instruction with keys as
// rows and queries as columns leaves lane l with query l % 32 and, in
// register i, key 8 (i / 4) + 4 (l / 32) + i % 4.  The softmax statistics of
// a query then live in its two lanes, and the exponentials are, rounded to
// bf16, already the column operand of the product with the values: step s of
// 16 keys takes registers 8 s .. 8 s + 7, that is keys 16 s + 4 (l / 32) +
// 0..3 and 16 s + 8 + 4 (l / 32) + 0..3 of the lane's half, and the value
// operand is read in the same order.
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
// LDS addresses are kept as 32-bit integers (the host pass, whose pointers
// are wider, would warn at each use)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Wint-to-pointer-cast"

// Value operand: 32 columns by 16 keys, read transposed out of rows of keys.
// lo and hi: this lane's LDS addresses in the rows of its first and second
// four keys.
__device__ __forceinline__ bf16x8 values_transposed(unsigned lo, unsigned hi) {
    const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)lo);
    const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)hi);
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    const i16x8 v = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return __builtin_bit_cast(bf16x8, v);
}

// The same of 8-bit codes, one read: 16 columns (by lane) by eight keys, whose
// rows' first or last eight bytes this lane's address names.
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
__device__ __forceinline__ u32x2 codes_transposed(unsigned addr) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)addr));
}

__device__ __forceinline__ bf16x8 lds_chunk(unsigned addr) {
    return __builtin_bit_cast(bf16x8, *(lds_u32x4*)addr);
}
__device__ __forceinline__ unsigned lds_dword(unsigned addr) { return *(__attribute__((address_space(3))) unsigned*)addr; }
__device__ __forceinline__ void lds_store(unsigned addr, u32x4 v) { *(lds_u32x4*)addr = v; }
#pragma clang diagnostic pop

// Largest value of the two lanes (halves of the wave) that share a query.
__device__ __forceinline__ float half_max(float v) {
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned a = r[0], b = r[1];
    return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float half_sum(float v) {
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned a = r[0], b = r[1];
    return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}

// Values that are not finite.  A masked key has an exponential of zero, and
// zero times infinity is NaN: in tiles where some query does not see a key
// that others do, values are looked over first, and where one is not finite
// only the finite ones enter the sums; a query that does see such a key
// becomes NaN through its exponential.
// Largest magnitudes, as bits, of the even and the odd values; not_finite says
// whether one of them is not finite.
__device__ __forceinline__ u16x2 magnitudes(u32x4 v) {
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7FFF7FFFu));
    return m;
}
__device__ __forceinline__ bool not_finite(u16x2 m) { return m[0] >= 0x7F80 || m[1] >= 0x7F80; }
__device__ __forceinline__ u32x4 finite_only(u32x4 u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned low = (u[i] & 0x7F80u) == 0x7F80u ? 0u : u[i] & 0xFFFFu;
        const unsigned high = (u[i] & 0x7F800000u) == 0x7F800000u ? 0u : u[i] & 0xFFFF0000u;
        u[i] = low | high;
    }
    return u;
}

// Exponentials of eight scores as the product with the values takes them, and
// their sum added to l (of the rounded ones, two at a time, so that numerator
// and denominator agree).
__device__ __forceinline__ bf16x8 exponentials(const float* s, float c, float mc, float& l) {
    bf16x8 p;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float e = __builtin_amdgcn_exp2f(fmaf(s[i], c, -mc)), f = __builtin_amdgcn_exp2f(fmaf(s[i + 1], c, -mc));
        const unsigned pair = pack_bf16(e, f);
        const unsigned one = 0x3F803F80u;
        l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(i16x2, pair), __builtin_bit_cast(i16x2, one), l, false);
        const bf16x2 v = __builtin_bit_cast(bf16x2, pair);
        p[i] = v[0];
        p[i + 1] = v[1];
    }
    return p;
}

// Running statistics start from a finite value, so that a row of masked
// scores (-inf) gives exponentials of zero and never inf - inf.
constexpr float kNoMax = -1e30f;
// The running maximum only moves (and the sums are only rescaled) when a new
// score exceeds it by more than this many powers of two: exponentials stay
// below 2^8, which costs fp32 sums and bf16 exponentials no relative accuracy.
constexpr float kMaxSlack = 8.0f;
// The same bound on a tile's sum of exponentials.
constexpr float kMaxSum = 65536.0f;

}  // namespace
}  // namespace moe
