// Kernel arguments and launchers of the attention half of a decoder block
// (include/moe.h, "attention half of a decoder block").  The launchers assume
// arguments that moe_block_abi.cpp has validated and return the launch error.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace moe {

struct NormArgs {
    const void* x;
    const void* residual;  // or nullptr
    const void* weight;
    void* sum;             // residual's type (x's without one), or nullptr
    uint16_t* y;           // bf16, or nullptr
    uint8_t* q;            // E4M3, or nullptr
    float* scale;
    long x_stride, residual_stride, sum_stride, y_stride, q_stride, scale_stride_t, scale_stride_g;
    int T, H;
    float eps;
    bool x_f32, residual_f32, weight_f32, sum_f32;
};
hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s);
constexpr int kNormMaxWidth = 32768;

struct AppendArgs {
    const uint16_t* kv;
    const void* weight;
    const float* table;        // [n_positions][rope]: cosines, then sines
    const int32_t* positions;
    const int64_t* slots;
    uint16_t* cache;           // [n_slots][rank + rope], or nullptr
    const uint16_t* q;         // [T][heads][rope] strided, or nullptr
    uint16_t* q_out;
    uint8_t* lat_q;            // [T][rank] E4M3, or nullptr
    float* lat_scale;
    uint16_t* rows;            // [T][rank + rope], or nullptr
    long kv_stride, n_slots, q_stride_t, q_stride_h, qo_stride_t, qo_stride_h, lat_stride, ls_stride_t, ls_stride_g,
        rows_stride;
    int T, rank, rope, heads, n_positions;
    float eps;
    bool weight_f32;
};
hipError_t launch_latent_append(const AppendArgs& a, hipStream_t s);
constexpr int kAppendMaxRank = 2048;

struct HeadArgs {
    const uint16_t* x;
    const uint16_t* w;  // [heads][N][K]
    uint16_t* out;
    long x_stride_t, x_stride_h, o_stride_t, o_stride_h;
    int T, heads, K, N;
    bool out_vec;  // eight neighbouring outputs may be stored at once
};
hipError_t launch_head_linear(const HeadArgs& a, hipStream_t s);

struct Fp8Args {
    const uint8_t* a;
    const float* a_scale;
    const uint8_t* w;
    const float* w_scale;
    void* out;
    long lda, as_t, as_k, ldw, ws_n, ldo;
    int M, N, K;
    bool out_f32, out_vec;  // out_vec: eight consecutive columns may be stored at once
};
hipError_t launch_fp8_linear(const Fp8Args& a, hipStream_t s);

struct LatentArgs {
    const uint16_t* q;      // [T][heads][rank + rope]
    const uint16_t* cache;  // [n_pages][page_size][rank + rope]
    const int32_t* pages;   // [B][pages_stride]
    const int32_t* lens;    // [B]
    const int32_t* cu_q;    // [B + 1], or nullptr: T / B tokens each
    const int64_t* tree;    // [T] masks, or nullptr
    uint16_t* out;          // [T][heads][rank]
    uint8_t* ws;            // latent_workspace() bytes
    long q_stride_t, q_stride_h, o_stride_t, o_stride_h, pages_stride, cache_page_stride;
    int T, B, heads, rank, rope, n_pages, page_size, pages_per_seq, max_q, max_len;
    int group, runs, per_seq;  // how the call is cut, filled in by the launcher
    float scale;
};
// Device workspace of a call (partial sums of the split sequences).
size_t latent_workspace(int B, int max_q, int heads, int rank, int max_len);
bool latent_shape_supported(int rank, int rope);
hipError_t launch_latent_attention(const LatentArgs& a, hipStream_t s);

struct PromptArgs {
    const uint16_t* q;       // [Tq][heads][nope + rope]
    const uint16_t* k;       // [Tk][heads][nope]
    const uint16_t* k_rope;  // [Tk][rope]
    const uint16_t* v;       // [Tk][heads][vdim]
    const int32_t* cu_q;
    const int32_t* cu_k;
    uint16_t* out;           // [Tq][heads][vdim]
    long q_stride_t, q_stride_h, k_stride_t, k_stride_h, kr_stride_t, v_stride_t, v_stride_h, o_stride_t, o_stride_h;
    int Tq, Tk, B, heads, nope, rope, vdim, max_q;
    float scale;
    bool causal;
};
bool prompt_shape_supported(int nope, int rope, int vdim);
hipError_t launch_prompt_attention(const PromptArgs& a, hipStream_t s);

}  // namespace moe
