// Host side of the attention half of the C ABI (include/moe.h): argument
// validation and dispatch.  Nothing is enqueued on an argument error.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/moe.h"
#include "moe_block.h"
#include "moe_internal.h"

using namespace moe;

namespace {

bool on(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool type_ok(int t) { return t == MOE_BF16 || t == MOE_F32; }
// offsets inside a tile are 32-bit: 256 rows of this many bytes
bool stride_fits(int64_t bytes) { return bytes >= 0 && bytes < (int64_t)1 << 23; }

moe_status_t launched(hipError_t e, const char* who) { return e == hipSuccess ? MOE_OK : hip_fail(e, who); }

// The bf16 cache or the 8-bit one (with its scales), or neither.
moe_status_t append(const char* who, uint8_t* d_cache8, float* d_cache_scale, const uint16_t* d_kv, int64_t kv_stride,
                    const void* d_weight, int weight_type, float eps, int rank, int rope, const float* d_table,
                    int n_positions, const int32_t* d_positions, const int64_t* d_slots, int T, uint16_t* d_cache,
                    int64_t n_slots, const uint16_t* d_q_rope, int heads, int64_t q_stride_t, int64_t q_stride_h,
                    uint16_t* d_q_out, int64_t qo_stride_t, int64_t qo_stride_h, uint8_t* d_lat_q, int64_t lat_stride,
                    float* d_lat_scale, int64_t ls_stride_t, int64_t ls_stride_g, uint16_t* d_rows, int64_t rows_stride,
                    void* stream) {
    if (T < 0 || rank < 1 || rope < 1 || n_positions < 0 || n_slots < 0 || (d_q_rope && heads < 1))
        return fail(MOE_EINVAL, "%s: T (%d), rank (%d), rope (%d), heads (%d), positions (%d) or slots", who, T, rank,
                    rope, heads, n_positions);
    if (!type_ok(weight_type)) return fail(MOE_EINVAL, "%s: unknown weight type %d", who, weight_type);
    if (!(eps >= 0.0f)) return fail(MOE_EINVAL, "%s: eps must be >= 0", who);
    if (T == 0) return MOE_OK;
    if (!d_kv || !d_weight || !d_table || !d_positions) return fail(MOE_EINVAL, "%s: NULL pointer", who);
    if ((d_cache || d_cache8) && !d_slots) return fail(MOE_EINVAL, "%s: a cache without slots", who);
    if (!d_q_rope != !d_q_out) return fail(MOE_EINVAL, "%s: queries need both an input and an output", who);
    if (!d_lat_q != !d_lat_scale) return fail(MOE_EINVAL, "%s: the 8-bit latent needs codes and scales", who);
    if (!d_cache && !d_cache8 && !d_q_rope && !d_lat_q && !d_rows) return fail(MOE_EINVAL, "%s: no output", who);
    if (kv_stride < rank + rope || (d_lat_q && lat_stride < rank) || (d_rows && rows_stride < rank + rope))
        return fail(MOE_EINVAL, "%s: a row stride is below its row", who);
    if (rank > kAppendMaxRank) return fail(MOE_EUNSUPPORTED, "%s: rank (%d) is over %d", who, rank, kAppendMaxRank);
    if (rank % 8 || rope % 8 || kv_stride % 8 || q_stride_t % 8 || q_stride_h % 8 || qo_stride_t % 8 ||
        qo_stride_h % 8 || lat_stride % 8 || rows_stride % 8 || !on(d_kv, 16) || !on(d_weight, 16) ||
        !on(d_cache, 16) || !on(d_q_rope, 16) || !on(d_q_out, 16) || !on(d_lat_q, 8) || !on(d_rows, 16))
        return fail(MOE_EUNSUPPORTED, "%s: rank, rope and the strides must be multiples of 8, pointers 16-byte aligned",
                    who);
    if (d_cache8 && (rank % 16 || !on(d_cache8, 16)))
        return fail(MOE_EUNSUPPORTED, "%s: rows of 8 bits need a rank (%d) that is a multiple of 16, 16-byte aligned", who,
                    rank);
    if (!on(d_table, 4) || !on(d_positions, 4) || !on(d_slots, 8) || !on(d_lat_scale, 4) || !on(d_cache_scale, 4))
        return fail(MOE_EINVAL, "%s: a pointer is not aligned to its type", who);
    AppendArgs a{};
    a.kv = d_kv, a.weight = d_weight, a.table = d_table, a.positions = d_positions, a.slots = d_slots;
    a.cache = d_cache, a.cache8 = d_cache8, a.cache_scale = d_cache_scale, a.q = d_q_rope, a.q_out = d_q_out, a.lat_q = d_lat_q, a.lat_scale = d_lat_scale, a.rows = d_rows;
    a.kv_stride = kv_stride, a.n_slots = n_slots, a.q_stride_t = q_stride_t, a.q_stride_h = q_stride_h;
    a.qo_stride_t = qo_stride_t, a.qo_stride_h = qo_stride_h, a.lat_stride = lat_stride, a.ls_stride_t = ls_stride_t;
    a.ls_stride_g = ls_stride_g, a.rows_stride = rows_stride;
    a.T = T, a.rank = rank, a.rope = rope, a.heads = heads, a.n_positions = n_positions, a.eps = eps;
    a.weight_f32 = weight_type == MOE_F32;
    return launched(launch_latent_append(a, static_cast<hipStream_t>(stream)), who);
}

// Over rows of either width (8 bits where there are scales; the page stride
// counts bytes then), with prefixes if there are any.
moe_status_t attend(const char* who, const float* d_cache_scale, const PrefixArgs& prefix, const uint16_t* d_q,
                    int64_t q_stride_t, int64_t q_stride_h, int T, int heads, int rank, int rope, const void* d_cache,
                    int n_pages, int page_size, int64_t page_stride, const int32_t* d_pages, int64_t pages_stride,
                    int pages_per_seq, const int32_t* d_lens, int B, const int32_t* d_cu_q, int max_q, int max_len,
                    const int64_t* d_tree, float scale, uint16_t* d_out, int64_t out_stride_t, int64_t out_stride_h,
                    void* d_ws, size_t ws_bytes, void* stream) {
    if (T < 0 || B < 0 || heads < 1 || n_pages < 0 || page_size < 1 || pages_per_seq < 0 || max_q < 0 || max_len < 0)
        return fail(MOE_EINVAL, "%s: a size is negative (or heads or page_size below 1)", who);
    if (!(scale > 0.0f) || !std::isfinite(scale)) return fail(MOE_EINVAL, "%s: scale must be positive", who);
    if (!latent_shape_supported(rank, rope))
        return fail(MOE_EUNSUPPORTED, "%s: no kernel for rank %d and rope %d", who, rank, rope);
    if (T == 0) return MOE_OK;
    if (B < 1 || max_q < 1) return fail(MOE_EINVAL, "%s: tokens without a sequence", who);
    if (!d_q || !d_lens || !d_out || (n_pages > 0 && !d_cache) || (pages_per_seq > 0 && !d_pages))
        return fail(MOE_EINVAL, "%s: NULL pointer", who);
    if (!d_cu_q && (T % B || T / B > max_q))
        return fail(MOE_EINVAL, "%s: T (%d) is not B (%d) times at most max_q (%d) tokens", who, T, B, max_q);
    const bool narrow = d_cache_scale != nullptr, shared = prefix.count > 0;
    if (page_stride < (int64_t)page_size * (narrow ? rank + 2 * rope : rank + rope) || pages_stride < pages_per_seq)
        return fail(MOE_EINVAL, "%s: a stride is below its row", who);
    if (q_stride_t % 8 || q_stride_h % 8 || page_stride % (narrow ? 16 : 8) || out_stride_t % 4 || out_stride_h % 4 ||
        !on(d_q, 16) || !on(d_cache, 16) || !on(d_out, 8))
        return fail(MOE_EUNSUPPORTED, "%s: strides must be multiples of 8 (out: 4; pages of 8 bits: 16), q and cache "
                    "16-byte aligned, out 8-byte", who);
    if (!on(d_pages, 4) || !on(d_lens, 4) || !on(d_cu_q, 4) || !on(d_tree, 8) || !on(d_cache_scale, 4) ||
        !on(prefix.pages, 4) || !on(prefix.lens, 4) || !on(prefix.groups, 4))
        return fail(MOE_EINVAL, "%s: a pointer is not aligned to its type", who);
    // tile counts are 32-bit: row blocks of all sequences times tiles of the longest
    const int64_t rows_per_table = (int64_t)pages_per_seq * page_size;
    if (rows_per_table > ((int64_t)1 << 31) - 128 || B > 65535 || (int64_t)max_q * heads > (int64_t)1 << 30 ||
        (double)(B + (int64_t)T * heads / 32) * (double)(rows_per_table / 64 + 1) > (double)(1 << 30))
        return fail(MOE_EUNSUPPORTED, "%s: too many tiles", who);
    // the second launch has a wave per row of the longest sequence, and 32-bit grids count lanes
    if ((int64_t)(max_q < T ? max_q : T) * heads >= (int64_t)1 << 26)
        return fail(MOE_EUNSUPPORTED, "%s: 2^26 or more rows (tokens times heads) in a sequence", who);
    if (shared) {
        const int64_t reach = (int64_t)prefix.pages_per_seq * page_size;
        if (reach > ((int64_t)1 << 31) - 128 || (int64_t)T * heads >= (int64_t)1 << 26 ||
            (double)(prefix.count + (int64_t)T * heads / 32) * (double)(reach / 64 + 1) > (double)(1 << 30))
            return fail(MOE_EUNSUPPORTED, "%s: 2^26 or more rows (tokens times heads) or too many tiles of prefixes", who);
    }
    const size_t need = shared ? latent_shared_workspace(B, T, max_q, heads, rank, max_len, prefix.count, prefix.max_len)
                               : latent_workspace(B, max_q, heads, rank, max_len);
    if (!d_ws || ws_bytes < need || !on(d_ws, 256))
        return fail(MOE_EINVAL, "%s: workspace of %zu bytes given, %zu needed (256-byte aligned)", who, ws_bytes, need);
    LatentArgs a{};
    a.q = d_q, a.cache = static_cast<const uint16_t*>(d_cache), a.cache_scale = d_cache_scale, a.pages = d_pages;
    a.lens = d_lens, a.cu_q = d_cu_q, a.tree = d_tree, a.out = d_out;
    a.ws = static_cast<uint8_t*>(d_ws);
    a.q_stride_t = q_stride_t, a.q_stride_h = q_stride_h, a.o_stride_t = out_stride_t, a.o_stride_h = out_stride_h;
    a.pages_stride = pages_stride, a.cache_page_stride = narrow ? page_stride / 2 : page_stride;
    a.T = T, a.B = B, a.heads = heads, a.rank = rank, a.rope = rope, a.n_pages = n_pages, a.page_size = page_size;
    a.pages_per_seq = pages_per_seq, a.max_q = max_q, a.max_len = max_len, a.scale = scale;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return launched(shared ? launch_latent_shared(a, prefix, s) : launch_latent_attention(a, s), who);
}

}  // namespace

extern "C" {

moe_status_t moe_add_rmsnorm(const void* d_x, int x_type, int64_t x_stride, const void* d_residual,
                             int residual_type, int64_t residual_stride, const void* d_weight, int weight_type,
                             int T, int H, float eps, void* d_sum, int64_t sum_stride, uint16_t* d_y,
                             int64_t y_stride, uint8_t* d_q, int64_t q_stride, float* d_scale,
                             int64_t scale_stride_t, int64_t scale_stride_g, void* stream) {
    const char* who = "moe_add_rmsnorm";
    if (T < 0 || H < 1) return fail(MOE_EINVAL, "%s: T (%d) must be >= 0 and H (%d) >= 1", who, T, H);
    if (!type_ok(x_type) || !type_ok(weight_type) || (d_residual && !type_ok(residual_type)))
        return fail(MOE_EINVAL, "%s: unknown type", who);
    if (!(eps >= 0.0f)) return fail(MOE_EINVAL, "%s: eps must be >= 0", who);
    if (H > kNormMaxWidth) return fail(MOE_EUNSUPPORTED, "%s: H (%d) is over %d", who, H, kNormMaxWidth);
    if (T == 0) return MOE_OK;
    if (!d_x) return fail(MOE_EINVAL, "%s: NULL x", who);
    if (!d_sum && !d_y && !d_q) return fail(MOE_EINVAL, "%s: no output", who);
    if (d_q && !d_scale) return fail(MOE_EINVAL, "%s: 8-bit output without scales", who);
    const bool sum_f32 = (d_residual ? residual_type : x_type) == MOE_F32;
    if (x_stride < H || (d_residual && residual_stride < H) || (d_sum && sum_stride < H) || (d_y && y_stride < H) ||
        (d_q && q_stride < H))
        return fail(MOE_EINVAL, "%s: a row stride is below H (%d)", who, H);
    if (!on(d_x, x_type == MOE_F32 ? 4 : 2) || (d_sum && !on(d_sum, sum_f32 ? 4 : 2)) ||
        (d_residual && !on(d_residual, residual_type == MOE_F32 ? 4 : 2)) ||
        !on(d_weight, weight_type == MOE_F32 ? 4 : 2) || !on(d_y, 2) || !on(d_scale, 4))
        return fail(MOE_EINVAL, "%s: a pointer is not aligned to its type", who);
    NormArgs a{};
    a.x = d_x, a.residual = d_residual, a.weight = d_weight, a.sum = d_sum, a.y = d_y, a.q = d_q, a.scale = d_scale;
    a.x_stride = x_stride, a.residual_stride = residual_stride, a.sum_stride = sum_stride, a.y_stride = y_stride;
    a.q_stride = q_stride, a.scale_stride_t = scale_stride_t, a.scale_stride_g = scale_stride_g;
    a.T = T, a.H = H, a.eps = eps;
    a.x_f32 = x_type == MOE_F32, a.residual_f32 = residual_type == MOE_F32, a.weight_f32 = weight_type == MOE_F32;
    a.sum_f32 = sum_f32;
    return launched(launch_add_rmsnorm(a, static_cast<hipStream_t>(stream)), who);
}

moe_status_t moe_fp8_linear(const uint8_t* d_a, int64_t a_stride, const float* d_a_scale, int64_t as_stride_m,
                            int64_t as_stride_b, const uint8_t* d_w, int64_t w_stride, const float* d_w_scale,
                            int64_t ws_stride, int M, int N, int K, void* d_out, int out_type, int64_t out_stride,
                            void* stream) {
    const char* who = "moe_fp8_linear";
    if (M < 0 || N < 1 || K < 1) return fail(MOE_EINVAL, "%s: M (%d), N (%d), K (%d)", who, M, N, K);
    if (!type_ok(out_type)) return fail(MOE_EINVAL, "%s: unknown output type %d", who, out_type);
    if (M == 0) return MOE_OK;
    if (!d_a || !d_a_scale || !d_w || !d_w_scale || !d_out) return fail(MOE_EINVAL, "%s: NULL pointer", who);
    if (a_stride < K || w_stride < K || out_stride < N || ws_stride < (K + 127) / 128)
        return fail(MOE_EINVAL, "%s: a row stride is below its row", who);
    if (K % 16 || a_stride % 16 || w_stride % 16 || !on(d_a, 16) || !on(d_w, 16))
        return fail(MOE_EUNSUPPORTED, "%s: K (%d) and the strides must be multiples of 16, a and w 16-byte aligned",
                    who, K);
    if (!stride_fits(a_stride) || !stride_fits(w_stride)) return fail(MOE_EUNSUPPORTED, "%s: rows over 8 MiB", who);
    if (M > 65535 * 4) return fail(MOE_EUNSUPPORTED, "%s: M (%d) is over %d", who, M, 65535 * 4);
    if (!on(d_a_scale, 4) || !on(d_w_scale, 4) || !on(d_out, out_type == MOE_F32 ? 4 : 2))
        return fail(MOE_EINVAL, "%s: a pointer is not aligned to its type", who);
    Fp8Args a{};
    a.a = d_a, a.a_scale = d_a_scale, a.w = d_w, a.w_scale = d_w_scale, a.out = d_out;
    a.lda = a_stride, a.as_t = as_stride_m, a.as_k = as_stride_b, a.ldw = w_stride, a.ws_n = ws_stride;
    a.ldo = out_stride, a.M = M, a.N = N, a.K = K;
    a.out_f32 = out_type == MOE_F32;
    a.out_vec = out_stride % 8 == 0 && on(d_out, 16);
    return launched(launch_fp8_linear(a, static_cast<hipStream_t>(stream)), who);
}

moe_status_t moe_int4_linear(const uint16_t* d_x, int64_t x_stride, const uint8_t* d_w, int64_t w_stride,
                             const uint16_t* d_scale, int64_t scale_stride, int group, int M, int N, int K, void* d_out,
                             int out_type, int64_t out_stride, void* stream) {
    const char* who = "moe_int4_linear";
    if (M < 0 || N < 1 || K < 1) return fail(MOE_EINVAL, "%s: M (%d), N (%d), K (%d)", who, M, N, K);
    if (group != 32 && group != 64 && group != 128)
        return fail(MOE_EUNSUPPORTED, "%s: groups of %d columns (32, 64 or 128)", who, group);
    if (K % group) return fail(MOE_EINVAL, "%s: K (%d) is not a multiple of the group (%d)", who, K, group);
    if (!type_ok(out_type)) return fail(MOE_EINVAL, "%s: unknown output type %d", who, out_type);
    if (M == 0) return MOE_OK;
    if (!d_x || !d_w || !d_scale || !d_out) return fail(MOE_EINVAL, "%s: NULL pointer", who);
    if (x_stride < K || w_stride < K / 2 || scale_stride < K / group || out_stride < N)
        return fail(MOE_EINVAL, "%s: a row stride is below its row", who);
    if (x_stride % 8 || w_stride % 16 || !on(d_x, 16) || !on(d_w, 16))
        return fail(MOE_EUNSUPPORTED, "%s: the strides of x and w must be multiples of 16 bytes, both 16-byte aligned", who);
    if (!on(d_scale, 2) || !on(d_out, out_type == MOE_F32 ? 4 : 2))
        return fail(MOE_EINVAL, "%s: a pointer is not aligned to its type", who);
    if (!stride_fits(x_stride * 2) || !stride_fits(w_stride) || !stride_fits(scale_stride * 2))
        return fail(MOE_EUNSUPPORTED, "%s: rows over 8 MiB apart", who);
    // grids count lanes in 32 bits
    if (M > 1 << 26 || N > 1 << 26 || (int64_t)M * N > (int64_t)1 << 36)
        return fail(MOE_EUNSUPPORTED, "%s: M (%d) or N (%d) over 2^26, or M x N over 2^36", who, M, N);
    Int4Args a{};
    a.x = d_x, a.w = d_w, a.scale = d_scale, a.out = d_out;
    a.ldx = x_stride, a.ldw = w_stride, a.lds = scale_stride, a.ldo = out_stride;
    a.M = M, a.N = N, a.K = K, a.group = group;
    a.out_f32 = out_type == MOE_F32;
    return launched(launch_int4_linear(a, static_cast<hipStream_t>(stream)), who);
}

moe_status_t moe_head_linear(const uint16_t* d_x, int64_t x_stride_t, int64_t x_stride_h, const uint16_t* d_w, int T,
                             int heads, int K, int N, uint16_t* d_out, int64_t out_stride_t, int64_t out_stride_h,
                             void* stream) {
    const char* who = "moe_head_linear";
    if (T < 0 || heads < 1 || K < 1 || N < 1)
        return fail(MOE_EINVAL, "%s: T (%d), heads (%d), K (%d), N (%d)", who, T, heads, K, N);
    if (T == 0) return MOE_OK;
    if (!d_x || !d_w || !d_out) return fail(MOE_EINVAL, "%s: NULL pointer", who);
    if (K % 8 || N % 4 || x_stride_t % 8 || x_stride_h % 8 || out_stride_t % 4 || out_stride_h % 4 || !on(d_x, 16) ||
        !on(d_w, 16) || !on(d_out, 8))
        return fail(MOE_EUNSUPPORTED, "%s: K and the x strides must be multiples of 8, N and the out strides of 4, "
                    "x and w 16-byte aligned, out 8-byte", who);
    if (heads > 65535 || T > 65535 * 16) return fail(MOE_EUNSUPPORTED, "%s: too many heads or tokens", who);
    HeadArgs a{};
    a.x = d_x, a.w = d_w, a.out = d_out;
    a.x_stride_t = x_stride_t, a.x_stride_h = x_stride_h, a.o_stride_t = out_stride_t, a.o_stride_h = out_stride_h;
    a.T = T, a.heads = heads, a.K = K, a.N = N;
    a.out_vec = N % 8 == 0 && out_stride_t % 8 == 0 && out_stride_h % 8 == 0 && on(d_out, 16);
    return launched(launch_head_linear(a, static_cast<hipStream_t>(stream)), who);
}

moe_status_t moe_latent_append(const uint16_t* d_kv, int64_t kv_stride, const void* d_weight, int weight_type,
                               float eps, int rank, int rope, const float* d_table, int n_positions,
                               const int32_t* d_positions, const int64_t* d_slots, int T, uint16_t* d_cache,
                               int64_t n_slots, const uint16_t* d_q_rope, int heads, int64_t q_stride_t,
                               int64_t q_stride_h, uint16_t* d_q_out, int64_t qo_stride_t, int64_t qo_stride_h,
                               uint8_t* d_lat_q, int64_t lat_stride, float* d_lat_scale, int64_t ls_stride_t,
                               int64_t ls_stride_g, uint16_t* d_rows, int64_t rows_stride, void* stream) {
    return append("moe_latent_append", nullptr, nullptr, d_kv, kv_stride, d_weight, weight_type, eps, rank, rope, d_table,
                  n_positions, d_positions, d_slots, T, d_cache, n_slots, d_q_rope, heads, q_stride_t, q_stride_h, d_q_out,
                  qo_stride_t, qo_stride_h, d_lat_q, lat_stride, d_lat_scale, ls_stride_t, ls_stride_g, d_rows, rows_stride,
                  stream);
}

moe_status_t moe_latent_append_fp8(const uint16_t* d_kv, int64_t kv_stride, const void* d_weight, int weight_type,
                                   float eps, int rank, int rope, const float* d_table, int n_positions,
                                   const int32_t* d_positions, const int64_t* d_slots, int T, uint8_t* d_cache,
                                   float* d_cache_scale, int64_t n_slots, const uint16_t* d_q_rope, int heads,
                                   int64_t q_stride_t, int64_t q_stride_h, uint16_t* d_q_out, int64_t qo_stride_t,
                                   int64_t qo_stride_h, uint16_t* d_rows, int64_t rows_stride, void* stream) {
    const char* who = "moe_latent_append_fp8";
    if (T > 0 && (!d_cache || !d_cache_scale)) return fail(MOE_EINVAL, "%s: NULL cache or scales", who);
    return append(who, d_cache, d_cache_scale, d_kv, kv_stride, d_weight, weight_type, eps, rank, rope, d_table, n_positions,
                  d_positions, d_slots, T, nullptr, n_slots, d_q_rope, heads, q_stride_t, q_stride_h, d_q_out, qo_stride_t,
                  qo_stride_h, nullptr, 0, nullptr, 0, 0, d_rows, rows_stride, stream);
}

moe_status_t moe_latent_read_fp8(const uint8_t* d_cache, const float* d_cache_scale, int64_t n_slots, int rank, int rope,
                                 const int64_t* d_slots, int T, uint16_t* d_out, int64_t out_stride, void* stream) {
    const char* who = "moe_latent_read_fp8";
    if (T < 0 || rank < 1 || rope < 1 || n_slots < 0)
        return fail(MOE_EINVAL, "%s: T (%d), rank (%d), rope (%d) or slots", who, T, rank, rope);
    if (T == 0) return MOE_OK;
    if (!d_slots || !d_out || (n_slots > 0 && (!d_cache || !d_cache_scale))) return fail(MOE_EINVAL, "%s: NULL pointer", who);
    if (out_stride < rank + rope) return fail(MOE_EINVAL, "%s: a row stride is below its row", who);
    if (rank % 16 || rope % 8 || out_stride % 8 || !on(d_cache, 16) || !on(d_out, 16))
        return fail(MOE_EUNSUPPORTED, "%s: rank must be a multiple of 16, rope and the stride of 8, pointers 16-byte aligned",
                    who);
    if (!on(d_cache_scale, 4) || !on(d_slots, 8)) return fail(MOE_EINVAL, "%s: a pointer is not aligned to its type", who);
    // grids count lanes in 32 bits, 16 bytes of a row each
    if (rank > kAppendMaxRank || (int64_t)T * ((rank + 2 * (int64_t)rope) / 16) >= (int64_t)1 << 32)
        return fail(MOE_EUNSUPPORTED, "%s: rank over %d, or too many rows", who, kAppendMaxRank);
    ReadArgs a{};
    a.cache = d_cache, a.scale = d_cache_scale, a.slots = d_slots, a.out = d_out;
    a.n_slots = n_slots, a.o_stride = out_stride, a.T = T, a.rank = rank, a.rope = rope;
    return launched(launch_latent_read(a, static_cast<hipStream_t>(stream)), who);
}

size_t moe_latent_attention_workspace(int B, int max_q, int heads, int rank, int max_len) {
    if (B < 1 || max_q < 1 || heads < 1 || rank < 1 || max_len < 0) return 0;
    return latent_workspace(B, max_q, heads, rank, max_len);
}

moe_status_t moe_latent_attention(const uint16_t* d_q, int64_t q_stride_t, int64_t q_stride_h, int T, int heads,
                                  int rank, int rope, const uint16_t* d_cache, int n_pages, int page_size,
                                  int64_t page_stride, const int32_t* d_pages, int64_t pages_stride,
                                  int pages_per_seq, const int32_t* d_lens, int B, const int32_t* d_cu_q, int max_q,
                                  int max_len, const int64_t* d_tree, float scale, uint16_t* d_out,
                                  int64_t out_stride_t, int64_t out_stride_h, void* d_ws, size_t ws_bytes,
                                  void* stream) {
    return attend("moe_latent_attention", nullptr, PrefixArgs{}, d_q, q_stride_t, q_stride_h, T, heads, rank, rope, d_cache,
                  n_pages, page_size, page_stride, d_pages, pages_stride, pages_per_seq, d_lens, B, d_cu_q, max_q, max_len,
                  d_tree, scale, d_out, out_stride_t, out_stride_h, d_ws, ws_bytes, stream);
}

size_t moe_latent_attention_shared_workspace(int B, int T, int max_q, int heads, int rank, int max_len, int n_prefixes,
                                             int max_prefix_len) {
    if (n_prefixes < 1) return moe_latent_attention_workspace(B, max_q, heads, rank, max_len);
    if (B < 1 || T < 1 || max_q < 1 || heads < 1 || rank < 1 || max_len < 0 || max_prefix_len < 0) return 0;
    return latent_shared_workspace(B, T, max_q, heads, rank, max_len, n_prefixes, max_prefix_len);
}

moe_status_t moe_latent_attention_shared(const uint16_t* d_q, int64_t q_stride_t, int64_t q_stride_h, int T, int heads,
                                         int rank, int rope, const void* d_cache, const float* d_cache_scale,
                                         int n_pages, int page_size, int64_t page_stride, const int32_t* d_pages,
                                         int64_t pages_stride, int pages_per_seq, const int32_t* d_lens, int B,
                                         const int32_t* d_cu_q, int max_q, int max_len, const int64_t* d_tree,
                                         const int32_t* d_prefix_pages, int64_t prefix_pages_stride,
                                         int pages_per_prefix, const int32_t* d_prefix_lens, const int32_t* d_groups,
                                         int n_prefixes, int max_prefix_len, float scale, uint16_t* d_out,
                                         int64_t out_stride_t, int64_t out_stride_h, void* d_ws, size_t ws_bytes,
                                         void* stream) {
    const char* who = "moe_latent_attention_shared";
    if (n_prefixes < 0 || pages_per_prefix < 0 || max_prefix_len < 0)
        return fail(MOE_EINVAL, "%s: a size of the prefixes is negative", who);
    PrefixArgs p{};
    if (n_prefixes > 0) {
        if (T > 0 && (!d_prefix_lens || (pages_per_prefix > 0 && !d_prefix_pages) || (n_prefixes > 1 && !d_groups)))
            return fail(MOE_EINVAL, "%s: NULL pointer for %d prefixes", who, n_prefixes);
        if (prefix_pages_stride < pages_per_prefix) return fail(MOE_EINVAL, "%s: a stride is below its row", who);
        if (n_prefixes > 65535) return fail(MOE_EUNSUPPORTED, "%s: over 65535 prefixes", who);
        p.pages = d_prefix_pages, p.lens = d_prefix_lens, p.groups = d_groups, p.pages_stride = prefix_pages_stride;
        p.pages_per_seq = pages_per_prefix, p.count = n_prefixes, p.max_len = max_prefix_len;
    }
    return attend(who, d_cache_scale, p, d_q, q_stride_t, q_stride_h, T, heads, rank, rope, d_cache, n_pages, page_size,
                  page_stride, d_pages, pages_stride, pages_per_seq, d_lens, B, d_cu_q, max_q, max_len, d_tree, scale, d_out,
                  out_stride_t, out_stride_h, d_ws, ws_bytes, stream);
}

moe_status_t moe_prompt_attention(const uint16_t* d_q, int64_t q_stride_t, int64_t q_stride_h, const uint16_t* d_k,
                                  int64_t k_stride_t, int64_t k_stride_h, const uint16_t* d_k_rope,
                                  int64_t kr_stride_t, const uint16_t* d_v, int64_t v_stride_t, int64_t v_stride_h,
                                  int Tq, int Tk, int heads, int nope, int rope, int vdim, const int32_t* d_cu_q,
                                  const int32_t* d_cu_k, int B, int max_q, int causal, float scale, uint16_t* d_out,
                                  int64_t out_stride_t, int64_t out_stride_h, void* stream) {
    const char* who = "moe_prompt_attention";
    if (Tq < 0 || Tk < 0 || B < 0 || heads < 1 || max_q < 0)
        return fail(MOE_EINVAL, "%s: a size is negative (or heads below 1)", who);
    if (!(scale > 0.0f) || !std::isfinite(scale)) return fail(MOE_EINVAL, "%s: scale must be positive", who);
    if (!prompt_shape_supported(nope, rope, vdim))
        return fail(MOE_EUNSUPPORTED, "%s: no kernel for widths %d + %d and %d", who, nope, rope, vdim);
    if (Tq == 0) return MOE_OK;
    if (B < 1 || max_q < 1) return fail(MOE_EINVAL, "%s: queries without a sequence", who);
    if (!d_q || !d_out || !d_cu_q || !d_cu_k || (Tk > 0 && (!d_k || !d_k_rope || !d_v)))
        return fail(MOE_EINVAL, "%s: NULL pointer", who);
    if (q_stride_t % 8 || q_stride_h % 8 || k_stride_t % 8 || k_stride_h % 8 || kr_stride_t % 8 || v_stride_t % 8 ||
        v_stride_h % 8 || out_stride_t % 4 || out_stride_h % 4 || !on(d_q, 16) || !on(d_k, 16) || !on(d_k_rope, 16) ||
        !on(d_v, 16) || !on(d_out, 8))
        return fail(MOE_EUNSUPPORTED, "%s: strides must be multiples of 8 (out: 4), pointers 16-byte aligned (out: "
                    "8-byte)", who);
    if (!stride_fits(k_stride_t * 2) || !stride_fits(kr_stride_t * 2) || !stride_fits(v_stride_t * 2))
        return fail(MOE_EUNSUPPORTED, "%s: rows over 8 MiB apart, or a negative row stride", who);
    if (!on(d_cu_q, 4) || !on(d_cu_k, 4)) return fail(MOE_EINVAL, "%s: a pointer is not aligned to its type", who);
    if (B > 65535 || max_q > 65535 * 128) return fail(MOE_EUNSUPPORTED, "%s: too many sequences or queries", who);
    PromptArgs a{};
    a.q = d_q, a.k = d_k, a.k_rope = d_k_rope, a.v = d_v, a.cu_q = d_cu_q, a.cu_k = d_cu_k, a.out = d_out;
    a.q_stride_t = q_stride_t, a.q_stride_h = q_stride_h, a.k_stride_t = k_stride_t, a.k_stride_h = k_stride_h;
    a.kr_stride_t = kr_stride_t, a.v_stride_t = v_stride_t, a.v_stride_h = v_stride_h;
    a.o_stride_t = out_stride_t, a.o_stride_h = out_stride_h;
    a.Tq = Tq, a.Tk = Tk, a.B = B, a.heads = heads, a.nope = nope, a.rope = rope, a.vdim = vdim, a.max_q = max_q;
    a.scale = scale, a.causal = causal != 0;
    return launched(launch_prompt_attention(a, static_cast<hipStream_t>(stream)), who);
}

}  // extern "C"
