// Attention over a paged cache with one latent vector per token, the heads
// absorbed into the queries: per sequence the rows are (token, head) pairs,
// every row reads the same cache rows of RANK + 64 values as keys and their
// first RANK values as values.
//
//   o[row] = sum_j softmax_j(scale q[row] . c_j) c_j[:RANK]
//
// A new token sees the context and, among the new tokens, itself and the
// earlier ones, or those of its bit mask (a tree of drafted tokens).
//
// One pass with the running maximum and sum.  At rank 512 and 64 heads a
// cache row of 1152 bytes carries 64 x 2176 operations, 121 per byte, so one
// token per sequence is bound by reading the cache and several tokens by the
// matrix cores.  A tile of 64 cache rows is loaded asynchronously one ahead
// into the other of two LDS buffers and serves as keys (row reads) and as
// values (transposed reads).  Two waves share 32 rows: each computes the
// scores of its half of the tile's keys and the sums of its half of the
// columns, so a wave holds 144 registers of queries and 128 of sums (rows
// whole in one wave would need 400, more than the compiler can place), and
// hands the other wave its exponentials, rounded to bf16, through LDS: the
// two layouts agree lane by lane, 32 bytes each.  A workgroup is one or two
// such pairs.
//
// The tiles of all sequences and row blocks form one list that is cut into
// equal runs, one per workgroup (lengths are only known on the device, and
// ragged batches would leave compute units idle).  A run that does not hold
// the whole of a (sequence, row block) leaves fp32 sums, maximum and total in
// the workspace, and a second launch joins them in run order.
#include "moe_block.h"
#include "moe_block_device.h"

namespace moe {
namespace {

constexpr int kTile = 64;          // cache rows per tile
constexpr int kMaxRuns = 256;      // one workgroup per CU
constexpr int kMinRun = 2;         // tiles a run is worth starting for
constexpr int kRopeWidth = 64;

// How one call is cut up (the same arithmetic in both launches).
__device__ __forceinline__ int seq_len(const LatentArgs& a, int b) {
    const int n = a.lens[b];
    const long most = (long)a.pages_per_seq * a.page_size;
    return n < 0 ? 0 : (n > most ? (int)most : n);
}
__device__ __forceinline__ void seq_tokens(const LatentArgs& a, int b, int& first, int& count) {
    if (a.cu_q) {
        const int u = a.cu_q[b], v = a.cu_q[b + 1];
        first = u < 0 ? 0 : (u > a.T ? a.T : u);
        count = (v > a.T ? a.T : v) - first;
        if (count < 0) count = 0;
    } else {
        count = a.T / a.B;
        first = b * count;
    }
}
__device__ __forceinline__ int seq_tiles(const LatentArgs& a, int b) {
    const int n = (seq_len(a, b) + kTile - 1) / kTile;
    return n > 1 ? n : 1;  // an empty sequence still writes its zeros
}
template <int ROWS>
__device__ __forceinline__ int seq_blocks(const LatentArgs& a, int b) {
    int first, count;
    seq_tokens(a, b, first, count);
    return (count * a.heads + ROWS - 1) / ROWS;
}

__device__ __forceinline__ int wave_sum_int(int v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}
// Inclusive sum over the lanes up to this one.
__device__ __forceinline__ int wave_scan_int(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v += u;
    }
    return v;
}

// Tiles of the whole call (each wave by itself).
template <int ROWS>
__device__ __forceinline__ int total_tiles(const LatentArgs& a, int lane) {
    int n = 0;
    for (int b = lane; b < a.B; b += 64) n += seq_tiles(a, b) * seq_blocks<ROWS>(a, b);
    return __builtin_amdgcn_readfirstlane(wave_sum_int(n));
}

// The sequence that holds tile `at` of the list (tiles of a sequence: its row
// blocks one after another), and the tile its part starts with.
template <int ROWS>
__device__ __forceinline__ void find_tile(const LatentArgs& a, int at, int lane, int& seq, int& start) {
    int before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const int b = b0 + lane;
        const int mine = b < a.B ? seq_tiles(a, b) * seq_blocks<ROWS>(a, b) : 0;
        const int upto = wave_scan_int(mine, lane) + before;
        const unsigned long long hit = __ballot(b < a.B && upto > at);
        if (hit) {
            const int w = __builtin_ctzll(hit);
            seq = b0 + w;
            start = __builtin_amdgcn_readlane(upto - mine, w);
            return;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    seq = a.B;
    start = before;
}

__device__ __forceinline__ int run_count(int total, int most) {
    const int n = (total + kMinRun - 1) / kMinRun;
    return n < most ? n : most;
}
__device__ __forceinline__ int run_start(int total, int runs, int g) { return (int)((long)total * g / runs); }

// Partial sums of one run: [2 per run][ROWS][RANK] fp32, then (maximum, total) pairs.
template <int ROWS, int RANK>
__device__ __forceinline__ float* part_sums(const LatentArgs& a, int slot) {
    return reinterpret_cast<float*>(a.ws) + (size_t)slot * ROWS * (RANK + 2);
}

// Place of chunk c (16 bytes) of the latent of row r in its LDS row of
// RANK x 2 bytes: the low four bits of c are mixed with the row so that both
// an operand read of 16 rows (same chunk) and a transposed read of four rows
// by four chunks cover all banks.
__device__ __forceinline__ int place_mix(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }

// The n lowest bits (none below 0, all from 64 up).
__device__ __forceinline__ unsigned long long low_bits(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

template <int RANK, int RG>
__global__ void __launch_bounds__(RG * 128, 1) latent_attention_kernel(LatentArgs a) {
    constexpr int kWaves = RG * 2, ROWS = RG * 32;
    constexpr int kLat = RANK / 16, kRope = kRopeWidth / 16, kOut = RANK / 64, WIDTH = RANK + kRopeWidth;
    constexpr int kLatBytes = kTile * RANK * 2, kTileBytes = kLatBytes + kTile * kRopeWidth * 2;
    constexpr int kRowsPerLoad = 1024 / (RANK * 2);  // cache rows per asynchronous load
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kTileBytes];
    __shared__ u32x4 shared_p[kWaves][2][64];   // exponentials of a wave's half of the keys
    __shared__ float shared_top[kWaves][32];    // largest score of its rows in this tile (at the end: totals)
    __shared__ int shared_raise[2][kWaves];     // a row's maximum has to move (by tile parity)
    const int lane = threadIdx.x & 63, wave = wave_in_block(), half = lane >> 5, col = lane & 31;
    const int rg = wave >> 1, side = wave & 1, other = wave ^ 1;
    const int total = total_tiles<ROWS>(a, lane), runs = run_count(total, gridDim.x);
    const int run = blockIdx.x;
    if (run >= runs) return;
    const int run_end = run_start(total, runs, run + 1);
    int at = run_start(total, runs, run);
    if (at >= run_end) return;
    int seq, seq_at;
    find_tile<ROWS>(a, at, lane, seq, seq_at);

    const unsigned lds0 = lds_address(lds);
    const float c = a.scale * 1.44269504088896340736f;
    const unsigned page_magic = 0xFFFFFFFFu / (unsigned)a.page_size;

    // This lane's places in a tile: keys (row reads, 16 bytes; the low bits of
    // the chunk are mixed with the row, the rest is an immediate offset) and
    // values (transposed reads of four keys, 8 bytes).
    unsigned key_at[8], rope_at[kRope], value_lo[4], value_hi[4];
    {
        const int r = side * 32 + col;
#pragma unroll
        for (int k = 0; k < 8; ++k) key_at[k] = r * RANK * 2 + ((k * 2 + half) ^ place_mix(r)) * 16;
#pragma unroll
        for (int k = 0; k < kRope; ++k)
            rope_at[k] = kLatBytes + r * kRopeWidth * 2 + (((k * 2 + half) ^ (r >> 1)) & 7) * 16;
        const int vr = half * 4 + ((lane & 15) >> 2);
        const int chunk = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1), sub = (lane & 1) * 8 + side * RANK;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            value_lo[k] = vr * RANK * 2 + ((k * 4 + chunk) ^ place_mix(vr)) * 16 + sub;
            value_hi[k] = (vr + 8) * RANK * 2 + ((k * 4 + chunk) ^ place_mix(vr + 8)) * 16 + sub;
        }
    }

    while (at < run_end) {
        int first, count;
        seq_tokens(a, seq, first, count);
        const int len = seq_len(a, seq), tiles = seq_tiles(a, seq), blocks = seq_blocks<ROWS>(a, seq);
        if (at >= seq_at + tiles * blocks) {
            seq_at += tiles * blocks;
            ++seq;
            continue;
        }
        const int block = (at - seq_at) / tiles, t_first = (at - seq_at) % tiles;
        const int t_last = tiles - t_first < run_end - at ? tiles : t_first + run_end - at;
        const int context = len - count;  // keys before the first new token
        const int row = block * ROWS + rg * 32 + col;
        const bool row_ok = row < count * a.heads;
        const int token = row_ok ? row / a.heads : 0, head = row_ok ? row % a.heads : 0;
        const long long mask = a.tree && row_ok ? a.tree[first + token] : 0;
        bf16x8 qf[kLat + kRope];
        {
            const uint16_t* p = a.q + (first + token) * a.q_stride_t + head * a.q_stride_h + half * 8;
#pragma unroll
            for (int k = 0; k < kLat + kRope; ++k)
                qf[k] = __builtin_bit_cast(bf16x8, *as_global<u32x4>(p + k * 16));
        }
        // Page and place of cache row t * 64 + lane (-1 past the end).
        const int32_t* my_pages = a.pages + seq * a.pages_stride;
        auto page_of = [&](int t, int& off) {
            const int pos = t * kTile + lane;
            int p = (int)__umulhi((unsigned)pos, page_magic);
            off = pos - p * a.page_size;
            if (off >= a.page_size) {
                off -= a.page_size;
                ++p;
            }
            return pos < len ? as_global<int32_t>(my_pages)[p] : -1;
        };
        // Its address; a row past the end or on a page that is not in the
        // pool reads as zero and is masked.
        auto address = [&](int page, int off) {
            const uint16_t* p = a.cache + (long)page * a.cache_page_stride + (long)off * WIDTH;
            return (unsigned long long)((unsigned)page < (unsigned)a.n_pages ? static_cast<const void*>(p) : kZeros);
        };
        auto issue = [&](int buf, unsigned long long addr) {
            const unsigned dst = lds0 + buf * kTileBytes;
            int chunk = lane;
            asm volatile("" : "+v"(chunk));  // the mixed places are not worth a register each across the loop
#pragma unroll
            for (int i = 0; i < kTile / kRowsPerLoad / kWaves; ++i) {
                const int r0 = (i * kWaves + wave) * kRowsPerLoad;
                if constexpr (kRowsPerLoad == 1) {
                    const unsigned lo = __builtin_amdgcn_readlane((unsigned)addr, r0),
                                   hi = __builtin_amdgcn_readlane((unsigned)(addr >> 32), r0);
                    load_to_lds16((const void*)((unsigned long long)hi << 32 | lo),
                                  (unsigned)(chunk ^ place_mix(r0)) * 16, dst + r0 * RANK * 2);
                } else {
                    const int r = r0 + chunk / (RANK / 8);
                    const unsigned long long p = __shfl(addr, r);
                    load_to_lds16((const uint8_t*)p + ((chunk % (RANK / 8)) ^ place_mix(r)) * 16, dst + r0 * RANK * 2);
                }
            }
#pragma unroll
            for (int i = 0; i < kTile / 8 / kWaves; ++i) {
                const int r0 = (i * kWaves + wave) * 8, r = r0 + (chunk >> 3);
                const unsigned long long p = __shfl(addr, r);
                load_to_lds16((const uint8_t*)p + RANK * 2 + (((chunk & 7) ^ (r >> 1)) & 7) * 16,
                              dst + kLatBytes + r0 * kRopeWidth * 2);
            }
        };

        float m = kNoMax, l = 0.0f;
        f32x16 o[kOut] = {};
        int off, page = page_of(t_first, off);
        unsigned long long valid = __ballot((unsigned)page < (unsigned)a.n_pages);
        issue(0, address(page, off));
        page = page_of(t_first + 1, off);
        for (int t = t_first; t < t_last; ++t) {
            const int buf = (t - t_first) & 1;
            wait_vmem<0>();
            asm volatile("" : "+v"(page));  // the next tile's pages have landed: no later wait covers its loads
            lds_barrier();                  // tile t is in LDS, and every wave is done with the other buffer
            const unsigned long long now = valid;
            if (t + 1 < t_last) {
                valid = __ballot((unsigned)page < (unsigned)a.n_pages);
                const unsigned long long next = address(page, off);
                page = page_of(t + 2, off);
                issue(buf ^ 1, next);
            }
            const unsigned tile = lds0 + buf * kTileBytes;
            f32x16 s = {};
            {
                // operands are read kAhead instructions before their use; the
                // scheduling barriers keep the compiler from reading them all
                // at once
                constexpr int kAhead = 6;
                bf16x8 x[kAhead];
                auto key_chunk = [&](int k) {
                    return lds_chunk(k < kLat ? key_at[k & 7] + tile + (k >> 3) * 256 : rope_at[k - kLat] + tile);
                };
#pragma unroll
                for (int k = 0; k < kAhead; ++k) x[k] = key_chunk(k);
#pragma unroll
                for (int k = 0; k < kLat + kRope; ++k) {
                    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[k % kAhead], qf[k], s, 0, 0, 0);
                    if (k + kAhead < kLat + kRope) x[k % kAhead] = key_chunk(k + kAhead);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (now != ~0ull || (t + 1) * kTile > context + (a.tree ? 0 : 1)) {
                // visible keys of this tile, a bit each; this lane's registers
                // hold keys 8 (i / 4) + 4 half + i % 4 of the wave's half
                const int before = context - t * kTile;  // place of the first new token
                unsigned long long sees;
                if (a.tree) {
                    const unsigned long long drawn = before >= 64    ? 0ull
                                                     : before >= 0   ? (unsigned long long)mask << before
                                                     : before > -64 ? (unsigned long long)mask >> -before
                                                                     : 0ull;
                    sees = low_bits(before) | drawn;
                } else {
                    sees = low_bits(before + token + 1);
                }
                sees &= now;
                const unsigned word = (unsigned)(sees >> (side * 32)) >> (4 * half);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[i] = word >> (8 * (i / 4) + i % 4) & 1 ? s[i] : -__builtin_inff();
            }
            float top = s[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
            top = half_max(top);
            const bool raise = __any((top - m) * c > kMaxSlack);
            bf16x8 p[4];  // of both waves' keys, in key order
            auto exponentials = [&]() {
                const float mc = m * c;
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float e = __builtin_amdgcn_exp2f(fmaf(s[i], c, -mc));
                    sum += e;
                    p[i / 8][i % 8] = (__bf16)e;
                }
                shared_p[wave][0][lane] = __builtin_bit_cast(u32x4, p[0]);
                shared_p[wave][1][lane] = __builtin_bit_cast(u32x4, p[1]);
                return sum;
            };
            float sum = exponentials();
            if (half == 0) shared_top[wave][col] = top;
            if (lane == 0) shared_raise[t & 1][wave] = raise;
            lds_barrier();
            int any = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) any |= shared_raise[t & 1][w];
            if (__builtin_amdgcn_readfirstlane(any)) {
                // some row's maximum moves: both waves of each pair take the
                // new one and compute their exponentials again
                const float nm = fmaxf(m, fmaxf(top, shared_top[other][col]));
                const float f = __builtin_amdgcn_exp2f((m - nm) * c);
                m = nm;
                l *= f;
#pragma unroll
                for (int k = 0; k < kOut; ++k)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[k][i] *= f;
                sum = exponentials();
                lds_barrier();
            }
            l += sum;
            {
                const bf16x8 q0 = __builtin_bit_cast(bf16x8, shared_p[other][0][lane]),
                             q1 = __builtin_bit_cast(bf16x8, shared_p[other][1][lane]);
                const bf16x8 p0 = p[0], p1 = p[1];
                p[0] = side ? q0 : p0;
                p[1] = side ? q1 : p1;
                p[2] = side ? p0 : q0;
                p[3] = side ? p1 : q1;
            }
            {
                constexpr int kAhead = 6;
                bf16x8 x[kAhead];
                auto value_chunk = [&](int j) {
                    const int k = j >> 2, v = j & 3;
                    const unsigned at_key = tile + v * 16 * RANK * 2 + (k >> 2) * 256;
                    return values_transposed(value_lo[k & 3] + at_key, value_hi[k & 3] + at_key);
                };
#pragma unroll
                for (int j = 0; j < kAhead; ++j) x[j] = value_chunk(j);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < 4 * kOut; ++j) {
                    o[j >> 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[j % kAhead], p[j & 3], o[j >> 2], 0, 0, 0);
                    if (j + kAhead < 4 * kOut) x[j % kAhead] = value_chunk(j + kAhead);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        // totals over the tile halves of both waves
        l = half_sum(l);
        __syncthreads();
        if (half == 0) shared_top[wave][col] = l;
        __syncthreads();
        l += shared_top[other][col];
        if (t_first == 0 && t_last == tiles) {
            if (row_ok) {
                // a row that sees no key gives zero
                const float inv = l != 0.0f ? 1.0f / l : 0.0f;
                uint16_t* out = a.out + (first + token) * a.o_stride_t + head * a.o_stride_h + side * (RANK / 2) + half * 4;
#pragma unroll
                for (int k = 0; k < kOut; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<u32x2*>(out + k * 32 + i * 8) =
                            u32x2{pack_bf16(o[k][i * 4] * inv, o[k][i * 4 + 1] * inv),
                                  pack_bf16(o[k][i * 4 + 2] * inv, o[k][i * 4 + 3] * inv)};
            }
        } else {
            float* part = part_sums<ROWS, RANK>(a, run * 2 + (t_first == 0));
            const int r = rg * 32 + col;
#pragma unroll
            for (int k = 0; k < kOut; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<f32x4*>(part + (long)r * RANK + side * (RANK / 2) + k * 32 + i * 8 + half * 4) =
                        f32x4{o[k][i * 4], o[k][i * 4 + 1], o[k][i * 4 + 2], o[k][i * 4 + 3]};
            if (half == 0 && side == 0) {
                part[ROWS * RANK + r * 2] = m;
                part[ROWS * RANK + r * 2 + 1] = l;
            }
        }
        at += t_last - t_first;
        __syncthreads();  // the buffers are free for the next part's first tile
    }
}

// Joins the partial sums of every (sequence, row block) that more than one
// run worked on: a wave per row, the runs in order.
template <int RANK, int ROWS>
__global__ void __launch_bounds__(256) latent_join_kernel(LatentArgs a, int most_runs) {
    constexpr int V = RANK / 64;  // columns per lane
    const int lane = threadIdx.x & 63;
    const int seq = blockIdx.y, row = blockIdx.x * 4 + wave_in_block();
    int first, count;
    seq_tokens(a, seq, first, count);
    if (row >= count * a.heads) return;
    const int total = total_tiles<ROWS>(a, lane), runs = run_count(total, most_runs);
    int before = 0;
    for (int b = lane; b < seq; b += 64) before += seq_tiles(a, b) * seq_blocks<ROWS>(a, b);
    before = __builtin_amdgcn_readfirstlane(wave_sum_int(before));
    const int tiles = seq_tiles(a, seq), block = row / ROWS, r = row % ROWS;
    const int u0 = before + block * tiles, u1 = u0 + tiles;
    // runs that hold the first and the last tile of the block
    auto run_of = [&](int tile) {
        int g = (int)((long)tile * runs / total);
        while (g + 1 < runs && run_start(total, runs, g + 1) <= tile) ++g;
        while (g > 0 && run_start(total, runs, g) > tile) --g;
        return g;
    };
    const int g0 = run_of(u0), g1 = run_of(u1 - 1);
    if (g0 == g1) return;  // one run held it all and wrote the result
    const float c = a.scale * 1.44269504088896340736f;
    float m = kNoMax, l = 0.0f, o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.0f;
    for (int g = g0; g <= g1; ++g) {
        const float* part = part_sums<ROWS, RANK>(a, g * 2 + (run_start(total, runs, g) <= u0));
        const float pm = part[ROWS * RANK + r * 2], pl = part[ROWS * RANK + r * 2 + 1];
        const float nm = fmaxf(m, pm), f = __builtin_amdgcn_exp2f((m - nm) * c), pf = __builtin_amdgcn_exp2f((pm - nm) * c);
        m = nm;
        l = l * f + pl * pf;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = o[i] * f + part[(long)r * RANK + lane * V + i] * pf;
    }
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    uint16_t* out = a.out + (long)(first + row / a.heads) * a.o_stride_t + (row % a.heads) * a.o_stride_h + lane * V;
#pragma unroll
    for (int i = 0; i < V; i += 2) *reinterpret_cast<unsigned*>(out + i) = pack_bf16(o[i] * inv, o[i + 1] * inv);
}

// Most runs a call of these bounds can be cut into.
int most_runs(int B, int max_q, int heads, int max_len, int rows) {
    const long blocks = ((long)max_q * heads + rows - 1) / rows;
    const long tiles = max_len > kTile ? (max_len + kTile - 1) / kTile : 1;
    const long runs = (B * blocks * tiles + kMinRun - 1) / kMinRun;
    return (int)(runs < kMaxRuns ? runs : kMaxRuns);
}
int block_rows(int max_q, int heads) { return (long)max_q * heads > 32 ? 64 : 32; }

template <int RANK, int RG>
void launch_rows(const LatentArgs& a, hipStream_t s) {
    const int runs = most_runs(a.B, a.max_q, a.heads, a.max_len, RG * 32);
    hipLaunchKernelGGL((latent_attention_kernel<RANK, RG>), dim3(runs), dim3(RG * 128), 0, s, a);
    if (runs > 1) {
        const int rows = a.max_q * a.heads;
        hipLaunchKernelGGL((latent_join_kernel<RANK, RG * 32>), dim3((rows + 3) / 4, a.B), dim3(256), 0, s, a, runs);
    }
}
template <int RANK>
void launch_rank(const LatentArgs& a, hipStream_t s) {
    if (block_rows(a.max_q, a.heads) == 64)
        launch_rows<RANK, 2>(a, s);
    else
        launch_rows<RANK, 1>(a, s);
}

}  // namespace

bool latent_shape_supported(int rank, int rope) { return rope == kRopeWidth && (rank == 512 || rank == 256); }

size_t latent_workspace(int B, int max_q, int heads, int rank, int max_len) {
    const int rows = block_rows(max_q, heads);
    return (size_t)most_runs(B, max_q, heads, max_len, rows) * 2 * rows * (rank + 2) * sizeof(float);
}

hipError_t launch_latent_attention(const LatentArgs& a, hipStream_t s) {
    if (a.rank == 512)
        launch_rank<512>(a, s);
    else
        launch_rank<256>(a, s);
    return hipGetLastError();
}

}  // namespace moe
