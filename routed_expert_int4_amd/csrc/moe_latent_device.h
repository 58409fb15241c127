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
// values (transposed reads).  Four waves share 32 rows: each computes partial
// scores of half of the tile's keys over half of the inner dimension, takes
// the other half's from its neighbour, and then has the exponentials of a
// quarter of the keys, rounded to bf16, for all four, each of which sums a
// quarter of the columns.  A wave thus holds 72 registers of queries and 64 of
// sums, and two waves fit a SIMD (rows whole in one wave would need 400).  All
// exchanges go through LDS, which is full: 144 KB of tiles, 16 KB of slots.  A
// workgroup is one or two such fours, 32 or 64 rows.
//
// Measured, rank 512, 64 heads: 32 sequences of 16384 rows, one token each,
// 132 us (4.6 TB/s), four tokens 357 us (0.82 PFLOP/s); trees of four tokens
// over ragged rows, 10400 on average, 208 us.  One sequence, one token: 1013 rows
// 17.5 us, 16384 rows 32 us, 65536 rows 39 us.  Rank 256: 80, 240, and
// 16, 27 and 30 us.  A tile takes a workgroup 2.6 us, of which matrix
// instructions are 1.0; the loads stall the waves that issue them for about 0.5
// (issued all at once: 4 % slower; some of them after the scores, so that they
// arrive late: 3 to 9 %).
//
// Row blocks of one sequence read the same cache rows, so GS workgroups work
// as a group: on the same die (one L2), over the same tiles, each on its own
// row block; a sequence of more blocks takes several passes.  The tiles of all
// (sequence, pass) units form one list that is cut into equal runs, one per
// group (lengths are only known on the device, and ragged batches would leave
// compute units idle).  A run that does not hold the whole of a unit leaves
// fp32 sums, maximum and total in the workspace, and a second launch joins
// them in run order.
#pragma once

#include "moe_block.h"
#include "moe_block_device.h"

namespace moe {
namespace {

constexpr int kTile = 64;          // cache rows per tile
constexpr int kMaxGroup = 8;       // workgroups of a group
constexpr int kMaxWorkgroups = 256;  // one per CU
constexpr int kRopeWidth = 64;
// What a load of eight rows of 8 bits reads where there is no page.
__device__ __attribute__((aligned(16))) const uint8_t kNoPage[8 * (512 + 2 * kRopeWidth)] = {};

__device__ __forceinline__ void seq_tokens(const LatentArgs& a, int b, int& first, int& count) {
    auto within = [](int v, int most) { return v < 0 ? 0 : (v > most ? most : v); };
    if (a.prefixes && !a.groups) {  // one prefix for all
        first = 0;
        count = a.T;
    } else if (a.cu_q || a.prefixes) {
        int s = b, e = b + 1;
        if (a.prefixes) {
            s = a.groups[b];
            e = a.groups[b + 1];
            s = within(s, a.seqs);
            e = within(e, a.seqs);
        }
        int u = s * a.per_seq, v = e * a.per_seq;
        if (a.cu_q) {
            u = a.cu_q[s];
            v = a.cu_q[e];
        }
        first = within(u, a.T);
        count = (v > a.T ? a.T : v) - first;
        if (count < 0) count = 0;
    } else {
        count = a.per_seq;
        first = b * count;
    }
}
// One sequence's part of the list: tiles of the cache, row blocks, passes.
struct SeqShape {
    int len, first, count, tiles, blocks, passes;
};
template <int ROWS>
__device__ __forceinline__ SeqShape seq_shape(const LatentArgs& a, int b) {
    SeqShape s;
    const int n = a.lens[b];
    seq_tokens(a, b, s.first, s.count);
    const long most = (long)a.pages_per_seq * a.page_size;
    s.len = n < 0 ? 0 : (n > most ? (int)most : n);
    s.tiles = s.len > kTile ? (s.len + kTile - 1) / kTile : 1;  // an empty sequence still writes its zeros
    s.blocks = (s.count * a.heads + ROWS - 1) / ROWS;
    s.passes = (s.blocks + a.group - 1) / a.group;
    return s;
}

// Inclusive sum over the lanes up to this one.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ int scan_step(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROW_MASK, 0xF, false);
}
__device__ __forceinline__ int wave_scan_int(int v) {
    v = scan_step<0x111, 0xF>(v);  // within rows of 16: shifts by 1, 2, 4, 8
    v = scan_step<0x112, 0xF>(v);
    v = scan_step<0x114, 0xF>(v);
    v = scan_step<0x118, 0xF>(v);
    v = scan_step<0x142, 0xA>(v);  // last lane of rows 0 and 2 into rows 1 and 3
    return scan_step<0x143, 0xC>(v);  // lane 31 into the upper half
}

// The whole list: its length, the tiles before sequence `upto`, and its
// pieces, a pass over a sequence's tiles each.  The host
// has seen to it that the tiles of T tokens fit 32 bits, so bounds in device
// memory that name more than T (some of them twice) leave the list empty.
template <int ROWS>
__device__ __forceinline__ int count_tiles(const LatentArgs& a, int upto, int lane, int& before, int* units = nullptr) {
    int total = 0, tokens = 0;  // this lane's sequences', T + 1 for any number above T
    int passes = 0;
    before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const int b = b0 + lane;
        int mine = 0;
        if (b < a.B) {
            const SeqShape s = seq_shape<ROWS>(a, b);
            mine = s.tiles * s.passes;
            passes += s.passes;
            tokens = tokens + s.count > a.T ? a.T + 1 : tokens + s.count;
        }
        const int scan = wave_scan_int(mine);
        if (upto > b0) before = total + __builtin_amdgcn_readlane(scan, (upto - b0 < 64 ? upto - b0 : 64) - 1);
        total += __builtin_amdgcn_readlane(scan, 63);
    }
    // (64 lanes of up to T, below 2^26, are below 2^32)
    if ((a.cu_q || a.prefixes) && (__any(tokens > a.T) || (unsigned)__builtin_amdgcn_readlane(wave_scan_int(tokens), 63) > (unsigned)a.T))
        return 0;
    if (units) *units = __builtin_amdgcn_readlane(wave_scan_int(passes), 63);
    return total;
}

// The sequence that holds tile `at` of the list (at < its length), its part,
// and the tile that starts with.
template <int ROWS>
__device__ __forceinline__ SeqShape find_tile(const LatentArgs& a, int at, int lane, int& seq, int& start) {
    int before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const int b = b0 + lane;
        int mine = 0;
        SeqShape s{};
        if (b < a.B) {
            s = seq_shape<ROWS>(a, b);
            mine = s.tiles * s.passes;
        }
        const int upto = wave_scan_int(mine) + before;
        const unsigned long long hit = __ballot(b < a.B && upto > at);
        if (hit) {
            const int w = __builtin_ctzll(hit);
            seq = b0 + w;
            start = __builtin_amdgcn_readlane(upto - mine, w);
            auto of = [&](int v) { return __builtin_amdgcn_readlane(v, w); };
            return {of(s.len), of(s.first), of(s.count), of(s.tiles), of(s.blocks), of(s.passes)};
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    seq = a.B - 1;
    start = at;
    return seq_shape<ROWS>(a, seq);
}

// Runs the list is cut into, and where run g starts.
__device__ __forceinline__ int run_count(int total, int most) { return total < most ? total : most; }
__device__ __forceinline__ int run_start(int total, int runs, int g) {
    const int each = total / runs, more = total - each * runs;  // the first `more` runs have one tile more
    return g * each + (g < more ? g : more);
}

// Partial sums of one workgroup: [2][ROWS][RANK] fp32, then (maximum, total)
// pairs; the second half is for the unit it starts, the first for the one it
// finds begun.
template <int ROWS, int RANK>
__device__ __forceinline__ float* part_sums(const LatentArgs& a, int slot) {
    return reinterpret_cast<float*>(a.ws) + (size_t)slot * ROWS * (RANK + 2);
}

// Place of chunk c (16 bytes) of the latent of row r in its LDS row of
// RANK x 2 bytes: the low four bits of c are mixed with the row so that both
// an operand read of 16 rows (same chunk) and a transposed read of four rows
// by four chunks cover all banks.
__device__ __forceinline__ int place_mix(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }

__device__ __forceinline__ void mfma(f32x16& c, bf16x8 a, bf16x8 b) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The n lowest bits (none below 0, all from 64 up).
__device__ __forceinline__ unsigned long long low_bits(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// Operands of the product with the values: bf16 as read, or eight codes.
template <bool NARROW>
struct ValueOperand {
    typedef bf16x8 type;
};
template <>
struct ValueOperand<true> {
    typedef u32x2 type;
};
__device__ __forceinline__ bf16x8 value_operand(bf16x8 v) { return v; }
__device__ __forceinline__ bf16x8 value_operand(u32x2 v) { return __builtin_bit_cast(bf16x8, codes_to_bf16(v[0], v[1], 1.0f)); }

// Whether 16 bytes of a tile hold a value that is not finite (a code of 8 bits
// has only NaN, all seven low bits set), and the bytes without them.
__device__ __forceinline__ unsigned nan_codes(unsigned u) { return ((u & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
template <bool NARROW>
__device__ __forceinline__ bool holds_not_finite(u32x4 u) {
    if constexpr (NARROW)
        return (nan_codes(u[0]) | nan_codes(u[1]) | nan_codes(u[2]) | nan_codes(u[3])) != 0;
    else
        return not_finite(magnitudes(u));
}
template <bool NARROW>
__device__ __forceinline__ u32x4 only_finite(u32x4 u) {
    if constexpr (NARROW) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned n = nan_codes(u[i]);
            u[i] &= ~((n << 1) - (n >> 7));
        }
        return u;
    } else {
        return finite_only(u);
    }
}

// One workgroup's run of a list: run `run` of `runs`, row blocks `member`,
// member + a.group and so on.  NARROW: the cache has 8 bits.  KEEP: units that
// are whole in a run leave fp32 sums too, in `whole` by row.  `slot`: where the
// workgroup's partial sums go.
template <int RANK, int RG, bool NARROW, bool KEEP>
__device__ __forceinline__ void attend(const LatentArgs& a, int total, int runs, int run, int member, int slot, float* whole) {
    constexpr int kWaves = RG * 4, ROWS = RG * 32, kBytes = NARROW ? 1 : 2;  // of a latent value in the cache
    constexpr int kRow = RANK * kBytes / 2 + kRopeWidth;                      // two-byte units of a cache row
    // a wave's inner steps of 16 (latent, position part), its columns by 32
    constexpr int kLat = RANK / 32, kRope = kRopeWidth / 32, kSteps = kLat + kRope, kOut = RANK / 128;
    constexpr int kLatRow = RANK * kBytes, kLatBytes = kTile * kLatRow, kTileBytes = kLatBytes + kTile * kRopeWidth * 2;
    constexpr int kRowsPerLoad = 1024 / kLatRow;  // cache rows per asynchronous load
    // Tiles are loaded one ahead, those of 8 bits two ahead.
    constexpr int kBuffers = NARROW ? 3 : 2;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kBuffers * kTileBytes];
    // Slots by which the four waves of 32 rows hand over partial scores, then
    // exponentials, maxima and flags.  A wave writes its scores to its own
    // slot, reads those of wave ^ 1, and then owns what it has read.
    __shared__ u32x4 slots[kWaves][2][64];
    __shared__ float powers[kBuffers][NARROW ? kTile : 1];  // of the tiles' rows
    __shared__ __attribute__((aligned(16))) unsigned value_powers[NARROW ? kTile : 1];  // of this tile's, as the weights take them
    __shared__ int pages_ahead[2][NARROW ? kTile : 1];       // of the tile after those
    const int lane = threadIdx.x & 63, wave = wave_in_block(), half = lane >> 5, col = lane & 31;
    const int rg = wave >> 2, quarter = wave & 3, side = quarter >> 1, inner = quarter & 1, other = wave ^ 1;
    float* const my_top = reinterpret_cast<float*>(slots[other][1]);  // 32 maxima (at the end: totals)
    auto slot_of = [&](int w) { return reinterpret_cast<const float*>(slots[w ^ 1][1]); };
    const int run_end = run_start(total, runs, run + 1);
    int at = run_start(total, runs, run);
    int seq, seq_at;
    SeqShape shape = find_tile<ROWS>(a, at, lane, seq, seq_at);

    const unsigned lds0 = lds_address(lds);
    const float c = a.scale * 1.44269504088896340736f;
    const unsigned page_magic = 0xFFFFFFFFu / (unsigned)a.page_size;

    // This lane's places in a tile: keys (row reads of 16 bytes) and values
    // (transposed reads of four keys, 8 bytes; the next four keys 8 rows on).
    // Only the low four bits of a row's chunk are mixed with the row and rows
    // are whole multiples of 256 bytes, so an exclusive or and an immediate
    // offset reach every chunk from these.
    unsigned key_at, rope_at, value_at;
    {
        // (a wave takes its keys so that those it keeps are the first 16
        // instruction rows, and those its neighbour keeps the others)
        const int r = side * 32 + (col ^ inner * 16);
        if constexpr (NARROW) {
            // keys: 16 codes, two steps of the inner dimension; values: the
            // first byte of eight keys' 16 columns
            const int unit = inner * (RANK / 32);
            key_at = lds0 + r * kLatRow + (unit >> 4) * 256 + (((unit & 15) | half) ^ place_mix(r)) * 16;
            const int i = (lane & 15) >> 1, vr = half * 4 + (i & 3) + (i >> 2) * 8;
            const int column = quarter * (RANK / 64) + ((lane >> 4) & 1);
            value_at = lds0 + vr * kLatRow + (column >> 4) * 256 + ((column & 15) ^ place_mix(vr)) * 16 + (lane & 1) * 8;
        } else {
            const int vr = half * 4 + ((lane & 15) >> 2);
            key_at = lds0 + r * RANK * 2 + inner * RANK + (half ^ place_mix(r)) * 16;
            const int first = quarter * (RANK / 32);  // the wave's first chunk of a row
            const int chunk = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1) + (first & 15);
            value_at = lds0 + vr * RANK * 2 + (first >> 4) * 256 + (chunk ^ place_mix(vr)) * 16 + (lane & 1) * 8;
        }
        rope_at = lds0 + kLatBytes + r * kRopeWidth * 2 + (((half | inner * 4) ^ (r >> 1)) & 7) * 16;
    }

    while (at < run_end) {
        const int len = shape.len, first = shape.first, count = shape.count, tiles = shape.tiles;
        if (at >= seq_at + tiles * shape.passes) {
            seq_at += tiles * shape.passes;
            shape = seq_shape<ROWS>(a, ++seq);
            continue;
        }
        const int pass = (at - seq_at) / tiles, t_first = (at - seq_at) % tiles;
        const int t_last = tiles - t_first < run_end - at ? tiles : t_first + run_end - at;
        const int block = pass * a.group + member;
        if (block >= shape.blocks) {  // the last pass of this sequence has no block for this member
            at += t_last - t_first;
            continue;
        }
        const int context = a.prefixes ? len : len - count;  // keys before the first new token
        // Page and place of cache row t * 64 + lane (-1 past the end).
        const int32_t* my_pages = a.pages + seq * a.pages_stride;
        auto place_of = [&](int t, int& off) {
            const int pos = t * kTile + lane;
            int p = (int)__umulhi((unsigned)pos, page_magic);
            off = pos - p * a.page_size;
            if (off >= a.page_size) {
                off -= a.page_size;
                ++p;
            }
            return pos < len ? p : -1;
        };
        auto page_of = [&](int t, int& off) {
            const int p = place_of(t, off);
            return p >= 0 ? as_global<int32_t>(my_pages)[p] : -1;
        };
        // The loads that the others hang on come first: page numbers, then the
        // queries.
        int off, page = page_of(t_first, off), off_next;
        const int page_next = page_of(t_first + 1, off_next);
        __builtin_amdgcn_sched_barrier(0);
        const int row = block * ROWS + rg * 32 + col;
        const bool row_ok = row < count * a.heads;
        const int token = row_ok ? row / a.heads : 0, head = row_ok ? row % a.heads : 0;
        const long long mask = a.tree && row_ok ? a.tree[first + token] : 0;
        // The workgroup's queries go to LDS by lines, behind the first tile's
        // buffer, and from there to the waves' registers: straight from memory
        // every wave's loads would touch 32 lines each (decode of 1013 rows 20.4
        // us, now 17.5).  Chunk c (16 bytes) of row r lies at place c ^ (r & 15), of its
        // position part at c ^ (r / 2 & 7).
        constexpr int kQueryRow = RANK * 2, kQueryRows = 1024 / kQueryRow, kQueryLoads = ROWS / kQueryRows / kWaves;
        static_assert(ROWS * (kQueryRow + kRopeWidth * 2) <= (kBuffers - 1) * kTileBytes, "queries");
        const unsigned query0 = lds0 + kTileBytes, query_rope0 = query0 + ROWS * kQueryRow;
        {
            // lane r has the address of row r
            const int row = block * ROWS + lane, at_row = row < count * a.heads ? row : 0;
            const auto from = (unsigned long long)(a.q + (first + at_row / a.heads) * a.q_stride_t + at_row % a.heads * a.q_stride_h);
#pragma unroll
            for (int i = 0; i < kQueryLoads; ++i) {
                const int r0 = (i * kWaves + wave) * kQueryRows, r = r0 + lane / (kQueryRow / 16);
                const unsigned in_row = ((lane % (kQueryRow / 16)) ^ (r & 15)) * 16;
                if constexpr (kQueryRows == 1) {
                    const unsigned lo = __builtin_amdgcn_readlane((unsigned)from, r0),
                                   hi = __builtin_amdgcn_readlane((unsigned)(from >> 32), r0);
                    load_to_lds16_lane((unsigned long long)hi << 32 | lo, in_row, query0 + r0 * kQueryRow);
                } else {
                    load_to_lds16(reinterpret_cast<const uint8_t*>(__shfl(from, r)) + in_row, query0 + r0 * kQueryRow);
                }
            }
            const int r = wave * 8 + (lane >> 3);
            load_to_lds16(reinterpret_cast<const uint8_t*>(__shfl(from, r)) + kQueryRow + (((lane & 7) ^ (r >> 1)) & 7) * 16,
                          query_rope0 + wave * 8 * kRopeWidth * 2);
        }
        wait_vmem<0>();  // all of these, as the page numbers are waited for in any case
        // Its address; a row past the end or on a page that is not in the
        // pool reads as zero and is masked.
        auto address = [&](int page, int off) {
            const uint16_t* p = a.cache + (long)page * a.cache_page_stride + (long)off * kRow;
            return (unsigned long long)((unsigned)page < (unsigned)a.n_pages ? static_cast<const void*>(p)
                                        : NARROW                             ? kNoPage
                                                                             : kZeros);
        };
        constexpr int kLatLoads = kTile / kRowsPerLoad / kWaves, kLoads = kLatLoads + kTile / 8 / kWaves;
        // Asynchronous load i of this wave's kLoads of a tile: the cache row
        // of a lane's 16 bytes, and the load from that row's address.
        auto row_of = [&](int i, int chunk) {
            return i < kLatLoads ? (i * kWaves + wave) * kRowsPerLoad + chunk / (kLatRow / 16)
                                 : ((i - kLatLoads) * kWaves + wave) * 8 + (chunk >> 3);
        };
        auto issue_from = [&](int i, int buf, unsigned long long p, int chunk) {
            const unsigned dst = lds0 + buf * kTileBytes;
            const int r = row_of(i, chunk);
            if (i < kLatLoads)
                load_to_lds16((const uint8_t*)p + ((chunk % (kLatRow / 16)) ^ place_mix(r)) * 16,
                              dst + (i * kWaves + wave) * kRowsPerLoad * kLatRow);
            else
                load_to_lds16((const uint8_t*)p + kLatRow + (((chunk & 7) ^ (r >> 1)) & 7) * 16,
                              dst + kLatBytes + ((i - kLatLoads) * kWaves + wave) * 8 * kRopeWidth * 2);
        };
        // Rows of 8 bits in pages of a multiple of 8 rows: all of a load's rows
        // follow its first one's address, rows past the sequence's end and all,
        // and the lanes' offsets are the same for every tile.
        const bool in_page = NARROW && a.page_size % 8 == 0;
        unsigned lat_offset = 0, rope_offset = 0;
        if constexpr (NARROW) {
            const int r = row_of(0, lane), u = row_of(kLatLoads, lane);
            lat_offset = lane / (kLatRow / 16) * (kRow * 2) + ((lane % (kLatRow / 16)) ^ place_mix(r)) * 16;
            rope_offset = (lane >> 3) * (kRow * 2) + kLatRow + (((lane & 7) ^ (u >> 1)) & 7) * 16;
        }
        auto issue_rows = [&](int i, int buf, unsigned long long addr) {
            const int r0 = i < kLatLoads ? (i * kWaves + wave) * kRowsPerLoad : ((i - kLatLoads) * kWaves + wave) * 8;
            const unsigned lo = __builtin_amdgcn_readlane((unsigned)addr, r0),
                           hi = __builtin_amdgcn_readlane((unsigned)(addr >> 32), r0);
            const unsigned long long base = (unsigned long long)hi << 32 | lo;
            // (the mixed place goes by the row's low four bits)
            constexpr int kStep = kWaves * kRowsPerLoad;
            const int mixed = place_mix(wave * kRowsPerLoad + i * kStep) ^ place_mix(wave * kRowsPerLoad);
            if (i < kLatLoads)
                load_to_lds16_lane(base, lat_offset ^ mixed * 16, lds0 + buf * kTileBytes + r0 * kLatRow);
            else
                load_to_lds16_lane(base, rope_offset, lds0 + buf * kTileBytes + kLatBytes + r0 * kRopeWidth * 2);
        };
        auto issue = [&](int i, int buf, unsigned long long addr, int chunk) {
            if (in_page) {
                issue_rows(i, buf, addr);
            } else if (kRowsPerLoad == 1 && i < kLatLoads) {
                const int r0 = i * kWaves + wave;
                const unsigned lo = __builtin_amdgcn_readlane((unsigned)addr, r0),
                               hi = __builtin_amdgcn_readlane((unsigned)(addr >> 32), r0);
                load_to_lds16_lane((unsigned long long)hi << 32 | lo, (unsigned)(chunk ^ place_mix(r0)) * 16,
                                   lds0 + buf * kTileBytes + r0 * kLatRow);
            } else {
                issue_from(i, buf, __shfl(addr, row_of(i, chunk)), chunk);
            }
        };
        // A tile's powers of two, by one of the waves.
        auto issue_powers = [&](int buf, int page, int off) {
            if constexpr (NARROW) {
                const float* p = a.cache_scale + (long)page * a.page_size + off;
                if (wave == kWaves - 1)
                    load_to_lds4((unsigned)page < (unsigned)a.n_pages ? static_cast<const void*>(p) : kZeros, lds_address(powers[buf]));
            }
        };

        float m = kNoMax, l = 0.0f;
        f32x16 o[kOut] = {};
        unsigned long long valid = __ballot((unsigned)page < (unsigned)a.n_pages), valid_next = 0;
        int place_next = -1;  // of this lane's row of the tile after the next
        {
            const unsigned long long addr = address(page, off);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) issue(i, 0, addr, lane);
            issue_powers(0, page, off);
        }
        lds_barrier();  // the queries of all waves have landed
        bf16x8 qf[kSteps];
        {
            const int r = rg * 32 + col;
            const unsigned lat_at = query0 + r * kQueryRow + inner * RANK + ((half << NARROW) ^ (r & 15)) * 16;
            const unsigned rope_from = query_rope0 + r * (kRopeWidth * 2) + (((inner * 4 + half) ^ (r >> 1)) & 7) * 16;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const int mixed = NARROW ? (k >> 1 & 3) * 64 + (k & 1) * 16 : (k & 7) * 32;
                qf[k] = lds_chunk(k < kLat ? (lat_at ^ mixed) + (k >> 3) * 256 : rope_from ^ (k - kLat) * 32);
            }
#pragma unroll
            for (int k = 0; k < kSteps; ++k) asm volatile("" : "+v"(qf[k]));
        }
        lds_barrier();  // their place may be loaded over
        page = page_next;
        off = off_next;
        // The tile after the next has its page numbers brought to LDS by one
        // wave: a load into a register would be waited for with all others.
        auto issue_pages = [&](int t, int slot) {
            place_next = place_of(t, off);
            if (wave == 0)
                load_to_lds4(place_next >= 0 ? static_cast<const void*>(my_pages + place_next) : kZeros, lds_address(pages_ahead[slot]));
        };
        int buf = 0;
        if constexpr (NARROW) {
            asm volatile("" : "+v"(page));
            valid_next = __ballot((unsigned)page < (unsigned)a.n_pages);
            const unsigned long long addr = address(page, off);
            if (t_first + 1 < t_last) issue_powers(1, page, off);
            if (t_first + 2 < t_last) issue_pages(t_first + 2, 0);
            if (t_first + 1 < t_last) {
#pragma unroll
                for (int i = 0; i < kLoads; ++i) issue(i, 1, addr, lane);
            }
        }
        for (int t = t_first; t < t_last; ++t) {
            unsigned long long now = valid, next;
            bool more;
            int into;  // the buffer that the loads of this turn go to
            if constexpr (NARROW) {
                // tile t and the page numbers for t + 2 are in LDS; the loads
                // of tile t + 1 may be on their way
                if (t + 1 < t_last)
                    wait_vmem<kLoads>();
                else
                    wait_vmem<0>();
                lds_barrier();  // every wave is done with the third buffer
                if (t > t_first) buf = buf == 2 ? 0 : buf + 1;
                buf = __builtin_amdgcn_readfirstlane(buf);
                into = buf == 0 ? 2 : buf - 1;
                more = t + 2 < t_last;
                valid = valid_next;
                next = 0;
            } else {
                buf = (t - t_first) & 1;
                into = buf ^ 1;
                wait_vmem<0>();
                asm volatile("" : "+v"(page));  // the next tile's pages have landed: no later wait covers its loads
                lds_barrier();                  // tile t is in LDS, and every wave is done with the other buffer
                valid = __ballot((unsigned)page < (unsigned)a.n_pages);
                next = address(page, off);
                more = t + 1 < t_last;
                page = page_of(t + 2, off);
            }
            // (8 bits) what the loads of tile t + 2 go by, once the first matrix
            // instructions are on their way
            auto look_ahead = [&]() {
                const int got = pages_ahead[(t - t_first) & 1][lane];
                page = more && place_next >= 0 ? got : -1;
                valid_next = __ballot((unsigned)page < (unsigned)a.n_pages);
                next = address(page, off);
                if (more) issue_powers(into, page, off);
                if (t + 3 < t_last) issue_pages(t + 3, (t + 1 - t_first) & 1);
            };
            int chunk = lane;
            asm volatile("" : "+v"(chunk));  // the mixed places are not worth a register each across the loop
            const unsigned tile = buf * kTileBytes;
            float s[8];  // of the wave's keys, a quarter of the tile's
            {
                f32x16 sum = {};  // over the wave's half of the inner dimension
                // operands are read kAhead instructions before their use; the
                // scheduling barriers keep the compiler from reading them all
                // at once
                unsigned rope_base[kRope];  // plus immediate offsets
#pragma unroll
                for (int k = 0; k < kRope; ++k) rope_base[k] = (rope_at + tile) ^ k * 32;
                if constexpr (NARROW) {
                    // An item is 16 codes, widened for two instructions, or a
                    // chunk of the position part
                    constexpr int kPairs = kLat / 2, kItems = kPairs + kRope, kAhead = 4, kFirst = 1;
                    u32x4 x[kAhead];
                    const int key = side * 32 + (col ^ inner * 16);
                    const float power = powers[buf][key];
                    auto item = [&](int k) {
                        return __builtin_bit_cast(u32x4, lds_chunk(k < kPairs ? (key_at + tile) ^ k * 32 : rope_base[k - kPairs]));
                    };
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) x[k] = item(k);
#pragma unroll
                    for (int k = 0; k < kItems; ++k) {
                        const u32x4 u = x[k % kAhead];
                        if (k < kPairs) {
                            mfma(sum, __builtin_bit_cast(bf16x8, codes_to_bf16(u[0], u[1], power)), qf[2 * k]);
                            mfma(sum, __builtin_bit_cast(bf16x8, codes_to_bf16(u[2], u[3], power)), qf[2 * k + 1]);
                        } else {
                            mfma(sum, __builtin_bit_cast(bf16x8, u), qf[kLat + k - kPairs]);
                        }
                        if (k + kAhead < kItems) x[k % kAhead] = item(k + kAhead);
                        if (k == kFirst) {
                            // The conversion goes by the scale's exponent, and so do
                            // the weights.  One that is not finite counts as 2^127
                            // there, for keys whose weight is zero; a row that sees
                            // such a key has it in its score.  (All waves leave the
                            // same values; masked by each wave for its own keys: 1 to
                            // 2 % slower.)
                            const unsigned exponent = __builtin_bit_cast(unsigned, power) & 0x7F800000u;
                            value_powers[key] = exponent < 0x7F000000u ? exponent : 0x7F000000u;
                            look_ahead();
                        }
                        if (k > kFirst) {
                            constexpr int kFor = kItems - 1 - kFirst;
                            const int j = k - 1 - kFirst;
#pragma unroll
                            for (int i = j * kLoads / kFor; i < (j + 1) * kLoads / kFor; ++i)
                                if (more) issue(i, into, next, chunk);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                } else {
                    constexpr int kAhead = 6;
                    bf16x8 x[kAhead];
                    unsigned key_base[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) key_base[k] = (key_at + tile) ^ k * 32;
                    auto key_chunk = [&](int k) {
                        return lds_chunk(k < kLat ? key_base[k & 7] + (k >> 3) * 256 : rope_base[k - kLat]);
                    };
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) x[k] = key_chunk(k);
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        mfma(sum, x[k % kAhead], qf[k]);
                        if (k + kAhead < kSteps) x[k % kAhead] = key_chunk(k + kAhead);
                        // the next tile's loads, spread over the instructions (a
                        // wave that issues them in one go stalls in the queue)
#pragma unroll
                        for (int i = k * kLoads / kSteps; i < (k + 1) * kLoads / kSteps; ++i)
                            if (more) issue(i, into, next, chunk);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                f32x4 give[2];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[i] = sum[i];
                    give[i / 4][i % 4] = sum[8 + i];
                }
                slots[wave][0][lane] = __builtin_bit_cast(u32x4, give[0]);
                slots[wave][1][lane] = __builtin_bit_cast(u32x4, give[1]);
                lds_barrier();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const f32x4 got = __builtin_bit_cast(f32x4, slots[other][j][lane]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[j * 4 + i] += got[i];
                }
            }
            bool bad = false;  // a value that is not finite
            if (now != ~0ull || (t + 1) * kTile > context + (a.tree ? 0 : 1)) {
                // visible keys of this tile, a bit each; this lane's registers
                // hold keys 16 inner + 8 (i / 4) + 4 half + i % 4 of the
                // wave's half
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
                const unsigned word = (unsigned)(sees >> (quarter * 16)) >> (4 * half);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s[i] = word >> (8 * (i / 4) + i % 4) & 1 ? s[i] : -__builtin_inff();
                // (rows past the end that a load of whole groups brought count too)
                if ((NARROW && now != ~0ull) || (before < kTile && (a.tree || count > 1))) {
                    // new tokens that some of them do not see: this wave looks
                    // over its share of the rows
                    unsigned p = lds0 + tile + wave * (kLatBytes / kWaves) + lane * 16;
#pragma unroll 4
                    for (int i = 0; i < kLatBytes / kWaves / 1024; ++i, p += 1024)
                        bad |= holds_not_finite<NARROW>(__builtin_bit_cast(u32x4, lds_chunk(p)));
                }
            }
            // the first values are read before the exchange
            constexpr int kAhead = 6;
            typedef typename ValueOperand<NARROW>::type value_t;
            value_t x[kAhead];
            unsigned lo[kOut], hi[kOut];
#pragma unroll
            for (int k = 0; k < kOut; ++k) {
                lo[k] = (value_at + tile) ^ k * (32 * kBytes);
                hi[k] = (lo[k] ^ 32) + 8 * RANK * 2;  // (the wide cache's)
            }
            auto value_chunk = [&](int j) {
                const int k = j >> 2, at_key = (j & 3) * 16 * kLatRow;
                if constexpr (NARROW)
                    return codes_transposed(lo[k] + at_key);
                else
                    return values_transposed(lo[k] + at_key, hi[k] + at_key);
            };
            // The powers of two of the wave's keys, in the order of its
            // scores: what a code stands for enters through the weights.
            f32x4 power_of[NARROW ? 2 : 1];
            if constexpr (NARROW) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    power_of[i] = *reinterpret_cast<const f32x4*>(&value_powers[quarter * 16 + half * 4 + i * 8]);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) x[j] = value_chunk(j);
            float top = s[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, s[i]);
            top = half_max(top);
            const bool raise = __any((top - m) * c > kMaxSlack);
            // the sum takes them before they are rounded to bf16: the roundings
            // of numerator and denominator do not cancel, but average out
            auto exponentials = [&]() {
                const float mc = m * c;
                float sum = 0.0f;
                bf16x8 p;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float e = __builtin_amdgcn_exp2f(fmaf(s[i], c, -mc));
                    sum += e;
                    if constexpr (NARROW)
                        p[i] = (__bf16)(e * power_of[i / 4][i % 4]);
                    else
                        p[i] = (__bf16)e;
                }
                slots[other][0][lane] = __builtin_bit_cast(u32x4, p);
                return sum;
            };
            float sum = exponentials();
            if (half == 0) my_top[col] = top;
            const bool guard = __any(bad);
            // the position part of this tile has served: flags lie there, a byte
            // per wave
            uint8_t* const flags = lds + tile + kLatBytes;
            if (lane == 0) flags[wave] = (uint8_t)(raise + 2 * guard);
            lds_barrier();
            unsigned any = reinterpret_cast<const unsigned*>(flags)[0];
            if constexpr (kWaves > 4) any |= reinterpret_cast<const unsigned*>(flags)[1];
            bf16x8 p[4];  // of all 64 keys, in key order
            auto take = [&]() {
#pragma unroll
                for (int w = 0; w < 4; ++w) p[w] = __builtin_bit_cast(bf16x8, slots[rg * 4 + (w ^ 1)][0][lane]);
            };
            take();
            any = __builtin_amdgcn_readfirstlane(any);
            if (any & 0x02020202u) {
                // Every wave has taken its scores: only the finite values stay
                // in the tile.  A row that sees one of the others has it in its
                // score, the value being part of the key.
                unsigned at_row = lds0 + tile + wave * (kLatBytes / kWaves) + lane * 16;
#pragma unroll 1
                for (int i = 0; i < kLatBytes / kWaves / 1024; ++i, at_row += 1024)
                    lds_store(at_row, only_finite<NARROW>(__builtin_bit_cast(u32x4, lds_chunk(at_row))));
                lds_barrier();
#pragma unroll
                for (int j = 0; j < kAhead; ++j) x[j] = value_chunk(j);
            }
            if (any & 0x01010101u) {
                // some row's maximum moves: the four waves of its block take
                // the new one and compute their exponentials again
                float nm = m;
#pragma unroll
                for (int w = 0; w < 4; ++w) nm = fmaxf(nm, slot_of(rg * 4 + w)[col]);
                const float f = __builtin_amdgcn_exp2f((m - nm) * c);
                m = nm;
                l *= f;
                if (t > t_first) {  // else there is nothing to bring to it
#pragma unroll
                    for (int k = 0; k < kOut; ++k)
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[k][i] *= f;
                }
                lds_barrier();  // the first ones are read
                sum = exponentials();
                lds_barrier();
                take();
            }
            l += sum;
            {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < 4 * kOut; ++j) {
                    mfma(o[j >> 2], value_operand(x[j % kAhead]), p[j & 3]);
                    if (j + kAhead < 4 * kOut) x[j % kAhead] = value_chunk(j + kAhead);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        // totals over the keys of all four waves
        l = half_sum(l);
        __syncthreads();
        if (half == 0) my_top[col] = l;
        __syncthreads();
        l = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) l += slot_of(rg * 4 + w)[col];
        const bool all = t_first == 0 && t_last == tiles;
        if (!KEEP && all) {
            if (row_ok) {
                // a row that sees no key gives zero
                const float inv = l != 0.0f ? 1.0f / l : 0.0f;
                uint16_t* out = a.out + (first + token) * a.o_stride_t + head * a.o_stride_h + quarter * (RANK / 4) + half * 4;
#pragma unroll
                for (int k = 0; k < kOut; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<u32x2*>(out + k * 32 + i * 8) =
                            u32x2{pack_bf16(o[k][i * 4] * inv, o[k][i * 4 + 1] * inv),
                                  pack_bf16(o[k][i * 4 + 2] * inv, o[k][i * 4 + 3] * inv)};
            }
        } else {
            float* part = part_sums<ROWS, RANK>(a, slot * 2 + (t_first == 0));
            int r = rg * 32 + col;
            float* stats = part + ROWS * RANK;
            if (KEEP && all) {
                part = whole;
                stats = whole + (long)a.T * a.heads * RANK;
                r = (first + token) * a.heads + head;
            }
            if (!(KEEP && all) || row_ok) {
#pragma unroll
                for (int k = 0; k < kOut; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<f32x4*>(part + (long)r * RANK + quarter * (RANK / 4) + k * 32 + i * 8 + half * 4) =
                            f32x4{o[k][i * 4], o[k][i * 4 + 1], o[k][i * 4 + 2], o[k][i * 4 + 3]};
                if (half == 0 && quarter == 0) {
                    stats[(long)r * 2] = m;
                    stats[(long)r * 2 + 1] = l;
                }
            }
        }
        at += t_last - t_first;
        lds_barrier();  // the buffers are free for the next part's first tile
    }
}

template <int RANK, int RG, bool NARROW>
__global__ void __launch_bounds__(RG * 256, 1) latent_attention_kernel(LatentArgs a) {
    touch_arguments<sizeof(a)>();
    // workgroups are dealt to the eight dies in turn: group g lies on die g % 8
    const int turn = blockIdx.x >> 3, run = (blockIdx.x & 7) + 8 * (turn / a.group), member = turn % a.group;
    int before;
    const int total = count_tiles<RG * 32>(a, 0, threadIdx.x & 63, before), runs = run_count(total, a.runs);
    if (run >= runs) return;
    attend<RANK, RG, NARROW, false>(a, total, runs, run, member, run * a.group + member, nullptr);
}

// Joins the partial sums of every unit that more than one run worked on:
// RANK / 64 columns per lane, the runs in order.  SPLIT waves share a row, 16
// runs each in turn, and are joined in wave order.
template <int RANK, int ROWS, int SPLIT>
__global__ void __launch_bounds__(256) latent_join_kernel(LatentArgs a) {
    touch_arguments<sizeof(a)>();
    constexpr int V = RANK / 64, kAtOnce = SPLIT > 1 ? 16 : 64;
    __shared__ float shared_o[SPLIT > 1 ? 4 : 1][V][64];
    __shared__ float shared_ml[4][2];
    const int lane = threadIdx.x & 63, wave = wave_in_block(), part_of = wave % SPLIT;
    const int seq = blockIdx.y, row = blockIdx.x * (4 / SPLIT) + wave / SPLIT;
    const SeqShape shape = seq_shape<ROWS>(a, seq);
    if (row >= shape.count * a.heads) return;
    int before;
    const int total = count_tiles<ROWS>(a, seq, lane, before), runs = run_count(total, a.runs);
    if (total == 0) return;  // nor has the first launch done anything
    const int block = row / ROWS, r = row % ROWS, member = block % a.group;
    const int u0 = before + block / a.group * shape.tiles, u1 = u0 + shape.tiles;
    // runs that hold the unit's first and last tile
    const int each = total / runs, more = total - each * runs, longer = more * (each + 1);
    auto run_of = [&](int tile) { return tile < longer ? tile / (each + 1) : more + (tile - longer) / each; };
    const int g0 = run_of(u0), g1 = run_of(u1 - 1);
    if (g0 == g1) return;  // one run held it all and wrote the result
    auto part = [&](int g) { return part_sums<ROWS, RANK>(a, (g * a.group + member) * 2 + (g == g0)); };
    const float c = a.scale * 1.44269504088896340736f;
    float m = kNoMax, l = 0.0f, o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.0f;
    for (int b0 = g0 + part_of * kAtOnce; b0 <= g1; b0 += SPLIT * kAtOnce) {
        // maxima and totals of these runs, one per lane
        const int n = g1 + 1 - b0 < kAtOnce ? g1 + 1 - b0 : kAtOnce;
        float pm = kNoMax, pl = 0.0f;
        if (lane < n) {
            const float* p = part(b0 + lane) + ROWS * RANK + r * 2;
            pm = p[0];
            pl = p[1];
        }
        float top = pm;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
        const float nm = fmaxf(m, top), f = __builtin_amdgcn_exp2f((m - nm) * c);
        const float w = __builtin_amdgcn_exp2f((pm - nm) * c);
        m = nm;
        l = l * f + wave_sum(w * pl);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] *= f;
        for (int k0 = 0; k0 < n; k0 += 4) {  // four runs' loads in flight
            f32x4 v[4][V / 4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float* p = part(b0 + (k0 + k < n ? k0 + k : n - 1)) + (long)r * RANK + lane * V;
#pragma unroll
                for (int i = 0; i < V / 4; ++i) v[k][i] = as_global<f32x4>(p)[i];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float wk = k0 + k < n ? readlane_f(w, k0 + k) : 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = fmaf(v[k][i / 4][i % 4], wk, o[i]);
            }
        }
    }
    if constexpr (SPLIT > 1) {
        static_assert(SPLIT == 4, "a workgroup per row");
#pragma unroll
        for (int i = 0; i < V; ++i) shared_o[wave][i][lane] = o[i];
        if (lane == 0) {
            shared_ml[wave][0] = m;
            shared_ml[wave][1] = l;
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int w = 1; w < SPLIT; ++w) m = fmaxf(m, shared_ml[w][0]);
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < SPLIT; ++w) {
            const float f = __builtin_amdgcn_exp2f((shared_ml[w][0] - m) * c);
            l = fmaf(shared_ml[w][1], f, l);
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = fmaf(shared_o[w][i][lane], f, o[i]);
        }
    }
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    uint16_t* out = a.out + (long)(shape.first + row / a.heads) * a.o_stride_t + (row % a.heads) * a.o_stride_h + lane * V;
#pragma unroll
    for (int i = 0; i < V; i += 4)
        *reinterpret_cast<u32x2*>(out + i) =
            u32x2{pack_bf16(o[i] * inv, o[i + 1] * inv), pack_bf16(o[i + 2] * inv, o[i + 3] * inv)};
}

// How a call of these bounds is cut: rows per workgroup, workgroups per
// group, most runs.
struct LatentCut {
    int rows, group, runs;
};
[[maybe_unused]] LatentCut latent_cut(int B, int max_q, int heads, int max_len, bool narrow) {
    LatentCut c;
    const long rows = (long)max_q * heads;
    c.rows = rows > 32 ? 64 : 32;
    const long blocks = (rows + c.rows - 1) / c.rows;
    c.group = (int)(blocks < kMaxGroup ? blocks : kMaxGroup);
    const long passes = (blocks + c.group - 1) / c.group;
    const long tiles = max_len > kTile ? (max_len + kTile - 1) / kTile : 1;
    // (a group's workgroups lie on one die, which holds 32 at once)
    const long most = narrow ? kMaxWorkgroups / 8 / c.group * 8 : kMaxWorkgroups / c.group, all = B * passes * tiles;
    c.runs = (int)(all < most ? all : most);
    return c;
}

// Up to this many rows get a workgroup each in the join, so that more of the
// chip reads the sums: one sequence of 16384 rows 54 to 34 us (64 heads),
// four tokens of it 37 to 35; at 8 sequences of 4096 a wave per row is
// better, 30 against 32.
constexpr long kFewRows = 256;

template <int RANK, int RG, bool NARROW>
void launch_rows(LatentArgs a, const LatentCut& cut, hipStream_t s) {
    a.group = cut.group;
    a.runs = cut.runs;
    a.per_seq = a.cu_q ? 0 : a.T / a.B;
    const int grid = (cut.runs + 7) / 8 * 8 * cut.group;
    hipLaunchKernelGGL((latent_attention_kernel<RANK, RG, NARROW>), dim3(grid), dim3(RG * 256), 0, s, a);
    if (cut.runs > 1) {
        const int rows = (a.max_q < a.T ? a.max_q : a.T) * a.heads;
        if ((long)rows * a.B <= kFewRows)
            hipLaunchKernelGGL((latent_join_kernel<RANK, RG * 32, 4>), dim3(rows, a.B), dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((latent_join_kernel<RANK, RG * 32, 1>), dim3((rows + 3) / 4, a.B), dim3(256), 0, s, a);
    }
}
template <int RANK, bool NARROW>
void launch_rank(const LatentArgs& a, hipStream_t s) {
    const LatentCut cut = latent_cut(a.B, a.max_q, a.heads, a.max_len, NARROW);
    if (cut.rows == 64)
        launch_rows<RANK, 2, NARROW>(a, cut, s);
    else
        launch_rows<RANK, 1, NARROW>(a, cut, s);
}

}  // namespace
}  // namespace moe
