// Latent attention of sequences that share long prefixes: a prefix is a
// sequence whose tokens are those of all the sequences on it, so that its rows
// are read once for up to 512 (token, head) rows of a group of workgroups, and
// not once per sequence.
//
// The prefixes' tiles form a list beside that of the sequences' own rows, and
// the workgroups of one launch are divided between the two by the lists' work,
// in runs of equal length each.  Either list leaves fp32 sums, maxima and
// totals; a second launch joins them, a row's own first.
//
// Bound by what a tile of 64 keys costs 64 rows (2.5 us, the matrix cores 31 %
// busy), as in the form without prefixes; the cache's bytes do not count any
// more.  Measured, rank 512, 64 heads: 32 tokens on a prefix of 16384 rows, up to
// 500 own ones, 103 us (0.72 PFLOP/s, bf16; join 12); trees of 4 tokens of 16
// sequences on prefixes of 8192 and 6554 rows, 8 bits, 113 us (0.61); 2 tokens
// on 517 rows 22.6 us, a chain of latencies.  Where a token's heads fill 64 rows,
// each sequence by itself over the same pages takes as long, a few per cent less
// (8 prefixes of 32768 rows, 302 MB, 4 tokens on each: 202 against 219) and up to
// a fifth less where there is little to do (8 tokens on 4096 rows: 34 against
// 39); with fewer heads the rows of several tokens share a tile (16 heads: 51
// against 93).  (128 rows to a workgroup, whole rows in a wave: 272 accumulators, which
// the compiler spills.)
#include "moe_latent_device.h"

namespace moe {
namespace {

constexpr int kRows = 64;  // (token, head) rows per workgroup

__device__ __forceinline__ void as_prefixes(LatentArgs& a, const PrefixArgs& p) {
    a.seqs = a.B;
    a.prefixes = true;
    a.groups = p.groups;
    a.pages = p.pages;
    a.lens = p.lens;
    a.pages_stride = p.pages_stride;
    a.pages_per_seq = p.pages_per_seq;
    a.B = p.count;
    a.group = p.group;
    a.tree = nullptr;
}

// How the workgroups of eight dies, per_die on each, serve lists of total_own
// and total_prefix tiles in own_units and prefix_units pieces: the prefixes'
// runs are dealt to the dies in turn, p.group workgroups each, and own runs
// take what is left on each die.  Whole numbers only: both launches have to
// come to the same.
struct Split {
    int own, prefix;       // runs
    int base, extra;       // prefix runs on each die, and dies that have one more
    int low, high;         // own runs on those dies, and on the others
};
struct Lists {
    int own, own_units, prefix, prefix_units;
};
__device__ __forceinline__ Split split_at(int prefix, int total_own, int own_group, int prefix_group, int per_die) {
    Split s;
    s.prefix = prefix;
    s.base = s.prefix >> 3;
    s.extra = s.prefix & 7;
    s.high = (per_die - s.base * prefix_group) / own_group;
    s.low = s.extra ? (per_die - (s.base + 1) * prefix_group) / own_group : s.high;
    const int room = s.low * 8 + (s.high - s.low) * (8 - s.extra);
    s.own = total_own < room ? total_own : room;
    return s;
}
// What starting and ending a unit costs a run, in tiles (measured: 8 sequences
// of 5 tiles took a run as long as 60 tiles of one).
constexpr unsigned kUnitTiles = 2;
__device__ __forceinline__ Split split_runs(const Lists& n, int own_group, int prefix_group, int per_die) {
    if (n.prefix == 0) return split_at(0, n.own, own_group, prefix_group, per_die);
    const unsigned long long p = (unsigned long long)(n.prefix + kUnitTiles * n.prefix_units) * prefix_group,
                             o = (unsigned long long)(n.own + kUnitTiles * n.own_units) * own_group;
    const int bits = 64 - __builtin_clzll(p + o), shift = bits > 20 ? bits - 20 : 0;
    const unsigned part = (unsigned)(p >> shift), whole = (unsigned)((p + o) >> shift) * (unsigned)prefix_group;
    const int near = (int)(per_die * 8 * part / whole);
    // at least one die keeps room for an own run
    const int most = 8 * ((per_die - own_group) / prefix_group) + 7, all = 8 * (per_die / prefix_group);
    int limit = most < all ? most : all;
    limit = limit < n.prefix ? limit : n.prefix;
    // of the numbers next to the even share, the one whose longer list is shortest
    Split best{};
    unsigned least = ~0u;
    for (int i = -1; i <= 1; ++i) {
        int at = near + i;
        at = at > limit ? limit : at;
        at = at < 1 ? 1 : at;
        const Split s = split_at(at, n.own, own_group, prefix_group, per_die);
        const unsigned a = (n.prefix + kUnitTiles * n.prefix_units + s.prefix - 1) / s.prefix,
                       b = (n.own + kUnitTiles * n.own_units + s.own - 1) / s.own, time = a > b ? a : b;
        if (time < least) {
            least = time;
            best = s;
        }
    }
    return best;
}
// The lists of both kinds: their tiles and units, and the tiles before
// sequence `seq` and prefix `g`.
__device__ __forceinline__ Lists count_lists(const LatentArgs& a, const LatentArgs& q, int seq, int g, int lane, int& before,
                                             int& before_prefix) {
    Lists n;
    n.own_units = n.prefix_units = 0;
    n.own = count_tiles<kRows>(a, seq, lane, before, &n.own_units);
    n.prefix = count_tiles<kRows>(q, g, lane, before_prefix, &n.prefix_units);
    return n;
}

// Sums of units that one run held whole, by row, after the partial ones.
template <int RANK>
__device__ __forceinline__ float* whole_sums(const LatentArgs& a, const PrefixArgs& p, bool prefix) {
    const long each = ((long)a.T * a.heads * (RANK + 2) + 3) & ~3l;
    return part_sums<kRows, RANK>(a, p.per_die * 8 * 2) + (prefix ? each : 0);
}

template <int RANK, bool NARROW>
__global__ void __launch_bounds__(512, 1) latent_shared_kernel(LatentArgs a, PrefixArgs p) {
    touch_arguments<sizeof(a) + sizeof(p)>();
    const int lane = threadIdx.x & 63, die = blockIdx.x & 7, turn = blockIdx.x >> 3;
    LatentArgs q = a;
    as_prefixes(q, p);
    int before, before_prefix;
    const Lists n = count_lists(a, q, 0, 0, lane, before, before_prefix);
    if (n.own == 0) return;
    const Split s = split_runs(n, a.group, p.group, p.per_die);
    const int prefix_turns = (s.base + (die < s.extra)) * p.group;
    const bool prefix = turn < prefix_turns;
    int run, member;
    if (prefix) {
        run = turn / p.group * 8 + die;
        member = turn % p.group;
        as_prefixes(a, p);
    } else {
        const int at = (turn - prefix_turns) / a.group;
        member = (turn - prefix_turns) % a.group;
        if (at >= (die < s.extra ? s.low : s.high)) return;
        run = at < s.low ? at * 8 + die : s.low * 8 + (at - s.low) * (8 - s.extra) + die - s.extra;
    }
    const int runs = prefix ? s.prefix : s.own;
    if (run >= runs) return;
    const int slot = run * a.group + member + (prefix ? 0 : s.prefix * p.group);
    attend<RANK, 2, NARROW, true>(a, prefix ? n.prefix : n.own, runs, run, member, slot, whole_sums<RANK>(a, p, prefix));
}

// The runs that hold a unit's sums for one row.
struct Sources {
    int first, count;     // runs
    int member, r;        // whose slot, and the row in it
    int slot, group;      // of run 0, and slots per run
};
__device__ __forceinline__ Sources sources_of(int total, int runs, int before, int tiles, int group, int row, int slot) {
    Sources s;
    const int block = row / kRows;
    s.r = row % kRows;
    s.member = block % group;
    s.group = group;
    s.slot = slot;
    const int u0 = before + block / group * tiles, u1 = u0 + tiles;
    const int each = total / runs, more = total - each * runs, longer = more * (each + 1);
    auto run_of = [&](int tile) { return tile < longer ? tile / (each + 1) : more + (tile - longer) / each; };
    s.first = run_of(u0);
    s.count = run_of(u1 - 1) - s.first + 1;
    return s;
}

// Joins a row's sums: SPLIT waves share it, 16 sources each in turn, or one
// wave takes 64 at once; RANK / 64 columns per lane.
template <int RANK, int SPLIT>
__global__ void __launch_bounds__(256) latent_shared_join_kernel(LatentArgs a, PrefixArgs p) {
    touch_arguments<sizeof(a) + sizeof(p)>();
    constexpr int V = RANK / 64, kAtOnce = SPLIT > 1 ? 16 : 64;
    __shared__ float shared_o[SPLIT > 1 ? 4 : 1][V][64];
    __shared__ float shared_ml[4][2];
    const int lane = threadIdx.x & 63, wave = wave_in_block();
    const int part_of = wave % SPLIT;
    const int seq = blockIdx.y, row = blockIdx.x * (4 / SPLIT) + wave / SPLIT;
    const SeqShape shape = seq_shape<kRows>(a, seq);
    if (row >= shape.count * a.heads) return;
    LatentArgs q = a;
    as_prefixes(q, p);
    // the sequence's prefix
    int g = p.groups ? -1 : 0;
    if (p.groups)
        for (int g0 = 0; g0 < p.count; g0 += 64) {
            const int i = g0 + lane;
            const unsigned long long hit = __ballot(i < p.count && p.groups[i < p.count ? i : 0] <= seq && seq < p.groups[i < p.count ? i + 1 : 0]);
            if (hit) {
                g = g0 + __builtin_ctzll(hit);
                break;
            }
        }
    int before, before_prefix;
    const Lists n = count_lists(a, q, seq, g < 0 ? 0 : g, lane, before, before_prefix);
    if (n.own == 0) return;  // nor has the first launch done anything
    const Split s = split_runs(n, a.group, p.group, p.per_die);
    const Sources own = sources_of(n.own, s.own, before, shape.tiles, a.group, row, s.prefix * p.group);
    Sources pre{};
    if (g >= 0 && n.prefix > 0) {
        const SeqShape of = seq_shape<kRows>(q, g);
        const int r = (shape.first - of.first) * a.heads + row;
        // (bounds in device memory that decrease can put a row outside its group)
        if (r >= 0 && r < of.count * a.heads)
            pre = sources_of(n.prefix, s.prefix, before_prefix, of.tiles, p.group, r, 0);
    }
    const int sources = own.count + pre.count;
    const long rows = (long)a.T * a.heads, at = (long)shape.first * a.heads + row;
    // where source i has its sums, and its maximum and total
    auto sums = [&](int i, const float*& o, const float*& ml) {
        const bool prefix = i >= own.count;
        const Sources& u = prefix ? pre : own;
        if (u.count == 1) {
            const float* w = whole_sums<RANK>(a, p, prefix);
            o = w + at * RANK;
            ml = w + rows * RANK + at * 2;
        } else {
            const int run = u.first + (prefix ? i - own.count : i);
            // (the second half of a slot is for the unit that the run starts with tile 0)
            const float* w = part_sums<kRows, RANK>(a, (u.slot + run * u.group + u.member) * 2 + (run == u.first));
            o = w + (long)u.r * RANK;
            ml = w + kRows * RANK + u.r * 2;
        }
    };
    const float c = a.scale * 1.44269504088896340736f;
    float m = kNoMax, l = 0.0f, o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.0f;
    for (int b0 = part_of * kAtOnce; b0 < sources; b0 += SPLIT * kAtOnce) {
        // maxima and totals of these sources, one per lane
        const int n = sources - b0 < kAtOnce ? sources - b0 : kAtOnce;
        float pm = kNoMax, pl = 0.0f;
        if (lane < n) {
            const float *unused, *ml;
            sums(b0 + lane, unused, ml);
            pm = ml[0];
            pl = ml[1];
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
        for (int k0 = 0; k0 < n; k0 += 4) {  // four sources' loads in flight
            f32x4 v[4][V / 4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float *from, *unused;
                sums(b0 + (k0 + k < n ? k0 + k : n - 1), from, unused);
#pragma unroll
                for (int i = 0; i < V / 4; ++i) v[k][i] = as_global<f32x4>(from + lane * V)[i];
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

// Workgroups per group of the sequences' own rows and of the prefixes, and
// workgroups per die: as many as there are tiles for, at most 32.
struct SharedCut {
    int own, prefix, per_die;
};
SharedCut shared_cut(int B, int T, int max_q, int heads, int max_len, int prefixes, int max_prefix) {
    auto least = [](long a, long b) { return a < b ? a : b; };
    auto up = [](long a, long b) { return (a + b - 1) / b; };
    const long own_blocks = up((long)(max_q < T ? max_q : T) * heads, kRows), blocks = up(up(T, prefixes) * heads, kRows);
    SharedCut c;
    c.own = (int)least(own_blocks, kMaxGroup / 2);
    c.prefix = (int)least(blocks, kMaxGroup);
    const long tiles = least((double)B * up(own_blocks, c.own) * c.own * up(max_len > 1 ? max_len : 1, kTile), 1 << 20) +
                       least((double)prefixes * up(blocks, c.prefix) * c.prefix * up(max_prefix > 1 ? max_prefix : 1, kTile), 1 << 20);
    const long wanted = up(tiles, 8) + c.own + c.prefix;
    c.per_die = (int)least(wanted, kMaxWorkgroups / 8);
    return c;
}

template <int RANK, bool NARROW>
void launch(LatentArgs a, PrefixArgs p, hipStream_t s) {
    const SharedCut cut = shared_cut(a.B, a.T, a.max_q, a.heads, a.max_len, p.count, p.max_len);
    a.group = cut.own;
    a.per_seq = a.cu_q ? 0 : a.T / a.B;
    p.group = cut.prefix;
    p.per_die = cut.per_die;
    hipLaunchKernelGGL((latent_shared_kernel<RANK, NARROW>), dim3(cut.per_die * 8), dim3(512), 0, s, a, p);
    const int rows = (a.max_q < a.T ? a.max_q : a.T) * a.heads;
    if ((long)rows * a.B <= kFewRows)
        hipLaunchKernelGGL((latent_shared_join_kernel<RANK, 4>), dim3(rows, a.B), dim3(256), 0, s, a, p);
    else
        hipLaunchKernelGGL((latent_shared_join_kernel<RANK, 1>), dim3((rows + 3) / 4, a.B), dim3(256), 0, s, a, p);
}

}  // namespace

size_t latent_shared_workspace(int B, int T, int max_q, int heads, int rank, int max_len, int prefixes, int max_prefix) {
    const SharedCut c = shared_cut(B, T, max_q, heads, max_len, prefixes, max_prefix);
    const size_t whole = ((size_t)T * heads * (rank + 2) + 3) & ~(size_t)3;
    return ((size_t)c.per_die * 8 * 2 * kRows * (rank + 2) + 2 * whole) * sizeof(float);
}

hipError_t launch_latent_shared(const LatentArgs& a, const PrefixArgs& p, hipStream_t s) {
    if (a.cache_scale) {
        if (a.rank == 512)
            launch<512, true>(a, p, s);
        else
            launch<256, true>(a, p, s);
    } else {
        if (a.rank == 512)
            launch<512, false>(a, p, s);
        else
            launch<256, false>(a, p, s);
    }
    return hipGetLastError();
}

}  // namespace moe
