"""GPU tests of the kernels' loops that only larger inputs enter: every tile
shape of the 8-bit product, the per-head product's passes over token tiles, and
latent attention over runs of several tiles and joins of many runs
(routed_expert_int4_amd/csrc).

References in 64 bits and tolerances are those of test_gpu_attention.py.  In
addition: the 8-bit matrix instructions align each group of eight products to
its largest and cut what lies more than 13 bits below it, so that seven
products of a group lose up to 2^-13 of the eighth each: 7 x 2^-13 of the sum
of magnitudes at the very worst, whatever the inputs (CUT); terms of one size
lose the 3e-5 of it that the other tests allow."""
import os
import re

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_int4_amd import attention as A  # noqa: E402
from test_gpu_attention import BF, D, DEV, U, close, cumulative, fp8_inputs, fp8_ref, gen, normal, strided  # noqa: E402

CUT = 7 * 2.0 ** -13
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routed_expert_int4_amd", "csrc")


# ---------------------------------------------------------------- 8-bit product
def tile_shape(M, N):
    """The shape that the dispatch takes, by its table of costs."""
    text = open(os.path.join(CSRC, "moe_fp8.hip")).read()
    table = re.search(r"kTileShapes\[\] = \{(.*?)\};", text, flags=re.S).group(1)
    shapes = [tuple(map(int, t)) for t in re.findall(r"\{(\d+), (\d+), (\d+), (\d+)\}", table)]
    assert len(shapes) == 5
    cost = [-(-(-(-N // bn) * -(-M // bt)) // slots) * cost for bn, bt, slots, cost in shapes]
    return cost.index(min(cost))


@pytest.mark.parametrize("K", [400, 8368, 1024])  # 4 blocks, the last of 16; 66, the last of 48; 8
@pytest.mark.parametrize("shape,M,N", [(0, 70, 577), (1, 1030, 1001), (1, 515, 2064), (2, 515, 4101), (2, 2050, 1000),
                                       (3, 2050, 2061), (3, 515, 8200), (4, 1030, 8203), (4, 2050, 4104)])
def test_fp8_linear_tile_shapes(shape, M, N, K):
    assert tile_shape(M, N) == shape
    g = gen(M + N + K)
    a, sa, w, sw = fp8_inputs(g, M, N, K)
    ref, mag = fp8_ref(a, sa, w, sw)
    close(A.fp8_linear(a, sa, w, sw, out_dtype=torch.float32), ref, 3e-5 * mag, "fp32")
    # operands and output as views of wider rows
    wide = torch.full((M, K + 32), 0x7F, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # NaN around the rows
    wide.view(torch.uint8)[:, :K] = a.view(torch.uint8)
    wide_w = torch.full((N, K + 16), 0x7F, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    wide_w.view(torch.uint8)[:, :K] = w.view(torch.uint8)
    for extra in (3, 8 - N % 8):
        out = torch.full((M, N + extra), -7.0, dtype=BF, device=DEV)
        A.fp8_linear(wide[:, :K], sa.t().contiguous().t(), wide_w[:, :K], sw, out=out[:, :N])
        close(out[:, :N], ref, U * ref.abs() + 3e-5 * mag, f"row of {N + extra}")
        assert (out[:, N:] == -7.0).all()


@pytest.mark.parametrize("M", [4, 70, 600])
@pytest.mark.parametrize("K", [80, 96, 128, 144, 272, 1040])
def test_fp8_linear_terms_of_many_sizes(M, K):
    g = gen(M + K)
    a, sa, w, sw = fp8_inputs(g, M, 260, K)

    def skewed(*shape):
        x = normal(g, *shape, dtype=torch.float32)
        return ((2 * x).exp() * x.sign()).clamp(-448, 448).to(torch.float8_e4m3fn)

    spread, spread_w = skewed(M, K), skewed(260, K)
    ref, mag = fp8_ref(spread, sa, spread_w, sw)
    close(A.fp8_linear(spread, sa, spread_w, sw, out_dtype=torch.float32), ref, CUT * mag, "log-normal terms")
    few = normal(g, M, K, dtype=torch.float32)
    few[:, 5::37] *= 300  # columns of large activations, as models have them
    few = few.clamp(-448, 448).to(torch.float8_e4m3fn)
    ref, mag = fp8_ref(few, sa, w, sw)
    close(A.fp8_linear(few, sa, w, sw, out_dtype=torch.float32), ref, CUT * mag, "a few large columns")
    # the last block, short or not, outweighs the others
    sa[:, -1] *= 1000
    ref, mag = fp8_ref(a, sa, w, sw)
    close(A.fp8_linear(a, sa, w, sw, out_dtype=torch.float32), ref, CUT * mag, "a heavy last block")


# ---------------------------------------------------------------- per-head product
@pytest.mark.parametrize("T,heads,K,N", [(1000, 64, 512, 128), (1000, 64, 128, 512), (300, 64, 1100, 128), (333, 128, 520, 132),
                                         (700, 40, 72, 200), (20, 3, 1100, 36), (129, 2, 520, 260), (2100, 16, 96, 1000)])
def test_head_linear_passes(T, heads, K, N):
    """Workgroups that pass over several token tiles (64 tokens, shared by
    some 256 to 1024 workgroups) and over several parts of the inner dimension
    (512 columns)."""
    g = gen(T + K + N)
    K8 = -(-K // 8) * 8
    x, w = strided(normal(g, T, heads, K8), 8), normal(g, heads, N, K8, std=K8 ** -0.5)
    out = torch.full((T, heads, N + 4), -7.0, dtype=BF, device=DEV)
    A.head_linear(x, w, out=out[..., :N])
    xd, wd = x.to(D).transpose(0, 1).contiguous(), w.to(D).transpose(1, 2).contiguous()
    ref, mag = torch.matmul(xd, wd).transpose(0, 1), torch.matmul(xd.abs(), wd.abs()).transpose(0, 1)
    close(out[..., :N], ref, U * ref.abs() + 1e-5 * mag)
    assert (out[..., N:] == -7.0).all()
    # the same rows for every head
    one = normal(g, T, 1, K8).expand(T, heads, K8)
    ref = torch.matmul(one[:, 0].to(D).contiguous(), wd).transpose(0, 1)
    mag = torch.matmul(one[:, 0].to(D).abs().contiguous(), wd.abs()).transpose(0, 1)
    close(A.head_linear(one, w), ref, U * ref.abs() + 1e-5 * mag, "one row for all heads")


# ---------------------------------------------------------------- latent attention
def long_case(g, lens, page, rank, heads, nq):
    """Cache, page table and lengths, with rows at random places of the pool."""
    used = [-(-n // page) for n in lens]
    order = torch.randperm(sum(used) + 2, device=DEV, generator=g).to(torch.int32)
    pages = torch.full((len(lens), max(used)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(used):
        pages[b, :n] = order[at:at + n]
        at += n
    cache = normal(g, sum(used) + 2, page, rank + 64)
    return normal(g, sum(nq), heads, rank + 64), cache, pages, torch.tensor(lens, dtype=torch.int32, device=DEV)


def long_ref(q, cache, pages, lens, nq, scale, rank, tree=None):
    """(sum p v, sum p |v|), sequence by sequence."""
    out, mag, t = [], [], 0
    for b, (n, m) in enumerate(zip(lens, nq)):
        kv = cache[pages[b, :-(-n // cache.shape[1])].long()].flatten(0, 1)[:n].to(D)
        s = torch.matmul(q[t:t + m].to(D), kv.t().contiguous()) * scale  # [m, heads, n]
        place = torch.arange(n, device=DEV) - (n - m)
        own = torch.arange(m, device=DEV)[:, None]
        sees = place <= own
        if tree is not None:
            sees = (place < 0) | ((tree[t:t + m, None] >> place.clamp(0, 63)) & 1 == 1)
        p = torch.softmax(s.masked_fill(~sees[:, None], -torch.inf), 2)
        out.append(torch.matmul(p, kv[:, :rank].contiguous()))
        mag.append(torch.matmul(p, kv[:, :rank].abs().contiguous()))
        t += m
    return torch.cat(out), torch.cat(mag)


LONG = [
    # rank, heads, page, lens, new tokens each
    (512, 64, 64, [5000], 1),              # 79 runs of one tile, joined by a workgroup per row
    (512, 64, 64, [20001], 1),             # 256 runs of one or two tiles, four turns of the join
    (256, 16, 100, [20001], 1),            # the same with 32 rows to a workgroup
    (512, 16, 16, [40000], 2),             # runs of two or three tiles, 32 rows
    (512, 64, 64, [20000, 70, 300, 1, 900], 1),   # over 256 rows: a wave per row joins some 240 runs
    (256, 64, 16, [13000, 70, 300, 1, 900], 2),
    (512, 128, 64, [5000, 333], 4),        # groups of eight workgroups, 32 runs
    (512, 128, 64, [700, 5000], 20),       # several passes over a sequence
    (512, 16, 64, [320 + i % 90 for i in range(200)], 1),  # runs over several sequences
    (256, 16, 16, [320 + i % 90 for i in range(200)], 2),
    (512, 64, 16, [1500 + 7 * i for i in range(40)], 3),
]


@pytest.mark.parametrize("rank,heads,page,lens,n", LONG)
def test_latent_attention_runs_and_joins(rank, heads, page, lens, n):
    g = gen(sum(lens) + heads)
    nq = [min(n, m) for m in lens]
    q, cache, pages, dl = long_case(g, lens, page, rank, heads, nq)
    bounds = dict(cu_q=cumulative(nq), max_q=n) if min(nq) < n else {}
    out = A.latent_attention(q, cache, pages, dl, 0.07, max_len=max(lens), **bounds)
    ref, mag = long_ref(q, cache, pages, lens, nq, 0.07, rank)
    close(out, ref, U * ref.abs() + U * mag)
    if n > 1:
        tree = torch.randint(0, 2 ** n, (sum(nq),), device=DEV, generator=g)
        out = A.latent_attention(q, cache, pages, dl, 0.07, max_len=max(lens), tree=tree, **bounds)
        ref, mag = long_ref(q, cache, pages, lens, nq, 0.07, rank, tree=tree | (torch.tensor(lens, device=DEV).repeat_interleave(
            torch.tensor(nq, device=DEV)) == 1).long())  # (a sequence of one row: its token sees itself, or nothing)
        seen = (torch.tensor(lens, device=DEV).repeat_interleave(torch.tensor(nq, device=DEV)) > 1) | (tree & 1 == 1)
        close(out[seen], ref[seen], U * ref[seen].abs() + U * mag[seen], "trees")
        assert (out[~seen] == 0).all()


@pytest.mark.parametrize("rank,heads,page,lens,n", LONG)
@pytest.mark.parametrize("falling", [False, True])
def test_latent_attention_maximum_moves(rank, heads, page, lens, n, falling):
    """Scores that rise by 6 (or fall by 6) from one tile of 64 rows to the
    next, and by less inside: the maximum moves in every tile of a run, or
    only in its first."""
    g = gen(sum(lens) + heads + 1)
    nq = [min(n, m) for m in lens]
    q, cache, pages, dl = long_case(g, lens, page, rank, heads, nq)
    flat = cache.view(-1, rank + 64)
    flat[:, rank:] = 0.0
    for b, m in enumerate(lens):
        row = torch.arange(m, device=DEV)
        tile = (row // 64) if not falling else (m - 1) // 64 - row // 64
        at = pages[b, row // page].long() * page + row % page
        # 48 (tile / 8) + 6 (tile % 8) + up to 3, each part exact in bf16
        flat[at, rank] = (48 * (tile // 8)).to(BF)
        flat[at, rank + 1] = (6 * (tile % 8)).to(BF)
        flat[at, rank + 2] = (row % 7 * 0.5).to(BF)
    q.zero_()
    q[..., rank:rank + 3] = 1.0
    out = A.latent_attention(q, cache, pages, dl, 1.0, max_len=max(lens), **(dict(cu_q=cumulative(nq), max_q=n) if min(nq) < n else {}))
    ref, mag = long_ref(q, cache, pages, lens, nq, 1.0, rank)
    # scores up to S are exact; times log2 e in fp32 they are off by S 1.44 2^-24, twice (the maximum's too), and exponentials with them
    S = 48.0 * (max(lens) // 512 + 1)
    close(out, ref, U * ref.abs() + (U + S * 2.0 ** -22) * mag)
