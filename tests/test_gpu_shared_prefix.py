"""Latent attention over the cache in 8 bits, and of sequences that share
prefixes, against the definitions in 64 bits.

Tolerance, as for the bf16 cache without prefixes (values of the 8-bit cache
are exact, and the sums that are joined are fp32): U |ref| + U sum_j p_j |v_j|
with U = 2^-8, twice one bf16 rounding, for the output and for each weight.
Beside that a weight, or its product with a row's power of two, may be below
2^-126, where fp32 and bf16 (8 bits of exponent) end, and count as nothing: of
each key at most 448 (the largest code) x 2^-126, and as much in the bf16
cache, whose values here are below 448."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U, DEV = 2.0 ** -8, "cuda:0"
BF, D, I32 = torch.bfloat16, torch.float64, torch.int32
FAR = 2 ** 30  # a page number outside the pool


@pytest.fixture(scope="module")
def A():
    from routed_expert_int4_amd import attention
    return attention


def ints(values):
    return torch.tensor(values, dtype=I32, device=DEV)


class Case:
    """Sequences of lens rows with nq new tokens each, on prefixes of
    prefix_lens rows by groups (sequence bounds); rows that nobody may see are
    NaN, in the 8-bit cache with a scale of NaN too."""

    def __init__(self, lens, nq, rank=512, heads=16, page=16, narrow=False, prefix_lens=(), groups=None, tree=None, std=1.0, seed=0):
        self.g = g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.nq, self.rank, self.heads, self.page, self.narrow = list(lens), list(nq), rank, heads, page, narrow
        self.prefix_lens, self.groups, self.tree = list(prefix_lens), groups, tree
        width, all_lens = rank + 64, self.lens + self.prefix_lens
        used = [-(-n // page) for n in all_lens]
        total = sum(used) + 3
        order = torch.randperm(total, generator=g, device=DEV).to(I32)
        values = torch.full((total, page, width), float("nan"), dtype=D, device=DEV)
        self.scale_of = torch.full((total, page), float("nan"), device=DEV)
        tables, at = [], 0
        for n, u in zip(all_lens, used):
            table = torch.full((max(used, default=0) + 1,), FAR, dtype=I32, device=DEV)
            table[:u] = order[at:at + u]
            tables.append(table)
            rows = torch.randn(u * page, width, generator=g, device=DEV)
            rows[n:] = float("nan")
            scales = 2.0 ** torch.randint(-12, 3, (u * page,), generator=g, device=DEV)
            if narrow:
                rows[:, :rank] = rows[:, :rank].mul(30).to(torch.float8_e4m3fn).float()  # codes
                scales[n:] = float("nan")
                self.scale_of[order[at:at + u].long()] = scales.view(u, page)
                rows[:, :rank] *= scales[:, None]
                if n:
                    rows[:n, :rank] *= 1 / 30
                    self.scale_of[order[at:at + u].long()] *= 1.0
            values[order[at:at + u].long()] = rows.to(BF).to(D).view(u, page, width)
            at += u
        if narrow:  # codes as drawn; a power of two near 1 / 30 makes values of about one
            self.scale_of = self.scale_of / 32
            codes = (values[..., :rank] * 30 / (self.scale_of.to(D) * 32)[..., None])
            codes = codes.float().to(torch.float8_e4m3fn)
            values[..., :rank] = codes.to(D) * self.scale_of.to(D)[..., None]
            self.cache = torch.cat([codes.view(torch.uint8), values[..., rank:].to(BF).view(torch.uint8)], -1).contiguous()
        else:
            self.cache = values.to(BF)
        self.values = values
        B = len(self.lens)
        self.pages = torch.stack(tables[:B])
        self.prefix_pages = torch.stack(tables[B:]) if self.prefix_lens else None
        self.q = (torch.randn(sum(self.nq), heads, width, generator=g, device=DEV) * std).to(BF)
        self.softmax_scale = 0.07

    def prefix(self, A, max_len=None):
        if not self.prefix_lens:
            return None
        groups = None if self.groups is None else ints(self.groups)
        return A.SharedPrefix(self.prefix_pages, ints(self.prefix_lens), max(self.prefix_lens) if max_len is None else max_len, groups)

    def run(self, A, **more):
        even = len(set(self.nq)) == 1
        keys = dict(max_len=max(self.lens), cache_scale=self.scale_of if self.narrow else None, prefix=self.prefix(A), tree=self.tree)
        if not even:
            keys |= dict(cu_q=ints([sum(self.nq[:i]) for i in range(len(self.nq) + 1)]), max_q=max(self.nq))
        return A.latent_attention(self.q, self.cache, self.pages, ints(self.lens), self.softmax_scale, **(keys | more))

    def rows(self, table, n):
        at = torch.arange(n, device=DEV)
        pages = table[at // self.page].long()
        ok = (pages >= 0) & (pages < self.values.shape[0])
        return self.values[pages.clamp(0, self.values.shape[0] - 1), at % self.page], ok

    def group_of(self, b):
        if not self.prefix_lens:
            return None
        if self.groups is None:
            return 0
        return next((i for i in range(len(self.prefix_lens)) if self.groups[i] <= b < self.groups[i + 1]), None)

    def check(self, out):
        t = 0
        for b, (n, new) in enumerate(zip(self.lens, self.nq)):
            own, ok = self.rows(self.pages[b], n)
            p = self.group_of(b)
            before, p_ok = self.rows(self.prefix_pages[p], self.prefix_lens[p]) if p is not None else (own[:0], ok[:0])
            for i in range(new):
                sees = ok.clone()
                for j in range(max(0, n - new), n):
                    k = j - (n - new)
                    sees[j] &= bool(int(self.tree[t]) >> k & 1) if self.tree is not None and k < 64 else (self.tree is None and k <= i)
                kv = torch.cat([before[p_ok], own[sees]])
                got = out[t].to(D)
                if len(kv) == 0:
                    assert bool((got == 0).all()), (b, i)
                else:
                    w = torch.softmax(self.q[t].to(D) @ kv.t() * self.softmax_scale, 1)
                    ref, mag = w @ kv[:, :self.rank], w @ kv[:, :self.rank].abs()
                    over = (got - ref).abs() - U * (ref.abs() + mag) - len(kv) * 448 * 2.0 ** -126
                    assert bool(torch.isfinite(got).all()) and float(over.max()) <= 0, (b, i, float(over.max()))
                t += 1


def trees(nq, seed):
    g = torch.Generator().manual_seed(seed)
    rows = []
    for n in nq:
        masks = []
        for j in range(n):
            parent = int(torch.randint(-1, j, (1,), generator=g)) if j else -1
            masks.append((masks[parent] if parent >= 0 else 0) | 1 << j)
        rows += masks
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in rows], dtype=torch.int64, device=DEV)


# ------------------------------------------------------------------ 8 bits alone
@pytest.mark.parametrize("rank", [512, 256])
@pytest.mark.parametrize("heads,page", [(1, 16), (16, 1), (64, 64), (20, 100), (128, 16)])
def test_narrow_single_tokens(A, rank, heads, page):
    lens = [1, 2, 63, 64, 65, 300, 128]
    c = Case(lens, [1] * len(lens), rank, heads, page, narrow=True, seed=heads)
    c.check(c.run(A))
    c.check(c.run(A, max_len=None))


@pytest.mark.parametrize("rank", [512, 256])
@pytest.mark.parametrize("heads,nq", [(16, 2), (16, 5), (64, 3), (4, 17), (64, 16)])
def test_narrow_chunks_and_trees(A, rank, heads, nq):
    lens = [nq, nq + 1, 100, 64 + nq // 2, 257]
    c = Case(lens, [nq] * 5, rank, heads, 16, narrow=True, seed=nq)
    c.check(c.run(A))
    c = Case(lens, [nq] * 5, rank, heads, 16, narrow=True, seed=nq, tree=trees([nq] * 5, nq))
    c.check(c.run(A))


def test_narrow_ragged_tokens(A):
    nq = [3, 0, 1, 70, 0, 2]
    c = Case([40, 100, 1, 200, 7, 0], nq, 512, 16, 64, narrow=True)
    c.check(c.run(A))


def test_narrow_sequences_without_rows_and_pages_outside(A):
    c = Case([300, 0, 64, 150], [1] * 4, 512, 64, 16, narrow=True)
    c.pages[0, 3], c.pages[2, :] = -1, FAR
    c.check(c.run(A))


@pytest.mark.parametrize("rank", [512, 256])
@pytest.mark.parametrize("lens,heads", [([9000], 64), ([5000, 70, 3000, 1, 700], 16), ([777] * 40, 64)])
def test_narrow_runs_and_joins(A, rank, lens, heads):
    c = Case(lens, [1] * len(lens), rank, heads, 64, narrow=True, seed=len(lens))
    c.check(c.run(A))


@pytest.mark.parametrize("std", [12.0, 40.0])
def test_narrow_maximum_moves(A, std):
    c = Case([700, 64, 2000], [2] * 3, 512, 64, 64, narrow=True, std=std)
    c.check(c.run(A))


@pytest.mark.parametrize("rank", [512, 256])
def test_narrow_values_that_are_not_finite_in_unseen_rows(A, rank):
    """Siblings in a tree do not see each other's codes, scales or keys."""
    tree = torch.tensor([1, 2, 4, 1, 3, 7], dtype=torch.int64, device=DEV)
    c = Case([67, 100], [3, 3], rank, 16, 16, narrow=True, tree=tree)
    want = c.run(A)
    c.check(want)
    at = c.lens[0] - 3 + 1  # the first sequence's second new token: seen by itself alone
    page, off = int(c.pages[0, at // 16]), at % 16
    for change in ("code", "scale", "infinite scale", "key"):
        cache, scale = c.cache.clone(), c.scale_of.clone()
        if change == "code":
            cache[page, off, 5:9] = torch.tensor([0x7F, 0xFF, 0x7F, 0xFF], dtype=torch.uint8, device=DEV)
        elif change == "scale":
            scale[page, off] = float("nan")
        elif change == "infinite scale":
            scale[page, off] = float("inf")
        else:
            cache[page, off, rank:] = 0xFF
        out = A.latent_attention(c.q, cache, c.pages, ints(c.lens), 0.07, max_len=100, tree=tree, cache_scale=scale)
        others = [0, 2, 3, 4, 5]
        assert torch.equal(out[others], want[others]), change
        assert not bool(torch.isfinite(out[1]).all()), change


@pytest.mark.parametrize("narrow", [True, False])
def test_views_of_wider_tensors(A, narrow):
    c = Case([40, 90], [2, 2], 256, 16, 16, narrow=narrow, prefix_lens=[130])
    want = c.run(A)
    wide = torch.full((4, 20, 400), float("nan"), dtype=BF, device=DEV)
    wide[:, 2:18, 16:336] = c.q
    out = torch.full((4, 18, 300), 7.0, dtype=BF, device=DEV)
    pool = torch.zeros(c.cache.shape[0], 2, *c.cache.shape[1:], dtype=c.cache.dtype, device=DEV)
    pool[:, 1] = c.cache
    c.q, c.cache = wide[:, 2:18, 16:336], pool[:, 1]
    got = c.run(A, out=out[:, 1:17, 4:260])
    assert torch.equal(got, want)
    out[:, 1:17, 4:260] = 7.0
    assert bool((out == 7).all())


# ------------------------------------------------------------------ prefixes
@pytest.mark.parametrize("narrow", [True, False])
@pytest.mark.parametrize("prefix", [1, 63, 64, 65, 517, 2000])
@pytest.mark.parametrize("rank,heads,page", [(512, 64, 64), (256, 16, 16), (512, 1, 100)])
def test_one_prefix_for_all(A, narrow, prefix, rank, heads, page):
    lens = [1, 40, 64, 130]
    c = Case(lens, [1] * 4, rank, heads, page, narrow, [prefix], seed=prefix)
    c.check(c.run(A))


@pytest.mark.parametrize("narrow", [True, False])
@pytest.mark.parametrize("heads,nq", [(16, 3), (64, 4), (64, 17), (128, 7)])
def test_chunks_and_trees_on_prefixes(A, narrow, heads, nq):
    lens = [nq, nq + 30, 64, 200 + nq]
    c = Case(lens, [nq] * 4, 512, heads, 16, narrow, [300, 70], [0, 1, 4], seed=nq)
    c.check(c.run(A))
    c = Case(lens, [nq] * 4, 512, heads, 16, narrow, [300, 70], [0, 3, 4], tree=trees([nq] * 4, nq), seed=nq)
    c.check(c.run(A))


@pytest.mark.parametrize("narrow", [True, False])
@pytest.mark.parametrize("groups", [[0, 2, 6], [1, 3, 4], [0, 0, 6], [0, 6, 6], [2, 2, 2], [0, 3, 100], [-5, 2, 5]])
def test_groups(A, narrow, groups):
    """Sequences outside all groups, groups without sequences, bounds past the last one."""
    c = Case([20, 65, 3, 150, 1, 64], [1] * 6, 512, 16, 16, narrow, [100, 333], groups)
    c.check(c.run(A))


def test_groups_that_overlap_are_unseen(A):
    """More tokens in groups than there are: no prefix is seen, nothing else changes."""
    c = Case([20, 65, 3], [2] * 3, 512, 16, 16, False, [100, 333, 50], [0, 3, 0, 3])
    out = c.run(A)
    c.prefix_lens = []
    c.check(out)


def test_bounds_that_decrease(A):
    """What lies outside its group has no prefix; no address is made of it."""
    c = Case([20, 65, 30, 40], [0, 2, 0, 4], 512, 16, 16, False, [100], [0, 3])
    out = A.latent_attention(c.q, c.cache, c.pages, ints(c.lens), 0.07, max_len=65, cu_q=ints([4, 0, 2, 6, 6]), max_q=6, prefix=c.prefix(A))
    assert out.shape == (6, 16, 512)
    torch.cuda.synchronize()


def test_many_groups(A):
    n = 150
    c = Case([1 + i % 5 for i in range(n)], [1] * n, 256, 16, 16, True, [1 + (i * 37) % 90 for i in range(n // 2)],
             [2 * i for i in range(n // 2 + 1)])
    c.check(c.run(A))


@pytest.mark.parametrize("narrow", [True, False])
def test_sequences_without_rows_of_their_own(A, narrow):
    c = Case([0, 0, 10], [1, 1, 1], 512, 64, 16, narrow, [200])
    c.check(c.run(A))
    c = Case([0, 5, 0], [1, 1, 1], 512, 64, 16, narrow, [0, 70], [0, 2, 3])
    c.check(c.run(A))  # the first sees nothing


@pytest.mark.parametrize("narrow", [True, False])
def test_ragged_tokens_on_prefixes(A, narrow):
    nq = [3, 0, 1, 70, 0, 2]
    c = Case([40, 100, 1, 200, 7, 5], nq, 512, 16, 64, narrow, [99, 500], [0, 3, 6])
    c.check(c.run(A))


def test_prefix_pages_outside_the_pool(A):
    c = Case([20, 30], [1, 1], 512, 64, 16, False, [200])
    c.prefix_pages[0, 2], c.prefix_pages[0, 7] = -1, FAR
    c.check(c.run(A))


@pytest.mark.parametrize("narrow", [True, False])
@pytest.mark.parametrize("B,nq,heads,prefix,most", [(33, 1, 64, 3000, 700), (3, 1, 64, 9000, 10), (50, 1, 16, 100, 900), (9, 4, 64, 2000, 300),
                                                    (70, 1, 128, 1000, 65)])
def test_many_runs(A, narrow, B, nq, heads, prefix, most):
    g = torch.Generator().manual_seed(B)
    lens = [nq + int(x) for x in torch.randint(0, most, (B,), generator=g)]
    groups = [0, B // 3, B]
    c = Case(lens, [nq] * B, 512, heads, 64, narrow, [prefix, prefix // 3], groups, seed=B)
    c.check(c.run(A))


@pytest.mark.parametrize("narrow", [True, False])
@pytest.mark.parametrize("std", [12.0, 40.0])
def test_maximum_moves_between_prefix_and_own_rows(A, narrow, std):
    c = Case([700, 64, 300], [2] * 3, 512, 64, 64, narrow, [500, 1000], [0, 1, 3], std=std)
    c.check(c.run(A))


def test_bounds_given_too_small_or_not_at_all(A):
    c = Case([100, 200], [1, 1], 512, 64, 16, False, [900])
    want = c.run(A)
    c.check(want)
    c.check(A.latent_attention(c.q, c.cache, c.pages, ints(c.lens), 0.07, prefix=c.prefix(A, max_len=1), max_len=1))
    c.check(A.latent_attention(c.q, c.cache, c.pages, ints(c.lens), 0.07, prefix=A.SharedPrefix(c.prefix_pages, ints([900]))))


@pytest.mark.parametrize("narrow", [True, False])
def test_as_one_long_sequence_each(A, narrow):
    """The same rows through the page tables of separate sequences."""
    c = Case([30, 100, 64], [1] * 3, 512, 64, 16, narrow, [160])
    got = c.run(A)
    pages = torch.cat([c.prefix_pages[:, :10].expand(3, -1), c.pages], 1).contiguous()
    lens = [n + 160 for n in c.lens]
    want = A.latent_attention(c.q, c.cache, pages, ints(lens), 0.07, max_len=max(lens), cache_scale=c.scale_of if narrow else None)
    c.check(got)
    c.check(want)


@pytest.mark.parametrize("narrow", [True, False])
def test_replayed_with_other_lengths(A, narrow):
    """Lengths, pages and groups are read on the device: a captured call follows them."""
    c = Case([30, 150, 64, 90], [1] * 4, 512, 64, 16, narrow, [160, 300], [0, 2, 4])
    lens, p = ints(c.lens), c.prefix(A)
    from routed_expert_int4_amd import binding as B
    size = B.lib().moe_latent_attention_shared_workspace(4, 4, 1, 64, 512, 150, 2, 300)
    out, ws = torch.zeros(4, 64, 512, dtype=BF, device=DEV), torch.empty(size, dtype=torch.uint8, device=DEV)

    def step():
        A.latent_attention(c.q, c.cache, c.pages, lens, 0.07, max_len=150, prefix=p, out=out, workspace=ws,
                           cache_scale=c.scale_of if narrow else None)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for own, prefixes, groups in (([30, 150, 64, 90], [160, 300], [0, 2, 4]), ([1, 2, 3, 4], [5, 299], [0, 1, 4]),
                                  ([29, 64, 1, 65], [160, 1], [0, 4, 4])):
        c.lens, c.prefix_lens, c.groups = own, prefixes, groups
        lens.copy_(ints(own))
        p.lens.copy_(ints(prefixes))
        p.groups.copy_(ints(groups))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        c.check(got)
        out.zero_()
        step()
        assert torch.equal(out, got)


def test_on_another_stream_and_repeated(A):
    c = Case([300] * 9, [2] * 9, 512, 64, 64, True, [1500, 100], [0, 5, 9])
    want = c.run(A)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = [c.run(A, stream=stream) for _ in range(3)]
    stream.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_no_tokens(A):
    c = Case([5], [1], 512, 16, 16, True, [10])
    out = A.latent_attention(c.q[:0], c.cache, c.pages[:0], ints([]), 0.07, cache_scale=c.scale_of, prefix=c.prefix(A))
    assert out.shape == (0, 16, 512)
