"""GPU tests of the attention half of a block (routed_expert_int4_amd/attention.py)
against plain implementations in 64 bits, written from the definitions.

Tolerances, element by element.  U = 2^-8 is one bf16 rounding at its worst
(half a unit in the last of 8 bits, 2^-9) with as much again for fp32
arithmetic and the hardware exponential.
  bf16 outputs of sums:   U |ref| + 1e-5 sum |terms|   (fp32 sums; the 8-bit
      matrix unit adds a block of 128 with a relative error near 1e-5: 3e-5)
  attention:              U |ref| + U sum_j p_j |v_j|  (each exponential is
      rounded to bf16 once, so each term moves by at most 2^-9 of itself)
  8-bit codes:            half a step of E4M3 around the unrounded value
      (2^-4 of it, 2^-10 below the smallest normal) and 1e-5 for a value that
      fp32 arithmetic moves across a tie
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_int4_amd import attention as A  # noqa: E402
from routed_expert_int4_amd import binding as B  # noqa: E402

U = 2.0 ** -8
DEV = "cuda:0"
D = torch.float64
BF = torch.bfloat16


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=BF):
    return torch.empty(*shape, device=DEV, dtype=torch.float32).normal_(0.0, std, generator=g).to(dtype)


def close(got, ref, tol, what=""):
    got = got.to(D)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - tol
    worst = over.max().item() if over.numel() else -1.0
    assert worst <= 0.0, f"{what}: off by {worst:.3g} more than allowed at {(over == over.max()).nonzero()[0].tolist()}"


def strided(t, pad):
    """The same values in rows `pad` elements longer."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), float("nan"), dtype=torch.float32, device=DEV).to(t.dtype)
    view = wide[..., : t.shape[-1]]
    view.copy_(t)
    return view


# ---------------------------------------------------------------- norm
def norm_ref(x, residual, weight, eps):
    h = x.to(D) + (residual.to(D) if residual is not None else 0.0)
    return h, h / (h.pow(2).mean(1, keepdim=True) + eps).sqrt() * weight.to(D)


def check_codes(q, scale, y):
    T, H = y.shape
    groups = [y[:, i:i + 128] for i in range(0, H, 128)]
    want = torch.stack([p.abs().amax(1) for p in groups], 1) / 448
    close(scale, want, 1e-5 * want + 1e-12, "scale")
    for i, p in enumerate(groups):
        v = q[:, i * 128:i * 128 + 128].to(D)
        s = scale[:, i:i + 1].to(D)
        x = p / s
        assert v.isfinite().all()
        step = torch.maximum(x.abs() * 2 ** -4, torch.full_like(x, 2.0 ** -10))
        close(v, x, step * (1 + 1e-5) + 1e-5 * x.abs(), f"codes of group {i}")


@pytest.mark.parametrize("T", [1, 3, 700])
@pytest.mark.parametrize("H", [1, 7, 128, 136, 1000, 2048, 6144, 8200, 32768])
def test_add_rmsnorm_shapes(T, H):
    if T * H > 8e6:
        T = 33
    g = gen(T * 7 + H)
    x = normal(g, T, H, std=0.5, dtype=torch.float32)
    r, w = normal(g, T, H, std=2.0), normal(g, H, std=0.3)
    out = A.add_rmsnorm(x, w, 1e-6, residual=r, out="both")
    h, y = norm_ref(x, r, w, 1e-6)
    close(out.sum, h, U * h.abs() + 1e-6, "sum")
    close(out.y, y, U * y.abs() + 1e-12, "y")
    check_codes(out.q, out.scale, y)


@pytest.mark.parametrize("xt", [torch.float32, BF])
@pytest.mark.parametrize("rt", [None, torch.float32, BF])
@pytest.mark.parametrize("wt", [torch.float32, BF])
def test_add_rmsnorm_types_and_strides(xt, rt, wt):
    g = gen(3)
    for T, H, pad in ((5, 1024, 8), (5, 1024, 3), (2, 300, 1), (600, 2056, 16)):
        x = strided(normal(g, T, H, dtype=xt), pad)
        r = strided(normal(g, T, H, dtype=rt), pad) if rt else None
        w = normal(g, H, dtype=wt)
        out = A.add_rmsnorm(x, w, 1e-5, residual=r, out="both")
        h, y = norm_ref(x, r, w, 1e-5)
        if rt is not None:
            assert out.sum.dtype == rt
            close(out.sum, h, (U if rt == BF else 2e-7) * h.abs() + 1e-6, "sum")
        else:
            assert out.sum is None
        close(out.y, y, U * y.abs(), "y")
        check_codes(out.q, out.scale, y)


def test_add_rmsnorm_in_place_and_single_outputs():
    g = gen(4)
    x, r, w = normal(g, 9, 6144), normal(g, 9, 6144), normal(g, 6144)
    h, y = norm_ref(x, r, w, 1e-6)
    one = A.add_rmsnorm(x, w, residual=r, out="bf16")
    keep = r.clone()
    two = A.add_rmsnorm(x, w, residual=r, out="fp8", sum_out=r)
    assert two.sum is r and two.y is None and one.q is None
    assert torch.equal(r, one.sum) and not torch.equal(r, keep)
    check_codes(two.q, two.scale, y)
    none = A.add_rmsnorm(x, w, residual=keep, out="bf16", want_sum=False)
    assert none.sum is None and torch.equal(none.y, one.y)


def test_add_rmsnorm_extremes():
    g = gen(5)
    w = normal(g, 512).abs() + 0.5
    x = normal(g, 6, 512, dtype=torch.float32)
    x[0] = 0.0                       # nothing: scales at their least, codes zero
    x[1] *= 1e15                     # the square still fits
    x[2] *= 1e-18
    x[3, 130] = float("nan")
    x[4, 3] = float("inf")
    out = A.add_rmsnorm(x, w, 1e-6, out="both")
    h, y = norm_ref(x[:3], None, w, 1e-6)
    close(out.y[:3], y, U * y.abs() + 1e-30, "y")
    assert (out.q[0].float() == 0).all() and (out.scale[0] == 1e-12).all()
    check_codes(out.q[1:2], out.scale[1:2], y[1:2])
    # a NaN spreads over its row, in every output
    assert out.y[3].isnan().all() and out.q[3].float().isnan().all() and out.scale[3].isnan().all()
    # an infinity makes itself NaN and the others zero
    assert out.y[4, 3].isnan() and (out.y[4, 4:] == 0).all() and out.scale[4, 0].isnan() and out.scale[4, 1] == 1e-12


# ---------------------------------------------------------------- 8-bit product
def fp8_inputs(g, M, N, K, pad=0):
    kb, nb = -(-K // 128), -(-N // 128)
    a = strided(normal(g, M, K, std=60.0).float().clamp(-448, 448).to(torch.float8_e4m3fn).float(), pad).to(torch.float8_e4m3fn) \
        if pad else normal(g, M, K, std=60.0).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    w = normal(g, N, K, std=60.0).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    sa = torch.empty(M, kb, device=DEV).uniform_(0.5, 2.0, generator=g) * 0.01
    sw = torch.empty(nb, kb, device=DEV).uniform_(0.5, 2.0, generator=g) * 0.01
    return a, sa, w, sw


def fp8_ref(a, sa, w, sw):
    (M, K), N = a.shape, w.shape[0]
    x = a.to(D) * sa.to(D).repeat_interleave(128, 1)[:, :K]
    y = w.to(D) * sw.to(D).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return x @ y.t(), x.abs() @ y.abs().t()


@pytest.mark.parametrize("M", [1, 2, 16, 17, 63, 65, 127, 128, 200, 300, 513])
@pytest.mark.parametrize("N,K", [(1, 16), (576, 1024), (130, 144), (1000, 400), (256, 2048), (128, 128), (515, 1168)])
def test_fp8_linear_shapes(M, N, K):
    a, sa, w, sw = fp8_inputs(gen(M * 31 + N + K), M, N, K)
    ref, mag = fp8_ref(a, sa, w, sw)
    close(A.fp8_linear(a, sa, w, sw), ref, U * ref.abs() + 3e-5 * mag, "bf16")
    # scales stored group by group, and fp32 output
    out = A.fp8_linear(a, sa.t().contiguous().t(), w, sw, out_dtype=torch.float32)
    close(out, ref, 3e-5 * mag, "fp32")


@pytest.mark.parametrize("M", [5, 40, 300, 1100])
def test_fp8_linear_strides_and_views(M):
    g = gen(M)
    N, K = 392, 656
    a, sa, w, sw = fp8_inputs(g, M, N, K)
    wide = torch.full((M, K + 48), 0x7F, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # NaN around the rows
    wide.view(torch.uint8)[:, :K] = a.view(torch.uint8)
    wide_w = torch.full((N, K + 16), 0x7F, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    wide_w.view(torch.uint8)[:, :K] = w.view(torch.uint8)
    ref, mag = fp8_ref(a, sa, w, sw)
    for extra in (0, 1, 4):
        out = torch.full((M, N + extra), -7.0, dtype=BF, device=DEV)
        A.fp8_linear(wide[:, :K], sa, wide_w[:, :K], sw, out=out[:, :N])
        close(out[:, :N], ref, U * ref.abs() + 3e-5 * mag, f"row of {N + extra}")
        assert (out[:, N:] == -7.0).all()


def test_fp8_linear_extremes():
    a, sa, w, sw = fp8_inputs(gen(9), 70, 140, 272)
    for M in (70, 3):
        x = a[:M].clone()
        x.view(torch.uint8)[1, 200] = 0x7F  # NaN in one row
        out = A.fp8_linear(x, sa[:M], w, sw)
        assert out[1].isnan().all() and out[0].isfinite().all() and out[2:].isfinite().all()
        s = sa[:M].clone()
        s[0, 1] = float("inf")
        out = A.fp8_linear(a[:M], s, w, sw)
        assert not out[0].isfinite().any() and out[1:].isfinite().all()
        zero = A.fp8_linear(torch.zeros_like(a[:M].view(torch.uint8)).view(torch.float8_e4m3fn), sa[:M], w, sw)
        assert (zero == 0).all()


# ---------------------------------------------------------------- per-head product
@pytest.mark.parametrize("T", [0, 1, 2, 16, 17, 64, 65, 200])
@pytest.mark.parametrize("heads,K,N", [(1, 8, 4), (3, 128, 512), (16, 512, 128), (5, 72, 36), (2, 200, 300)])
def test_head_linear(T, heads, K, N):
    g = gen(T + K)
    wide = strided(normal(g, T, heads, K), 24)
    w = normal(g, heads, N, K, std=K ** -0.5)
    out = torch.full((T, heads, N + 12), -7.0, dtype=BF, device=DEV)
    A.head_linear(wide, w, out=out[..., :N])
    ref = torch.einsum("thk,hnk->thn", wide.cpu().to(D), w.cpu().to(D)).to(DEV)
    mag = torch.einsum("thk,hnk->thn", wide.cpu().to(D).abs(), w.cpu().to(D).abs()).to(DEV)
    close(out[..., :N], ref, U * ref.abs() + 1e-5 * mag)
    assert (out[..., N:] == -7.0).all()


# ---------------------------------------------------------------- cache write
def rope_table(n, rope, base=10000.0):
    angle = torch.arange(n, dtype=D)[:, None] * base ** (-torch.arange(0, rope, 2, dtype=D) / rope)
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV)


def rotate_ref(x, row):
    c, s = row.to(D).chunk(2, -1)
    e, o = x.to(D)[..., 0::2], x.to(D)[..., 1::2]
    return torch.stack([e * c - o * s, e * s + o * c], -1).flatten(-2), torch.stack([(e * c).abs() + (o * s).abs()] * 2, -1).flatten(-2)


@pytest.mark.parametrize("T", [1, 5, 300])
@pytest.mark.parametrize("rank,rope,heads,page", [(512, 64, 64, 64), (256, 64, 3, 16), (8, 8, 1, 1), (2048, 32, 5, 7), (520, 24, 2, 100)])
def test_latent_append(T, rank, rope, heads, page):
    g = gen(T + rank)
    pages = T // page + 4
    kv = strided(normal(g, T, rank + rope), 8)
    w = normal(g, rank, dtype=torch.float32 if T == 5 else BF)
    table = rope_table(500, rope)
    positions = torch.randint(0, 500, (T,), device=DEV, generator=g, dtype=torch.int32)
    slots = torch.randperm(pages * page, device=DEV, generator=g)[:T].contiguous()
    q = strided(normal(g, T, heads, rope), 8)
    cache = torch.full((pages, page, rank + rope), -7.0, dtype=BF, device=DEV)
    slots[T // 2] = -1                      # not written
    if T > 2:
        slots[0] = pages * page             # past the pool: not written
    res = A.latent_append(kv, w, 1e-6, table, positions, slots, cache, q_rope=q, want_fp8=True, want_key=True)
    _, y = norm_ref(kv[:, :rank], None, w, 1e-6)
    row = table[positions.long()]
    key, key_mag = rotate_ref(kv[:, rank:], row)
    turned, mag = rotate_ref(q, row[:, None])
    ok = (slots >= 0) & (slots < pages * page)
    flat = cache.view(-1, rank + rope)
    close(flat[slots[ok], :rank], y[ok], U * y[ok].abs(), "latent")
    close(flat[slots[ok], rank:], key[ok], U * key[ok].abs() + 1e-6 * key_mag[ok], "key")
    rest = torch.ones(pages * page, dtype=torch.bool, device=DEV)
    rest[slots[ok]] = False
    assert (flat[rest] == -7.0).all(), "rows that no token owns are untouched"
    close(res.q_rope, turned, U * turned.abs() + 1e-6 * mag, "queries")
    close(res.key, key, U * key.abs() + 1e-6 * key_mag, "key copy")
    check_codes(res.q, res.scale, y)
    again = A.latent_append(kv, w, 1e-6, table, positions, slots, cache, q_rope=q, q_out=q)
    assert again.q_rope is q and torch.equal(q, res.q_rope), "rotation in place"


def test_latent_append_unknown_position():
    g = gen(1)
    kv, w, table = normal(g, 3, 320), normal(g, 256), rope_table(10, 64)
    positions = torch.tensor([3, 10, -1], dtype=torch.int32, device=DEV)
    slots = torch.tensor([0, 1, 2], device=DEV)
    cache = torch.zeros(1, 4, 320, dtype=BF, device=DEV)
    A.latent_append(kv, w, 1e-6, table, positions, slots, cache)
    assert cache[0, 0].isfinite().all() and cache[0, 1:3, 256:].isnan().all() and cache[0, 1:3, :256].isfinite().all()


# ---------------------------------------------------------------- absorbed attention
def softmax_ref(scores, values):
    """(sum p v, sum p |v|); zeros where no score is left (scores: [rows, keys] of the visible keys only)."""
    if scores.shape[1] == 0:
        z = torch.zeros(scores.shape[0], values.shape[1], dtype=D, device=values.device)
        return z, z
    p = torch.softmax(scores, 1)
    return p @ values, p @ values.abs()


def latent_ref(q, cache, pages, lens, nq, scale, rank, tree=None):
    out, mag, t = [], [], 0
    page = cache.shape[1]
    for b, n in enumerate(lens):
        index = [int(pages[b, j // page]) * page + j % page if 0 <= int(pages[b, j // page]) < cache.shape[0] else -1
                 for j in range(n)]
        rows = torch.tensor(index, dtype=torch.long, device=DEV)
        kv = cache.reshape(-1, cache.shape[2])[rows.clamp_min(0)].to(D)
        for i in range(nq[b]):
            sees = rows >= 0
            for j in range(max(0, n - nq[b]), n):
                k = j - (n - nq[b])
                sees[j] &= bool(int(tree[t]) >> k & 1) if tree is not None and k < 64 else (tree is None and k <= i)
            o, m = softmax_ref((q[t].to(D) @ kv[sees].t()) * scale, kv[sees][:, :rank])
            out.append(o)
            mag.append(m)
            t += 1
    return torch.stack(out), torch.stack(mag)


def latent_case(g, lens, nq, heads, rank, page, spare=3, q_pad=0, std=1.0):
    width = rank + 64
    used = [-(-n // page) for n in lens]
    total = sum(used) + spare
    cache = torch.full((total, page, width), float("nan"), dtype=BF, device=DEV)
    order = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    pages = torch.full((len(lens), max(max(used), 1) + 1), 2 ** 30, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(lens):  # rows past a sequence's end stay NaN
        pages[b, :used[b]] = order[at:at + used[b]]
        for i in range(used[b]):
            m = min(page, n - i * page)
            cache[int(order[at + i]), :m] = normal(g, m, width)
        at += used[b]
    q = strided(normal(g, sum(nq), heads, width, std=std), q_pad) if q_pad else normal(g, sum(nq), heads, width, std=std)
    return q, cache, pages, torch.tensor(lens, dtype=torch.int32, device=DEV)


def cumulative(n):
    return torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("rank", [512, 256])
@pytest.mark.parametrize("heads", [1, 16, 48, 64, 128])
@pytest.mark.parametrize("page", [1, 16, 64, 100])
def test_latent_attention_decode(rank, heads, page):
    g = gen(heads + page)
    lens = [1, 63, 64, 65, 200, 1000, 0, 129]
    q, cache, pages, dl = latent_case(g, lens, [1] * len(lens), heads, rank, page)
    out = A.latent_attention(q, cache, pages, dl, 0.07, max_len=max(lens))
    ref, mag = latent_ref(q, cache, pages, lens, [1] * len(lens), 0.07, rank)
    close(out, ref, U * ref.abs() + U * mag)
    assert (out[6] == 0).all(), "an empty sequence gives zeros"
    # without a bound the call covers the page table's reach, with the same result up to where it is cut
    wide = A.latent_attention(q, cache, pages, dl, 0.07)
    close(wide, ref, U * ref.abs() + U * mag)


@pytest.mark.parametrize("heads,nq", [(64, 4), (16, 2), (64, 1), (3, 17), (128, 2), (64, 33)])
def test_latent_attention_chunks_and_trees(heads, nq):
    g = gen(heads * 3 + nq)
    lens = [nq, nq + 1, 500, 64 + nq, 130, max(1, nq - 1)]  # the last has fewer rows than tokens
    n = [nq] * len(lens)
    q, cache, pages, dl = latent_case(g, lens, n, heads, 512, 16, q_pad=8)
    out = A.latent_attention(q, cache, pages, dl, 0.07, max_len=500)
    ref, mag = latent_ref(q, cache, pages, lens, n, 0.07, 512)
    close(out, ref, U * ref.abs() + U * mag, "causal")
    bits = torch.randint(0, 2 ** min(nq, 62), (sum(n),), device=DEV, generator=g)
    bits[0] = 0  # sees only the context: nothing in the first sequence
    out = A.latent_attention(q, cache, pages, dl, 0.07, max_len=500, tree=bits)
    ref, mag = latent_ref(q, cache, pages, lens, n, 0.07, 512, tree=bits)
    close(out, ref, U * ref.abs() + U * mag, "tree")
    assert (out[0] == 0).all(), "a row whose mask leaves nothing gives zeros"


def test_latent_attention_ragged_queries():
    g = gen(12)
    nq, lens = [0, 3, 1, 70, 0, 9], [10, 40, 1, 300, 0, 9]
    q, cache, pages, dl = latent_case(g, lens, nq, 64, 512, 64)
    out = A.latent_attention(q, cache, pages, dl, 0.07, max_len=300, cu_q=cumulative(nq), max_q=70)
    ref, mag = latent_ref(q, cache, pages, lens, nq, 0.07, 512)
    close(out, ref, U * ref.abs() + U * mag)


def test_latent_attention_many_sequences():
    g = gen(13)
    lens = [(i * 37) % 260 + 1 for i in range(150)]
    q, cache, pages, dl = latent_case(g, lens, [1] * 150, 16, 256, 32)
    out = A.latent_attention(q, cache, pages, dl, 0.07, max_len=260)
    ref, mag = latent_ref(q, cache, pages, lens, [1] * 150, 0.07, 256)
    close(out, ref, U * ref.abs() + U * mag)


def test_latent_attention_pages_outside_the_pool():
    g = gen(14)
    lens = [300, 200]
    q, cache, pages, dl = latent_case(g, lens, [2, 2], 64, 512, 16)
    pages[0, 3], pages[0, 7], pages[1, 0] = -1, cache.shape[0], -2 ** 31
    pages[1, 12] = 2 ** 30  # the last rows of the second sequence, its new tokens among them
    out = A.latent_attention(q, cache, pages, dl, 0.07, max_len=300)
    ref, mag = latent_ref(q, cache, pages, lens, [2, 2], 0.07, 512)
    close(out, ref, U * ref.abs() + U * mag)


def test_latent_attention_large_scores():
    # scores of hundreds: the maximum moves in almost every tile, single keys win
    g = gen(15)
    lens = [700, 90]
    q, cache, pages, dl = latent_case(g, lens, [1, 1], 64, 512, 64, std=12.0)
    out = A.latent_attention(q, cache, pages, dl, 1.0, max_len=700)
    ref, mag = latent_ref(q, cache, pages, lens, [1, 1], 1.0, 512)
    # fp32 scores near 1000 are off by about 1e-4, and so are their exponentials
    close(out, ref, U * ref.abs() + U * mag + 1e-3 * mag)
    # ascending scores: each key beats all before it
    cache.zero_()
    rows = torch.arange(700, device=DEV)
    at = pages[0, rows // 64].long() * 64 + rows % 64
    cache.view(-1, 576)[at, 0] = (rows.float() / 4).to(BF)
    cache.view(-1, 576)[at, 1] = normal(g, 700)
    q.zero_()
    q[:, :, 0] = 1.0
    out = A.latent_attention(q, cache, pages, dl, 1.0, max_len=700)
    ref, mag = latent_ref(q, cache, pages, lens, [1, 1], 1.0, 512)
    close(out, ref, U * ref.abs() + U * mag + 1e-5)


def test_latent_attention_cache_past_32_bits():
    # pages beyond 2^32 bytes (and 2^31 elements) into the pool
    g = gen(16)
    n_pages = (2 ** 32 + 2 ** 28) // (576 * 64 * 2)
    cache = torch.empty(n_pages, 64, 576, dtype=BF, device=DEV)
    last = [n_pages - 1, n_pages - 5, 0, n_pages // 2 + 9]
    for p in last:
        cache[p] = normal(g, 64, 576)
    pages = torch.tensor([last], dtype=torch.int32, device=DEV)
    lens = torch.tensor([251], dtype=torch.int32, device=DEV)
    q = normal(g, 1, 64, 576)
    out = A.latent_attention(q, cache, pages, lens, 0.07, max_len=251)
    ref, mag = latent_ref(q, cache, pages, [251], [1], 0.07, 512)
    close(out, ref, U * ref.abs() + U * mag)
    slots = torch.tensor([(n_pages - 3) * 64 + 5], device=DEV)
    A.latent_append(normal(g, 1, 576), normal(g, 512), 1e-6, rope_table(4, 64), torch.zeros(1, dtype=torch.int32, device=DEV), slots, cache)
    assert cache[n_pages - 3, 5].isfinite().all() and (cache[n_pages - 3, 5] != 0).any()


def test_latent_attention_repeats_and_streams():
    # the same call gives the same bits, also on another stream and in a graph
    g = gen(17)
    lens = [900, 333, 64]
    q, cache, pages, dl = latent_case(g, lens, [2] * 3, 64, 512, 64)
    first = A.latent_attention(q, cache, pages, dl, 0.07, max_len=900)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = A.latent_attention(q, cache, pages, dl, 0.07, max_len=900)
    side.synchronize()
    assert torch.equal(first, again)
    ws = torch.empty(B.lib().moe_latent_attention_workspace(3, 2, 64, 512, 900), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.latent_attention(q, cache, pages, dl, 0.07, max_len=900, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)


def test_calls_on_a_given_stream():
    # while `stream` is still busy, the current stream gets none of the memory
    # that a call on it has taken or still reads
    g = gen(18)
    q, cache, pages, dl = latent_case(g, [900, 333, 64], [2] * 3, 64, 512, 64)
    x, w, res = normal(g, 512, 2048), normal(g, 2048), normal(g, 512, 2048)
    k, v, kr = normal(g, 700, 4, 128), normal(g, 700, 4, 128), normal(g, 700, 64)
    pq = normal(g, 700, 4, 192)
    first = A.latent_attention(q, cache, pages, dl, 0.07, max_len=900)
    norm = A.add_rmsnorm(x, w, residual=res, out="both")
    prompt = A.prompt_attention(pq, k, kr, v, 0.07)
    busy = normal(g, 4096, 4096)
    torch.cuda.synchronize()
    for as_handle in (False, True):
        side = torch.cuda.Stream()
        stream = side.cuda_stream if as_handle else side
        with torch.cuda.stream(side):
            for _ in range(50):
                busy @ busy
        got = A.latent_attention(q, cache, pages, dl, 0.07, max_len=900, stream=stream)
        got_norm = A.add_rmsnorm(x, w, residual=res, out="both", stream=stream)
        got_prompt = A.prompt_attention(pq, k, kr, v, 0.07, stream=stream)
        size = B.lib().moe_latent_attention_workspace(3, 2, 64, 512, 900)
        mine = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(bool((m == 7).all()) for m in mine)
        assert torch.equal(got, first) and torch.equal(got_prompt, prompt)
        assert all(torch.equal(a.float(), b.float()) for a, b in zip(got_norm, norm))


# ---------------------------------------------------------------- expanded attention
def prompt_ref(q, k, kr, v, nq, nk, scale, causal=True):
    out, mag = [], []
    q0 = k0 = 0
    for n, m in zip(nq, nk):
        s = torch.matmul(q[q0:q0 + n, :, :k.shape[2]].to(D).transpose(0, 1).contiguous(),
                         k[k0:k0 + m].to(D).permute(1, 2, 0).contiguous())
        s = (s + torch.matmul(q[q0:q0 + n, :, k.shape[2]:].to(D).transpose(0, 1).contiguous(), kr[k0:k0 + m].to(D).t().contiguous())) * scale
        vv = v[k0:k0 + m].to(D).transpose(0, 1).contiguous()
        i = torch.arange(n, device=DEV)[:, None] + (m - n if causal else m)
        s = s.masked_fill(torch.arange(m, device=DEV)[None] > i, -math.inf)
        p = torch.softmax(s, 2).nan_to_num(0.0) if m else s
        out.append(torch.matmul(p, vv).transpose(0, 1))
        mag.append(torch.matmul(p, vv.abs()).transpose(0, 1))
        q0, k0 = q0 + n, k0 + m
    return torch.cat(out), torch.cat(mag)


@pytest.mark.parametrize("nope,vdim", [(64, 64), (128, 128), (192, 256)])
@pytest.mark.parametrize("nq,nk", [([1], [1]), ([1], [200]), ([64], [64]), ([129, 3, 65], [129, 3, 65]), ([40, 257], [300, 258]),
                                   ([5, 0, 70], [5, 9, 70]), ([10, 20], [0, 7]), ([512], [700])])
def test_prompt_attention(nope, vdim, nq, nk):
    g = gen(nope + sum(nq))
    heads = 5
    q = strided(normal(g, sum(nq), heads, nope + 64), 8)
    both = normal(g, sum(nk), heads, nope + vdim)
    k, v = both[..., :nope], both[..., nope:]
    kr = strided(normal(g, sum(nk), 64), 16)
    for causal in (True, False):
        out = A.prompt_attention(q, k, kr, v, 0.08, cu_q=cumulative(nq), cu_k=cumulative(nk), max_q=max(nq), causal=causal)
        ref, mag = prompt_ref(q, k, kr, v, nq, nk, 0.08, causal)
        close(out, ref, U * ref.abs() + U * mag, f"causal={causal}")


def test_prompt_attention_surroundings_and_scores():
    # NaN in the rows around a sequence's own, scores of hundreds
    g = gen(22)
    nq, nk = [100, 50], [150, 50]
    both = torch.full((300, 4, 256), float("nan"), dtype=BF, device=DEV)
    kr = torch.full((300, 64), float("nan"), dtype=BF, device=DEV)
    both[20:220] = normal(g, 200, 4, 256)
    kr[20:220] = normal(g, 200, 64)
    q = normal(g, 150, 4, 192, std=8.0)
    cu_k = torch.tensor([20, 170, 220], dtype=torch.int32, device=DEV)
    out = A.prompt_attention(q, both[..., :128], kr, both[..., 128:], 1.0, cu_q=cumulative(nq), cu_k=cu_k, max_q=100)
    ref, mag = prompt_ref(q, both[20:220, :, :128], kr[20:220], both[20:220, :, 128:], nq, nk, 1.0)
    close(out, ref, U * ref.abs() + U * mag + 1e-3 * mag)


def test_forms_agree():
    """Absorbed and expanded attention over the same latents, through the
    per-head products, against 64 bits."""
    g = gen(30)
    T, heads, rank, nope, vdim = 70, 16, 512, 128, 128
    kv = normal(g, T, rank + 64)
    w_uk, w_uv = normal(g, heads, nope, rank, std=rank ** -0.5), normal(g, heads, vdim, rank, std=rank ** -0.5)
    q = normal(g, T, heads, nope + 64)
    scale = 192 ** -0.5
    k = A.head_linear(kv[:, None, :rank].expand(T, heads, rank), w_uk)
    v = A.head_linear(kv[:, None, :rank].expand(T, heads, rank), w_uv)
    expanded = A.prompt_attention(q, k, kv[:, rank:], v, scale)
    ql = torch.empty(T, heads, rank + 64, dtype=BF, device=DEV)
    A.head_linear(q[..., :nope], w_uk.transpose(1, 2).contiguous(), out=ql[..., :rank])
    ql[..., rank:] = q[..., nope:]
    cache = torch.zeros(2, 64, rank + 64, dtype=BF, device=DEV)
    cache.view(-1, rank + 64)[:T] = kv
    pages = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    o = A.latent_attention(ql, cache, pages, torch.tensor([T], dtype=torch.int32, device=DEV), scale)
    absorbed = A.head_linear(o, w_uv)
    kd = torch.matmul(kv[:, :rank].to(D), w_uk.to(D).transpose(1, 2).contiguous()).transpose(0, 1)
    vd = torch.matmul(kv[:, :rank].to(D), w_uv.to(D).transpose(1, 2).contiguous()).transpose(0, 1)
    ref, mag = prompt_ref(q, kd, kv[:, rank:], vd, [T], [T], scale)
    # intermediates are rounded to bf16: keys move scores by up to 2^-9 of sum |q k|, about 0.05, and the values by 2^-9
    assert (expanded.to(D) - ref).norm() / ref.norm() < 0.01
    assert (absorbed.to(D) - ref).norm() / ref.norm() < 0.01


# ---------------------------------------------------------------- refusals
def refused(call, code=None):
    with pytest.raises(B.MoeError) as e:
        call()
    if code is not None:
        assert e.value.code == code, str(e.value)


def test_refusals():
    g = gen(40)
    x, w = normal(g, 4, 256), normal(g, 256)
    refused(lambda: A.add_rmsnorm(x, normal(g, 255)))
    refused(lambda: A.add_rmsnorm(x.half(), w))
    refused(lambda: A.add_rmsnorm(x, w, residual=normal(g, 3, 256)))
    refused(lambda: A.add_rmsnorm(x, w, -1.0), B.MOE_EINVAL)
    refused(lambda: A.add_rmsnorm(x.t(), normal(g, 4)))
    refused(lambda: A.add_rmsnorm(normal(g, 1, 40000), normal(g, 40000)), B.MOE_EUNSUPPORTED)
    a, sa, wq, sw = fp8_inputs(g, 4, 128, 256)
    refused(lambda: A.fp8_linear(a, sa[:, :1], wq, sw))
    refused(lambda: A.fp8_linear(a, sa, wq[:, :128], sw))
    refused(lambda: A.fp8_linear(a[:, :248].contiguous(), sa, wq[:, :248].contiguous(), sw), B.MOE_EUNSUPPORTED)
    refused(lambda: A.fp8_linear(a.view(torch.uint8), sa, wq, sw))
    refused(lambda: A.fp8_linear(a, sa, wq, sw, out_dtype=torch.float16))
    h = normal(g, 4, 2, 64)
    refused(lambda: A.head_linear(h, normal(g, 3, 8, 64)))
    refused(lambda: A.head_linear(h[..., :60], normal(g, 2, 8, 60)), B.MOE_EUNSUPPORTED)
    refused(lambda: A.head_linear(h, normal(g, 2, 6, 64)), B.MOE_EUNSUPPORTED)
    kv, table, pos = normal(g, 4, 320), rope_table(8, 64), torch.zeros(4, dtype=torch.int32, device=DEV)
    cache = torch.zeros(2, 16, 320, dtype=BF, device=DEV)
    refused(lambda: A.latent_append(kv, w, 1e-6, table, pos, None, cache))
    refused(lambda: A.latent_append(kv, w, 1e-6, table, pos))
    refused(lambda: A.latent_append(kv, w, 1e-6, table, pos[:3], pos.long(), cache))
    refused(lambda: A.latent_append(kv, w, 1e-6, rope_table(8, 32), pos, pos.long(), cache))
    q, pages = normal(g, 2, 4, 320), torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    lens = torch.tensor([5, 5], dtype=torch.int32, device=DEV)
    refused(lambda: A.latent_attention(q, cache, pages, lens, 0.0), B.MOE_EINVAL)
    refused(lambda: A.latent_attention(q, cache, pages, lens, -1.0), B.MOE_EINVAL)
    refused(lambda: A.latent_attention(normal(g, 3, 4, 320), cache, pages, lens, 1.0), B.MOE_EINVAL)
    refused(lambda: A.latent_attention(normal(g, 2, 4, 192), torch.zeros(2, 16, 192, dtype=BF, device=DEV), pages, lens, 1.0), B.MOE_EUNSUPPORTED)
    refused(lambda: A.latent_attention(q, cache, pages, lens[:1], 1.0))
    refused(lambda: A.latent_attention(q, cache, pages.long(), lens, 1.0))
    refused(lambda: A.latent_attention(q, cache, pages, lens, 1.0, workspace=torch.empty(8, dtype=torch.uint8, device=DEV)), B.MOE_EINVAL)
    refused(lambda: A.latent_attention(q, cache, pages, lens, 1.0, cu_q=pages[0]))
    k = normal(g, 6, 4, 128)
    refused(lambda: A.prompt_attention(normal(g, 6, 4, 192), k, normal(g, 6, 64), k, 0.0), B.MOE_EINVAL)
    refused(lambda: A.prompt_attention(normal(g, 6, 4, 192), k, normal(g, 5, 64), k, 1.0))
    refused(lambda: A.prompt_attention(normal(g, 6, 4, 160), normal(g, 6, 4, 96), normal(g, 6, 64), k, 1.0), B.MOE_EUNSUPPORTED)
    refused(lambda: A.prompt_attention(normal(g, 6, 4, 192), k, normal(g, 6, 64), k, 1.0, cu_q=cumulative([6])))


def test_no_tokens():
    g = gen(41)
    assert A.add_rmsnorm(normal(g, 0, 256), normal(g, 256)).y.shape == (0, 256)
    a, sa, wq, sw = fp8_inputs(g, 1, 128, 256)
    assert A.fp8_linear(a[:0], sa[:0], wq, sw).shape == (0, 128)
    pages = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    out = A.latent_attention(normal(g, 0, 4, 320), torch.zeros(2, 16, 320, dtype=BF, device=DEV), pages, pages[0], 1.0, cu_q=torch.zeros(3, dtype=torch.int32, device=DEV), max_q=0)
    assert out.shape == (0, 4, 256)
    z = normal(g, 0, 4, 128)
    assert A.prompt_attention(normal(g, 0, 4, 192), z, normal(g, 0, 64), z, 1.0).shape == (0, 4, 128)


@pytest.mark.parametrize("T,H", [(1, 6144), (5, 1000), (600, 512), (3, 7)])
def test_quantize(T, H):
    g = gen(T + H)
    for x in (normal(g, T, H, std=3.0), normal(g, T, H, std=3.0, dtype=torch.float32)):
        q, scale = A.quantize(x)
        check_codes(q, scale, x.to(D))
    r = normal(g, T, H)
    both = A.add_rmsnorm(x, None, residual=r, out="both")
    h = x.to(D) + r.to(D)
    close(both.y, h, U * h.abs() + 1e-6, "sum without a norm")
    check_codes(both.q, both.scale, h)


@pytest.mark.parametrize("N,K", [(128, 128), (576, 6144), (100, 272), (1, 16)])
def test_quantize_weight(N, K):
    w = normal(gen(N), N, K)
    code, scale = A.quantize_weight(w)
    full = scale.to(D).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    assert tuple(scale.shape) == (-(-N // 128), -(-K // 128))
    close(code.to(D) * full, w.to(D), torch.maximum(w.to(D).abs() * 2 ** -4, full * 2.0 ** -10) * (1 + 1e-5))


@pytest.mark.parametrize("nope,vdim", [(64, 64), (128, 128), (192, 256)])
@pytest.mark.parametrize("at", [0, 37, 63, 64, 150, 199])
def test_prompt_attention_not_finite_in_masked_places(nope, vdim, at):
    """What a query does not see does not reach it; what it does see, does."""
    g = gen(at)
    T, heads = 200, 2
    q, k, v, kr = normal(g, T, heads, nope + 64), normal(g, T, heads, nope), normal(g, T, heads, vdim), normal(g, T, 64)
    ref, mag = prompt_ref(q, k, kr, v, [T], [T], 0.08)
    for what, bad in (("v", float("nan")), ("v", float("inf")), ("v", -float("inf")), ("k", float("nan"))):
        kk, vv = k.clone(), v.clone()
        if what == "v":
            vv[at, 1, 5] = bad
        else:
            kk[at, 1, 5] = bad
        out = A.prompt_attention(q, kk, kr, vv, 0.08)
        close(out[:, 0], ref[:, 0], U * ref[:, 0].abs() + U * mag[:, 0], f"other head, {what} {bad}")
        close(out[:at], ref[:at], U * ref[:at].abs() + U * mag[:at], f"earlier queries, {what} {bad}")
        assert not out[at:, 1, 5].isfinite().any(), f"later queries, {what} {bad}"


@pytest.mark.parametrize("heads,rank", [(64, 512), (8, 512), (16, 256)])
def test_latent_attention_not_finite_in_masked_places(heads, rank):
    g = gen(heads)
    lens, nq = [130, 66, 7], 5
    q, cache, pages, dl = latent_case(g, lens, [nq] * 3, heads, rank, 16)
    tree = torch.tensor([0b1, 0b11, 0b101, 0b1001, 0b10011] * 3, dtype=torch.int64, device=DEV)
    for masks, sees in ((None, [2, 3, 4]), (tree, [2])):  # tokens that see the new token 2
        ref, mag = latent_ref(q, cache, pages, lens, [nq] * 3, 0.07, rank, tree=masks)
        for bad in (float("nan"), float("inf")):
            dirty = cache.clone()
            for b, n in enumerate(lens):
                p = n - nq + 2
                dirty[int(pages[b, p // 16]), p % 16, 3:300:7] = bad
            out = A.latent_attention(q, dirty, pages, dl, 0.07, max_len=130, tree=masks)
            for t in range(3 * nq):
                if t % nq in sees:
                    assert not out[t].isfinite().all(), (masks is None, t)
                else:
                    close(out[t], ref[t], U * ref[t].abs() + U * mag[t], f"token {t}, {bad}")
