"""GPU tests of the decoder block with 4-bit projections, with a cache of 8 bits
and with a prefix that its sequences share: its calls together, as a model runs
them.

Compared by norm, as the block's other tests are.  What differs between the
forms: bf16 roundings of heads and latents (2^-9 each), and with 8-bit
projections activations that fall to another code by them, at most one 8-bit
rounding of all activations, 3 %.  With 4-bit projections activations are bf16:
the forms differ by bf16 roundings alone, a few times 2^-9 of the norm, 1 %;
a cache of 8 bits holds another code only where fp32 sums differ, which the
same rows written by two forms do by a bf16 rounding of their inputs (then one
code in 16 moves by a step of 2^-3 of itself: 2^-3 / 16, 1 %)."""
import dataclasses

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_int4_amd import attention as A  # noqa: E402
from routed_expert_int4_amd.block import BlockConfig, DecoderBlock, LatentCache, random_weights  # noqa: E402

DEV = "cuda:0"
SMALL = BlockConfig(hidden=256, heads=4, q_rank=128, rank=256, rope=64, nope=64, vdim=64, page=16)
FORMS = [(8, 8), (4, 16), (4, 8)]
TOL = {8: 0.03, 4: 0.02}


def near(a, b, tol):
    a, b = a.double(), b.double()
    assert a.isfinite().all()
    off = ((a - b).norm() / b.norm()).item()
    assert off < tol, off


def make(bits, seqs=2, max_len=128):
    cfg = dataclasses.replace(SMALL, weight_bits=bits[0], cache_bits=bits[1])
    block = DecoderBlock(cfg, random_weights(cfg, 3), None, max_positions=256)
    return block, lambda: LatentCache(cfg, n_pages=40, max_seqs=seqs, max_len=max_len)


def inputs(T, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(T, SMALL.hidden, generator=g, device=DEV), torch.randn(T, SMALL.hidden, generator=g, device=DEV).bfloat16())


def held(cache, b):
    """Sequence b's rows as the cache holds them, in 64 bits."""
    slots = torch.tensor([cache._slot(b, p) for p in range(cache.host_lens[b])], device=DEV)
    if cache.scale is None:
        return cache.pool.view(-1, cache.pool.shape[2])[slots].double()
    return A.latent_read(cache.pool, cache.scale, slots).double()


@pytest.mark.parametrize("bits", FORMS)
def test_prompt_against_64_bits(bits):
    """From the weights that the block holds and the rows that its cache holds."""
    block, cache = make(bits)
    counts, D, cfg = [37, 70], torch.float64, block.cfg
    delta, residual = inputs(sum(counts), 1)
    one = cache()
    h, out = block.prompt(delta, residual, one, counts)

    def weight(name):
        code, s = block.lin[name]
        if name == "kv_b" or bits[0] == 8:
            return code.to(D) * s.to(D).repeat_interleave(128, 0)[:code.shape[0]].repeat_interleave(128, 1)[:, :code.shape[1]]
        q = torch.stack([code.to(torch.int16) & 15, code.to(torch.int16) >> 4], 2).flatten(1)
        return torch.where(q > 7, q - 16, q).to(D) * s.to(D).repeat_interleave(32, 1)

    def norm(x, name):
        return x / (x.pow(2).mean(-1, keepdim=True) + cfg.eps).sqrt() * block.norms[name].to(D)

    def rotate(x, at):
        c, s = block.table[at].to(D).chunk(2, -1)
        while c.dim() < x.dim():
            c, s = c[:, None], s[:, None]
        return torch.stack([x[..., 0::2] * c - x[..., 1::2] * s, x[..., 0::2] * s + x[..., 1::2] * c], -1).flatten(-2)

    want_h = delta.to(D) + residual.to(D)
    x = norm(want_h, "norm_in")
    q = (norm(x @ weight("q_a").t(), "norm_q") @ weight("q_b").t()).view(-1, cfg.heads, cfg.nope + cfg.rope)
    kv = x @ weight("kv_a").t()
    at = torch.cat([torch.arange(n, device=DEV) for n in counts])
    qr = rotate(q[..., cfg.nope:], at)
    first, outs = 0, []
    for b, n in enumerate(counts):
        s = slice(first, first + n)
        rows = held(one, b)
        # rows are the norm and the rotation of kv: to the cache's width
        near(rows[:, :cfg.rank], norm(kv[s, :cfg.rank], "norm_kv"), 0.06 if bits[1] == 8 else TOL[bits[0]])
        near(rows[:, cfg.rank:], rotate(kv[s, cfg.rank:], at[s]), TOL[bits[0]])
        e = (rows[:, :cfg.rank] @ weight("kv_b").t()).view(n, cfg.heads, cfg.nope + cfg.vdim)
        scores = torch.matmul(q[s, :, :cfg.nope].transpose(0, 1), e[..., :cfg.nope].permute(1, 2, 0).contiguous())
        scores = (scores + torch.matmul(qr[s].transpose(0, 1), rows[:, cfg.rank:].t().contiguous())) * cfg.scale
        scores = scores.masked_fill(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1), -torch.inf)
        outs.append(torch.matmul(torch.softmax(scores, -1), e[..., cfg.nope:].transpose(0, 1).contiguous()).transpose(0, 1))
        first += n
    near(h, want_h, 0.005)
    near(out, torch.cat(outs).flatten(1) @ weight("o").t(), 2 * TOL[bits[0]])


@pytest.mark.parametrize("bits", FORMS)
def test_decode_continues_a_prompt(bits):
    block, cache = make(bits)
    counts = [20, 33]
    delta, residual = inputs(80, 2)
    start = torch.tensor([*range(20), *range(40, 73)], device=DEV)
    one, whole, chunk = cache(), cache(), cache()
    block.prompt(delta[start], residual[start], one, counts)
    block.prompt(delta[start], residual[start], chunk, counts)
    for i in range(5):
        _, out = block.decode(delta[[20 + i, 73 + i]], residual[[20 + i, 73 + i]], one)
    longer = torch.tensor([*range(25), *range(40, 78)], device=DEV)
    _, ref = block.prompt(delta[longer], residual[longer], whole, [25, 38])
    near(out, ref[[24, 62]], TOL[bits[0]])
    rows = [*range(20, 25), *range(73, 78)]
    _, out = block.decode(delta[rows], residual[rows], chunk, 5)
    near(out, ref[[*range(20, 25), *range(58, 63)]], TOL[bits[0]])
    for b in range(2):
        near(held(one, b), held(whole, b), TOL[bits[0]])


@pytest.mark.parametrize("bits", [(8, 16), *FORMS])
def test_a_shared_prefix_is_every_sequences_own(bits):
    """Three sequences on one prefix against three that hold all rows; chunks,
    single tokens and a tree whose accepted branch goes on."""
    block, cache = make(bits, seqs=3)
    delta, residual = inputs(200, 3)
    common = list(range(50))
    shared, apart = cache(), cache()
    block.prompt(delta[common], residual[common], shared, [0, 50, 0])
    shared.share(1)
    block.prompt(delta[common * 3], residual[common * 3], apart, [50, 50, 50])

    def both(rows, count, **more):
        _, a = block.decode(delta[rows], residual[rows], shared, count, **more)
        _, b = block.decode(delta[rows], residual[rows], apart, count, **more)
        near(a, b, TOL[bits[0]])

    both(list(range(60, 78)), [7, 0, 11])  # a chunk each, one sits out
    assert shared.host_lens == [7, 0, 11] and apart.host_lens == [57, 50, 61]
    both([80, 81, 82], 1)
    tree = torch.tensor([1, 3, 5, 13] * 3, dtype=torch.int64, device=DEV)
    at = [n + d for n in apart.host_lens for d in (0, 1, 1, 2)]
    both(list(range(90, 102)), 4, tree=tree, positions=at)
    for c in (shared, apart):
        c.accept([[0, 2, 3], [0], []])
    assert shared.host_lens == [11, 2, 12]
    both([110, 111, 112], 1)


@pytest.mark.parametrize("bits", FORMS)
def test_refused_steps_leave_a_narrow_cache_alone(bits):
    block, cache = make(bits)
    one = cache()
    delta, residual = inputs(30, 4)
    block.prompt(delta[:20], residual[:20], one, [20, 0])
    before = one.pool.clone()
    with pytest.raises(Exception):
        block.decode(delta[:2, :100], residual[:2, :100], one)
    assert one.host_lens == [20, 0] and torch.equal(one.pool, before)
    _, a = block.decode(delta[20:22], residual[20:22], one)
    other = cache()
    block.prompt(delta[:20], residual[:20], other, [20, 0])
    _, b = block.decode(delta[20:22], residual[20:22], other)
    assert torch.equal(a, b)
