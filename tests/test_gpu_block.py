"""GPU tests of the decoder block (routed_expert_int4_amd/block.py): its calls
together, as a model runs them.

The expanded and the absorbed form are the same function of the same 8-bit
weights; what differs between them is rounding (keys and values of a head, or
queries and outputs in the latent space, to bf16, each 2^-9 of itself at most)
and where an 8-bit activation falls by it (steps of 2^-4 at most, the values
that change by one are few).  Outputs are compared by norm: 3 %, the size of
one 8-bit rounding of all activations (half a step of 2^-3 to 2^-4, uniformly
distributed: 2^-5)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_int4_amd import synth  # noqa: E402
from routed_expert_int4_amd.block import BlockConfig, DecoderBlock, LatentCache, random_weights  # noqa: E402

DEV = "cuda:0"
SMALL = BlockConfig(hidden=256, heads=4, q_rank=128, rank=256, rope=64, nope=64, vdim=64, page=16)


def near(a, b, tol=0.03):
    a, b = a.double(), b.double()
    assert a.isfinite().all()
    off = ((a - b).norm() / b.norm()).item()
    assert off < tol, off


def make(moe=None, seqs=2):
    block = DecoderBlock(SMALL, random_weights(SMALL, 3), moe, max_positions=256)
    return block, lambda: LatentCache(SMALL, n_pages=40, max_seqs=seqs, max_len=128)


def inputs(T, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(T, SMALL.hidden, generator=g, device=DEV), torch.randn(T, SMALL.hidden, generator=g, device=DEV).bfloat16())


def plain_attention(block, delta, residual, counts):
    """The attention half in 64 bits from the weights the block holds."""
    cfg, D = SMALL, torch.float64

    def weight(name):
        code, s = block.lin[name]
        return code.to(D) * s.to(D).repeat_interleave(128, 0)[:code.shape[0]].repeat_interleave(128, 1)[:, :code.shape[1]]

    def norm(x, name):
        return x / (x.pow(2).mean(-1, keepdim=True) + cfg.eps).sqrt() * block.norms[name].to(D)

    def rotate(x, at):
        c, s = block.table[at].to(D).chunk(2, -1)
        while c.dim() < x.dim():
            c, s = c[:, None], s[:, None]
        return torch.stack([x[..., 0::2] * c - x[..., 1::2] * s, x[..., 0::2] * s + x[..., 1::2] * c], -1).flatten(-2)

    h = delta.to(D) + residual.to(D)
    x = norm(h, "norm_in")
    q = (norm(x @ weight("q_a").t(), "norm_q") @ weight("q_b").t()).view(-1, cfg.heads, cfg.nope + cfg.rope)
    kv = x @ weight("kv_a").t()
    at = torch.cat([torch.arange(n, device=DEV) for n in counts])
    c, kr, qr = norm(kv[:, :cfg.rank], "norm_kv"), rotate(kv[:, cfg.rank:], at), rotate(q[..., cfg.nope:], at)
    e = (c @ weight("kv_b").t()).view(-1, cfg.heads, cfg.nope + cfg.vdim)
    out, first = [], 0
    for n in counts:
        s = slice(first, first + n)
        scores = torch.einsum("ihd,jhd->hij", q[s, :, :cfg.nope], e[s, :, :cfg.nope]) + torch.einsum("ihd,jd->hij", qr[s], kr[s])
        scores = (scores * cfg.scale).masked_fill(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1), -torch.inf)
        out.append(torch.einsum("hij,jhd->ihd", torch.softmax(scores, -1), e[s, :, cfg.nope:]))
        first += n
    return h, torch.cat(out).flatten(1) @ weight("o").t()


def test_prompt_against_64_bits():
    block, cache = make()
    counts = [37, 70]
    delta, residual = inputs(sum(counts), 1)
    h, out = block.prompt(delta, residual, cache(), counts)
    want_h, want = plain_attention(block, delta, residual, counts)
    near(h, want_h, 0.005)
    # four 8-bit roundings of activations lie between the input and the output
    near(out, want, 2 * 0.03)


def test_decode_continues_a_prompt():
    block, cache = make()
    counts = [20, 33]
    delta, residual = inputs(2 * 40, 2)
    first = [delta[:20], delta[40:73]], [residual[:20], residual[40:73]]
    one = cache()
    block.prompt(torch.cat(first[0]), torch.cat(first[1]), one, counts)
    for i in range(5):
        rows = [20 + i, 73 + i]
        _, out = block.decode(delta[rows], residual[rows], one)
    whole = cache()
    longer = [delta[:25], delta[40:78]], [residual[:25], residual[40:78]]
    _, ref = block.prompt(torch.cat(longer[0]), torch.cat(longer[1]), whole, [25, 38])
    near(out, ref[[24, 62]])
    # the same five tokens as one causal chunk
    chunk = cache()
    block.prompt(torch.cat(first[0]), torch.cat(first[1]), chunk, counts)
    rows = list(range(20, 25)) + list(range(73, 78))
    _, out = block.decode(delta[rows], residual[rows], chunk, 5)
    near(out, ref[list(range(20, 25)) + list(range(58, 63))])


def test_tree_of_drafted_tokens():
    """Each branch of a tree gives what decoding that branch alone gives."""
    block, cache = make(seqs=1)
    delta, residual = inputs(40, 5)
    # draft tokens a, b (after a), c (after a), d (after c)
    tree = torch.tensor([0b1, 0b11, 0b101, 0b1101], dtype=torch.int64, device=DEV)
    at = torch.tensor([30, 31, 31, 32], dtype=torch.int32, device=DEV)
    drafted = cache()
    block.prompt(delta[:30], residual[:30], drafted, [30])
    _, out = block.decode(delta[30:34], residual[30:34], drafted, 4, tree=tree, positions=at)
    for branch in ([0, 1], [0, 2, 3]):
        alone = cache()
        block.prompt(delta[:30], residual[:30], alone, [30])
        for j in branch:
            _, o = block.decode(delta[30 + j:31 + j], residual[30 + j:31 + j], alone)
            near(out[j], o[0], 0.01)  # the same calls on the same inputs; only the order of the sums differs


def test_block_with_the_moe_layer():
    from routed_expert_int4_amd.layer import DeviceLayer
    weights = synth.gen_layer(synth.TINY, seed=0)
    moe = DeviceLayer(weights, max_T=64)
    block, cache = make(moe)
    bare, _ = make()
    delta, residual = inputs(50, 7)
    h, out = block.prompt(delta, residual, cache(), [50, 0])
    h0, attn = bare.prompt(delta, residual, cache(), [50, 0])
    want_h = h0.float() + attn.float()
    near(h, want_h, 0.005)
    y = want_h / (want_h.pow(2).mean(1, keepdim=True) + SMALL.eps).sqrt() * block.norms["norm_moe"].float()
    again, ids, _ = moe.forward(y.bfloat16())
    # one bf16 unit in the layer's input moves its output by as much
    near(out, again, 0.02)
    assert out.dtype == torch.float32 and out.shape == (50, SMALL.hidden)
    moe.close()


def test_cache_refuses_what_does_not_fit():
    block, cache = make()
    small = LatentCache(SMALL, n_pages=2, max_seqs=2, max_len=64)
    with pytest.raises(ValueError):
        small.extend([65, 0])
    with pytest.raises(ValueError):
        small.extend([20, 20])
    full = cache()
    delta, residual = inputs(10, 1)
    block.prompt(delta, residual, full, [10, 0])
    with pytest.raises(ValueError):
        block.prompt(delta, residual, full, [5, 5])
