"""GPU tests of a decoder block and its cache over several steps
(routed_expert_int4_amd/block.py): refused steps, drafted tokens, sequences
that come and go.

Two ways to the same tokens run the same kernels on the same rows and differ
in the order of sums: outputs are compared by norm, 1 % (a bf16 unit in an
activation is 2^-8, and an 8-bit code that falls the other way is one value
of many)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_int4_amd import binding as B  # noqa: E402
from routed_expert_int4_amd import synth  # noqa: E402
from routed_expert_int4_amd.block import BlockConfig, DecoderBlock, LatentCache, random_weights  # noqa: E402

DEV = "cuda:0"
CFG = BlockConfig(hidden=256, heads=4, q_rank=128, rank=256, rope=64, nope=64, vdim=64, page=16)


def near(a, b, tol=0.01):
    a, b = a.double(), b.double()
    assert a.shape == b.shape and a.isfinite().all()
    off = ((a - b).norm() / b.norm()).item()
    assert off < tol, off


def make(moe=None, max_positions=256):
    return DecoderBlock(CFG, random_weights(CFG, 3), moe, max_positions=max_positions)


def cache(seqs=2, n_pages=40, max_len=128):
    return LatentCache(CFG, n_pages=n_pages, max_seqs=seqs, max_len=max_len)


def inputs(T, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(T, CFG.hidden, generator=g, device=DEV), torch.randn(T, CFG.hidden, generator=g, device=DEV).bfloat16()


def test_a_refused_step_can_be_made_again():
    from routed_expert_int4_amd.layer import DeviceLayer
    moe = DeviceLayer(synth.gen_layer(synth.TINY, seed=0), max_T=24)
    block, used, fresh = make(moe), cache(), cache()
    delta, residual = inputs(40, 1)
    tree = torch.ones(3, dtype=torch.int64, device=DEV)
    with pytest.raises(B.MoeError):
        block.prompt(delta, residual, used, [40, 0])  # the routed layer holds 24 tokens
    _, first = block.prompt(delta[:20], residual[:20], used, [20, 0])
    with pytest.raises(B.MoeError):
        block.decode(delta[:4], residual[:4], used, 2, tree=tree)  # four tokens, three masks
    assert used.host_lens == [20, 0] and used.lens.tolist() == [20, 0]
    _, second = block.decode(delta[20:22], residual[20:22], used)
    _, want = block.prompt(delta[:20], residual[:20], fresh, [20, 0])
    near(first, want)
    _, want = block.decode(delta[20:22], residual[20:22], fresh)
    near(second, want)
    moe.close()


@pytest.mark.parametrize("branch,depths", [([0, 1], [0, 1, 1, 2]), ([0, 2, 3], [0, 1, 1, 2])])
def test_decoding_goes_on_from_an_accepted_branch(branch, depths):
    """A prompt, a tree, one branch accepted, and on: as if only that branch
    had ever been decoded."""
    block = make()
    delta, residual = inputs(60, 5)
    # draft tokens a, b (after a), c (after a), d (after c)
    tree = torch.tensor([0b1, 0b11, 0b101, 0b1101] * 2, dtype=torch.int64, device=DEV)
    drafted, alone = cache(), cache()
    for used in (drafted, alone):
        block.prompt(delta[:45], residual[:45], used, [30, 15])
    at = torch.tensor([first + d for first in (30, 15) for d in depths], dtype=torch.int32, device=DEV)
    rows = slice(45, 49)
    both = [torch.cat([t[rows], t[rows]]) for t in (delta, residual)]
    block.decode(*both, drafted, 4, tree=tree, positions=at)
    with pytest.raises(ValueError):
        block.decode(delta[:2], residual[:2], drafted)
    drafted.accept([branch, branch])
    for j in branch:
        block.decode(delta[[45 + j] * 2], residual[[45 + j] * 2], alone)
    assert drafted.host_lens == alone.host_lens and torch.equal(drafted.lens, alone.lens)
    for i in range(3):
        step = [50 + 2 * i, 51 + 2 * i]
        _, out = block.decode(delta[step], residual[step], drafted)
        _, want = block.decode(delta[step], residual[step], alone)
        near(out, want)


def test_the_last_known_position():
    block, used = make(max_positions=24), cache(seqs=1)
    delta, residual = inputs(30, 6)
    block.prompt(delta[:23], residual[:23], used, [23])
    _, out = block.decode(delta[23:24], residual[23:24], used)
    assert out.isfinite().all()
    with pytest.raises(ValueError):
        block.decode(delta[24:25], residual[24:25], used)
    used.truncate(0, 21)
    tree = torch.tensor([1, 3, 5, 11], dtype=torch.int64, device=DEV)
    _, lists = block.decode(delta[21:25], residual[21:25], used, 4, tree=tree, positions=[21, 22, 22, 23])
    used.truncate(0, 21)
    at = torch.tensor([21, 22, 22, 23], dtype=torch.int32, device=DEV)
    _, tensors = block.decode(delta[21:25], residual[21:25], used, 4, tree=tree, positions=at)
    assert torch.equal(lists, tensors) and lists.isfinite().all()


def test_sequences_sit_out_end_and_start_again():
    block = make()
    delta, residual = inputs(100, 7)
    used = cache(seqs=3, n_pages=9)
    alone = [cache(seqs=1) for _ in range(3)]

    def both(call, *steps):
        """A step of (sequence, first row, rows) triples, together and each alone."""
        at = torch.cat([torch.arange(first, first + n) for _, first, n in steps]).to(DEV)
        counts = [0] * 3
        for b, _, n in steps:
            counts[b] = n
        _, out = getattr(block, call)(delta[at], residual[at], used, counts)
        done = 0
        for b, first, n in steps:
            rows = slice(first, first + n)
            _, want = getattr(block, call)(delta[rows], residual[rows], alone[b], [n])
            near(out[done:done + n], want)
            done += n
        assert used.lens.tolist() == [c.host_lens[0] for c in alone]

    both("prompt", (0, 0, 30), (2, 30, 17))       # the second sequence is empty
    both("decode", (0, 60, 1), (2, 61, 1))
    both("decode", (2, 62, 5))                    # a chunk of one of them
    both("decode", (0, 67, 2), (2, 69, 1))        # chunks of different lengths
    both("prompt", (1, 47, 13))
    both("decode", (0, 70, 1), (1, 71, 1), (2, 72, 1))
    used.truncate(0)
    alone[0].truncate(0)
    both("decode", (1, 73, 1), (2, 74, 1))
    both("prompt", (0, 75, 20))                   # on pages that were another sequence's
    both("decode", (0, 95, 1), (1, 96, 1), (2, 97, 1))
    with pytest.raises(ValueError):
        block.decode(delta[:1], residual[:1], used, [0, 0, 0, 1])
    # no token at all
    for call in (block.prompt, block.decode):
        _, out = call(delta[:0], residual[:0], cache(seqs=2), [0, 0])
        assert out.shape == (0, CFG.hidden)


def test_trees_of_different_sizes():
    block, used = make(), cache(seqs=3)
    delta, residual = inputs(60, 8)
    block.prompt(delta[:45], residual[:45], used, [20, 20, 5])
    tree = torch.tensor([0b1, 0b11, 0b101, 0b1, 0b11], dtype=torch.int64, device=DEV)
    _, out = block.decode(delta[45:50], residual[45:50], used, [3, 0, 2], tree=tree, positions=[20, 21, 21, 5, 6])
    used.accept([[0, 2], [], [0]])
    assert used.host_lens == [22, 20, 6]
    for b, first, have, branch, rows in ((0, 0, 20, [45, 47], [0, 2]), (2, 40, 5, [48, 49], [3, 4])):
        alone = cache(seqs=1)
        block.prompt(delta[first:first + have], residual[first:first + have], alone, [have])
        for at, row in zip(branch, rows):
            _, want = block.decode(delta[at:at + 1], residual[at:at + 1], alone)
            near(out[row], want[0])
    with pytest.raises(ValueError):
        block.decode(delta, residual, used, [65, 0, 0], tree=torch.ones(65, dtype=torch.int64, device=DEV), positions=[1] * 65)
