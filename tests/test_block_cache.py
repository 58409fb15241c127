"""CPU tests of the latent cache's bookkeeping (routed_expert_int4_amd/block.py):
lengths, page lists and free pages, held on the host."""
import pytest

torch = pytest.importorskip("torch")

from routed_expert_int4_amd import binding as B  # noqa: E402
from routed_expert_int4_amd.block import BlockConfig, DecoderBlock, LatentCache, random_weights  # noqa: E402

CFG = BlockConfig(hidden=256, heads=4, q_rank=128, rank=256, rope=64, nope=64, vdim=64, page=16)


def make(n_pages=8, max_seqs=2, max_len=64):
    return LatentCache(CFG, n_pages=n_pages, max_seqs=max_seqs, max_len=max_len, device="cpu")


def check(cache, lens):
    """Lengths on host and device, and pages that are each owned once, where the table says."""
    assert cache.host_lens == lens and cache.lens.tolist() == lens
    owned = []
    for b, n in enumerate(lens):
        used = -(-n // CFG.page)
        owned += cache.pages[b, :used].tolist()
    assert len(set(owned)) == len(owned) and all(0 <= p < cache.pool.shape[0] for p in owned)
    # every other page can still be had
    assert len(cache._free) == cache.pool.shape[0] - len(owned) and not set(cache._free) & set(owned)


@pytest.mark.parametrize("counts", [[20, 33], [1, 65], [33, 16], [1, 1, 1], [4, -1], [-1, 4]])
def test_a_refused_extend_changes_nothing(counts):
    # three pages: [20, 33] needs five, [33, 16] four; 65 rows are over a sequence's 64
    cache = make(n_pages=3)
    with pytest.raises(ValueError):
        cache.extend(counts)
    check(cache, [0, 0])
    positions, slots = cache.extend([17, 16])
    check(cache, [17, 16])
    assert positions.tolist() == [*range(17), *range(16)]
    assert len(set(slots.tolist())) == 33
    with pytest.raises(ValueError):
        cache.extend([15, 1])  # no page for the second
    check(cache, [17, 16])
    positions, slots = cache.extend([1, 0])
    assert positions.tolist() == [17]
    assert slots.tolist() == [int(cache.pages[0, 1]) * CFG.page + 1]
    check(cache, [18, 16])


def test_a_refused_step_counts_no_rows():
    # on the CPU every kernel call is refused: after the cache has made room
    block = DecoderBlock(CFG, random_weights(CFG, 1, device="cpu"), max_positions=64, device="cpu")
    cache = make()
    x = torch.zeros(21, CFG.hidden)
    with pytest.raises(B.MoeError):
        block.prompt(x, x, cache, [21, 0])
    check(cache, [0, 0])
    cache.extend([16, 20])
    with pytest.raises(B.MoeError):
        block.decode(x[:2], x[:2], cache)
    check(cache, [16, 20])


def fill(cache, b, n):
    """Row p of sequence b holds 100 b + p."""
    for p in range(n):
        page = int(cache.pages[b, p // CFG.page])
        cache.pool[page, p % CFG.page] = 100 * b + p


def rows(cache, b):
    return [int(cache.pool[int(cache.pages[b, p // CFG.page]), p % CFG.page, -1]) for p in range(cache.host_lens[b])]


@pytest.mark.parametrize("kept", [[], [0], [0, 1], [0, 2, 3], [3, 1], [0, 1, 2, 3]])
def test_accepted_drafts_move_together(kept):
    cache = make(n_pages=5)
    cache.extend([14, 3])
    cache.extend([4, 1], drafted=True)  # over the end of a page
    fill(cache, 0, 18)
    fill(cache, 1, 4)
    with pytest.raises(ValueError):
        cache.extend([1, 0])
    with pytest.raises(ValueError):
        cache.extend([0, 1])
    check(cache, [18, 4])
    cache.accept([kept, [0]])
    check(cache, [14 + len(kept), 4])
    assert rows(cache, 0) == [*range(14), *(14 + j for j in kept)] and rows(cache, 1) == [100, 101, 102, 103]
    positions, _ = cache.extend([1, 1])
    assert positions.tolist() == [14 + len(kept), 4]


def test_accept_refuses_what_was_not_drafted():
    cache = make()
    cache.extend([10, 5])
    cache.extend([3, 0], drafted=True)
    fill(cache, 0, 13)
    for kept in ([[3]], [[-1]], [[0, 0]], [[0], [0]], [[0], [], []]):
        with pytest.raises(ValueError):
            cache.accept(kept)
        check(cache, [13, 5])
    cache.extend([0, 2])  # a sequence without drafts goes on
    check(cache, [13, 7])
    cache.accept([[0, 1]])
    check(cache, [12, 7])
    with pytest.raises(ValueError):
        cache.accept([[0]])  # decided already


def test_truncate_frees_pages():
    cache = make(n_pages=4)
    cache.extend([33, 16])
    with pytest.raises(ValueError):
        cache.truncate(0, 34)
    with pytest.raises(ValueError):
        cache.truncate(0, -1)
    cache.truncate(0, 17)
    check(cache, [17, 16])
    cache.extend([2, 0], drafted=True)
    cache.truncate(0, 18)
    check(cache, [18, 16])
    cache.truncate(0)
    check(cache, [0, 16])
    cache.extend([48, 0])
    check(cache, [48, 16])


def test_a_refused_step_leaves_no_drafts():
    cache = make()
    cache.extend([5, 5])
    with pytest.raises(RuntimeError):
        with cache.step([3, 3], drafted=True):
            raise RuntimeError
    check(cache, [5, 5])
    cache.extend([1, 1])
    check(cache, [6, 6])


def test_positions_past_the_table_are_refused():
    # the refusal comes before the cache changes and before any kernel (which there is none of on the CPU)
    block = DecoderBlock(CFG, random_weights(CFG, 1, device="cpu"), max_positions=20, device="cpu")
    cache = make()
    x = torch.zeros(8, CFG.hidden)
    with pytest.raises(ValueError):
        block.prompt(x, x, cache, [21, 0])
    cache.extend([20, 18])
    for tokens in (1, 3):
        with pytest.raises(ValueError):
            block.decode(x[:2 * tokens], x[:2 * tokens], cache, tokens)
    for at in ([19, 20], [-1, 3]):
        with pytest.raises(ValueError):
            block.decode(x[:2], x[:2], cache, 1, tree=torch.ones(2, dtype=torch.int64), positions=at)
    check(cache, [20, 18])


def test_expansions_keep_the_bits_of_their_weights():
    weights = random_weights(CFG, 1, device="cpu")
    block = DecoderBlock(CFG, weights, max_positions=8, device="cpu")
    full = weights["kv_b"].view(CFG.heads, CFG.nope + CFG.vdim, CFG.rank)
    assert torch.equal(block.w_uk, full[:, :CFG.nope]) and torch.equal(block.w_uv, full[:, CFG.nope:])
    assert torch.equal(block.w_uk_t, full[:, :CFG.nope].transpose(1, 2))
    assert all(w.is_contiguous() for w in (block.w_uk, block.w_uk_t, block.w_uv))
    # in one piece again, where it is asked for
    w, scale = block.lin["kv_b"]
    assert torch.equal(w, weights["kv_b"]) and scale.shape == (4, 2) and (scale == 1).all()
    assert "kv_b" not in set(block.lin)
    with pytest.raises(KeyError):
        block.lin["kv"]
