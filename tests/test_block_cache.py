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
