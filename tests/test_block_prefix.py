"""CPU tests of a latent cache of 8 bits and of the prefix that its sequences
can share (routed_expert_int4_amd/block.py): bookkeeping, held on the host."""
import dataclasses

import pytest

torch = pytest.importorskip("torch")

from routed_expert_int4_amd.block import BlockConfig, DecoderBlock, LatentCache, random_weights  # noqa: E402

CFG = BlockConfig(hidden=256, heads=4, q_rank=128, rank=256, rope=64, nope=64, vdim=64, page=16)
NARROW = dataclasses.replace(CFG, cache_bits=8)


def make(cfg=CFG, n_pages=8, max_seqs=3, max_len=64):
    return LatentCache(cfg, n_pages=n_pages, max_seqs=max_seqs, max_len=max_len, device="cpu")


def pages_owned_once(cache):
    owned = [p for pages in cache._lists for p in pages] + cache._prefix_list + cache._free
    assert sorted(owned) == list(range(cache.pool.shape[0]))


@pytest.mark.parametrize("bits", [dict(weight_bits=16), dict(cache_bits=4), dict(weight_bits=0)])
def test_widths_that_are_not_there(bits):
    with pytest.raises(ValueError):
        dataclasses.replace(CFG, **bits)


def test_rows_of_8_bits_and_their_scales_move_together():
    cache = make(NARROW)
    assert cache.pool.dtype == torch.uint8 and cache.pool.shape == (8, 16, 256 + 128) and cache.scale.shape == (8, 16)
    cache.extend([14, 0, 0])
    cache.extend([4, 0, 0], drafted=True)
    for p in range(18):
        page = int(cache.pages[0, p // 16])
        cache.pool[page, p % 16], cache.scale[page, p % 16] = p, float(p)
    cache.accept([[0, 3]])
    assert cache.host_lens == [16, 0, 0]
    at = [(int(cache.pages[0, p // 16]), p % 16) for p in range(16)]
    assert [int(cache.pool[a, b, -1]) for a, b in at] == [*range(15), 17]
    assert [float(cache.scale[a, b]) for a, b in at] == [*range(15), 17]


def test_a_sequence_becomes_the_prefix():
    cache = make()
    cache.extend([0, 20, 0])
    pages = cache.pages[1, :2].tolist()
    cache.share(1)
    assert cache.prefix_len == 20 and cache.host_lens == [0, 0, 0] and cache.lens.tolist() == [0, 0, 0]
    assert cache.prefix.pages.tolist() == [pages] and cache.prefix.lens.tolist() == [20] and cache.prefix.groups is None
    pages_owned_once(cache)
    positions, slots = cache.extend([2, 0, 17])
    assert positions.tolist() == [20, 21, *range(20, 37)]
    assert not {s // 16 for s in slots.tolist()} & set(pages)
    pages_owned_once(cache)
    with pytest.raises(ValueError):
        cache.drop_prefix()
    cache.truncate(0)
    cache.truncate(2)
    cache.drop_prefix()
    assert cache.prefix is None and cache.prefix_len == 0 and len(cache._free) == 8
    pages_owned_once(cache)
    assert cache.extend([1, 0, 0])[0].tolist() == [0]


def test_what_cannot_be_shared():
    cache = make()
    with pytest.raises(ValueError):
        cache.share(0)  # no rows
    cache.extend([3, 1, 0])
    with pytest.raises(ValueError):
        cache.share(0)  # another has rows
    cache.truncate(1)
    cache.extend([2, 0, 0], drafted=True)
    with pytest.raises(ValueError):
        cache.share(0)  # undecided drafts
    cache.accept([[0]])
    cache.share(0)
    assert cache.prefix_len == 4
    cache.extend([1, 0, 0])
    with pytest.raises(ValueError):
        cache.share(0)  # there is one
    pages_owned_once(cache)


def test_prompts_do_not_start_after_a_prefix():
    block = DecoderBlock(CFG, random_weights(CFG, 1, device="cpu"), max_positions=30, device="cpu")
    cache = make()
    cache.extend([20, 0, 0])
    cache.share(0)
    x = torch.zeros(5, CFG.hidden)
    with pytest.raises(ValueError, match="decode"):
        block.prompt(x, x, cache, [5, 0, 0])
    with pytest.raises(ValueError, match="position 30"):  # 20 + 11 tokens
        block.decode(torch.zeros(11, CFG.hidden), torch.zeros(11, CFG.hidden), cache, [11, 0, 0])
    assert cache.host_lens == [0, 0, 0]


def test_4_bit_weights_by_name():
    cfg = dataclasses.replace(CFG, weight_bits=4)
    block = DecoderBlock(cfg, random_weights(cfg, 1, device="cpu"), max_positions=30, device="cpu")
    codes, scale = block.lin["o"]
    assert codes.shape == (256, 128) and codes.dtype == torch.uint8 and scale.shape == (256, 8) and scale.dtype == torch.float16
