"""Scales of an 8-bit latent cache that are not powers of two: a row is read
with the power of two that has the scale's exponent, whatever its sign and
mantissa, as key, as value and by latent_read.  So a cache gives the same bits
as with these powers of two in it."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
I32 = torch.int32


@pytest.fixture(scope="module")
def A():
    from routed_expert_int4_amd import attention
    return attention


def power_of_two(scale):
    return (scale.view(I32) & 0x7F800000).view(torch.float32)


class Cache:
    """Sequences of `own` rows on pages of their own, and a prefix of `prefix` rows."""

    def __init__(self, B, own, rank, heads, nq, page, prefix, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        per, before = -(-own // page), -(-prefix // page)
        n = B * per + before
        codes = torch.randn(n, page, rank, generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
        key = torch.randn(n, page, 64, generator=g, device=DEV).bfloat16().view(torch.uint8)
        self.cache = torch.cat([codes, key], -1).contiguous()
        mantissa = torch.rand(n, page, generator=g, device=DEV) + 1
        sign = torch.randint(0, 2, (n, page), generator=g, device=DEV) * 2 - 1
        self.scale = mantissa * sign * 2.0 ** torch.randint(-4, 3, (n, page), generator=g, device=DEV)
        order = torch.randperm(n, generator=g, device=DEV).to(I32)
        self.pages, self.prefix_pages = order[:B * per].view(B, per), order[B * per:][None]
        self.own, self.prefix, self.lens = own, prefix, torch.full((B,), own, dtype=I32, device=DEV)
        self.q = torch.randn(B * nq, heads, rank + 64, generator=g, device=DEV).bfloat16()

    def attend(self, A, scale, **more):
        prefix = A.SharedPrefix(self.prefix_pages, torch.tensor([self.prefix], dtype=I32, device=DEV)) if self.prefix else None
        return A.latent_attention(self.q, self.cache, self.pages, self.lens, 0.05, max_len=self.own, cache_scale=scale, prefix=prefix, **more)


@pytest.mark.parametrize("B,own,rank,heads,nq,page,prefix", [(1, 1, 512, 64, 1, 64, 0), (1, 1013, 512, 64, 1, 64, 0), (3, 200, 256, 16, 2, 100, 0),
                                                              (2, 300, 512, 64, 5, 16, 0), (2, 40, 512, 64, 1, 64, 517), (3, 70, 256, 16, 2, 16, 100)])
def test_same_bits_as_powers_of_two(A, B, own, rank, heads, nq, page, prefix):
    c = Cache(B, own, rank, heads, nq, page, prefix, own)
    clean = power_of_two(c.scale)
    assert bool((clean != c.scale).any()) and bool((c.scale < 0).any())
    want = c.attend(A, clean)
    assert bool(want.isfinite().all()) and torch.equal(c.attend(A, c.scale), want)
    three = torch.full_like(c.scale, 3.0)
    assert torch.equal(c.attend(A, three), c.attend(A, torch.full_like(three, 2.0)))


def test_rows_read_back(A):
    c = Cache(2, 300, 512, 1, 1, 16, 0, 7)
    slots = torch.randperm(c.scale.numel(), device=DEV)
    got, want = (A.latent_read(c.cache, s, slots) for s in (c.scale, power_of_two(c.scale)))
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    codes = c.cache.view(-1, 640)[slots, :512].contiguous().view(torch.float8_e4m3fn).double()
    assert torch.equal(want[:, :512].double(), codes * power_of_two(c.scale).view(-1)[slots, None].double())


@pytest.mark.parametrize("prefix", [0, 200])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_scales_that_are_not_finite(A, prefix, bad):
    """A token that sees such a row is NaN; one that does not has its usual bits."""
    c = Cache(2, 150, 512, 16, 3, 64, prefix, 3)
    want = c.attend(A, c.scale)
    last = c.own - 1  # the last new token's row, seen by it alone
    c.scale[c.pages[1, last // 64].long(), last % 64] = bad
    out = c.attend(A, c.scale)
    assert bool(out[5].isnan().all()) and torch.equal(out[:5], want[:5])


@pytest.mark.parametrize("prefix", [0, 100])
@pytest.mark.parametrize("tiny", [0.0, -0.0, 1e-40, -1e-45])
def test_scales_without_an_exponent(A, prefix, tiny):
    """At most 2^-127, and codes are at most 448: no column above 448 x 2^-127
    beside one rounding to bf16, and the position part counts as ever."""
    c = Cache(2, 150, 512, 16, 1, 64, prefix, 4)
    out = c.attend(A, torch.full_like(c.scale, tiny))
    assert bool((out.double().abs() <= 448 * 2.0 ** -127 * (1 + 2.0 ** -7)).all())
