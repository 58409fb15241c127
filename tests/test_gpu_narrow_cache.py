"""The latent cache in 8 bits: rows written, read back and attended to, against
the definitions in 64 bits.

A code is the value over the row's power of two rounded to nearest E4M3: off by
at most half a step, 2^-4 of it (2^-10 below 2^-6).  The value that is rounded
is an fp32 norm, off by at most (rank / 2 + 8) 2^-24 of itself, which can move
it across a tie; the power of two is exact, but a largest value next to
448 x 2^e can fall on either side of it."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 1e-6


@pytest.fixture(scope="module")
def A():
    from routed_expert_int4_amd import attention
    return attention


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def power(top):
    """The definition, from fp64 magnitudes."""
    e = torch.ceil(torch.log2(top / 448))
    return torch.where(top == 0, torch.ones_like(top), 2.0 ** e.clamp_min(-100))


def parts(cache, rank):
    rows = cache.view(-1, cache.shape[-1])
    return rows[:, :rank].contiguous().view(torch.float8_e4m3fn), rows[:, rank:].contiguous().view(torch.bfloat16)


def write(A, T, rank, rope=64, page=16, std=1.0, seed=0, slots=None, pages=None, **more):
    g = generator(seed)
    kv = (torch.randn(T, rank + rope, generator=g, device=DEV) * std).bfloat16()
    weight = (torch.rand(rank, generator=g, device=DEV) + 0.5).bfloat16()
    table = torch.randn(200, rope, generator=g, device=DEV)
    positions = torch.randint(0, 200, (T,), generator=g, device=DEV, dtype=torch.int32)
    pages = pages or -(-T // page) + 2
    if slots is None:
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:T]
    cache = torch.full((pages, page, rank + 2 * rope), 0x55, dtype=torch.uint8, device=DEV)
    scale = torch.full((pages, page), 3.0, device=DEV)
    r = A.latent_append(kv, weight, EPS, table, positions, slots, cache, cache_scale=scale, **more)
    return kv, weight, table, positions, slots, cache, scale, r


def normed(kv, weight):
    c = kv[:, :weight.shape[0]].double()
    return c / ((c * c).mean(1, keepdim=True) + EPS).sqrt() * weight.double()


@pytest.mark.parametrize("T,rank,rope,page,std", [(1, 512, 64, 64, 1.0), (7, 256, 64, 1, 1e-3), (100, 512, 64, 100, 50.0), (33, 16, 8, 5, 1.0),
                                                   (20, 1040, 64, 16, 1.0), (9, 2048, 128, 16, 1.0), (1000, 512, 64, 64, 3.0)])
def test_written_rows(A, T, rank, rope, page, std):
    kv, weight, table, positions, slots, cache, scale, _ = write(A, T, rank, rope, page, std, seed=T)
    c = normed(kv, weight)
    want = power(c.abs().amax(1))
    got = scale.view(-1)[slots].double()
    top = c.abs().amax(1) / want
    edge = (top > 448 * (1 - 1e-5)) | (top < 224 * (1 + 1e-5))
    assert bool(((got == want) | edge & ((got / want).log2().abs() <= 1)).all())
    codes, key = parts(cache, rank)
    exact = c / got[:, None]
    back = codes[slots].float().double()
    fp32 = (rank / 2 + 8) * 2.0 ** -24 * exact.abs()
    assert bool(((back - exact).abs() <= torch.maximum(2.0 ** -4 * exact.abs(), torch.full_like(exact, 2.0 ** -10)) * (1 + 2.0 ** -4) + fp32).all())
    # to nearest, but for ties that fp32 moves
    both = torch.stack([back, codes[slots].view(torch.uint8).add(1).view(torch.float8_e4m3fn).float().double().nan_to_num(1e9),
                        codes[slots].view(torch.uint8).sub(1).view(torch.float8_e4m3fn).float().double().nan_to_num(1e9)])
    off = (both - exact).abs()
    assert bool((off[0] <= off[1:].amin(0) + 2 * fp32).all())
    # the position part as in bf16
    cos, sin = table[positions.long()].double().split(rope // 2, 1)
    even, odd = kv[:, rank:].double()[:, 0::2], kv[:, rank:].double()[:, 1::2]
    rotated = torch.stack([even * cos - odd * sin, even * sin + odd * cos], 2).flatten(1)
    spread = torch.stack([(even * cos).abs() + (odd * sin).abs(), (even * sin).abs() + (odd * cos).abs()], 2).flatten(1)
    assert bool(((key[slots].double() - rotated).abs() <= 2.0 ** -8 * rotated.abs() + 2.0 ** -22 * spread).all())
    # rows of no token are as they were
    others = torch.ones(scale.numel(), dtype=torch.bool, device=DEV)
    others[slots] = False
    assert bool((cache.view(-1, cache.shape[-1])[others] == 0x55).all()) and bool((scale.view(-1)[others] == 3).all())


def test_same_rows_as_the_wide_cache(A):
    """Everything but the codes agrees with the bf16 cache bit for bit."""
    kv, weight, table, positions, slots, cache, scale, r = write(A, 50, 512, seed=5, want_key=True)
    wide = torch.zeros(cache.shape[0], cache.shape[1], 576, dtype=torch.bfloat16, device=DEV)
    q = torch.randn(50, 4, 64, device=DEV).bfloat16()
    other = A.latent_append(kv, weight, EPS, table, positions, slots, wide, q_rope=q, want_key=True)
    narrow = A.latent_append(kv, weight, EPS, table, positions, slots, cache, q_rope=q, want_key=True, cache_scale=scale)
    assert torch.equal(narrow.rows, other.rows) and torch.equal(narrow.key, other.key) and torch.equal(narrow.q_rope, other.q_rope)
    assert torch.equal(r.rows, other.rows)
    back = A.latent_read(cache, scale, slots)
    assert torch.equal(back[:, 512:], other.rows[:, 512:])
    off = (back[:, :512].float() - other.rows[:, :512].float()).abs()
    top = other.rows[:, :512].float().abs().amax(1, keepdim=True)
    # half a step of E4M3 and of bf16; below the smallest normal code 2^-10 x 2 / 448 of the largest
    assert bool((off <= other.rows[:, :512].float().abs() * (2.0 ** -4 + 2.0 ** -7) + top * 2.0 ** -17).all())


@pytest.mark.parametrize("exponent", [-100, -30, -7, 0, 3, 60, 119])
def test_every_code_is_read_exactly(A, exponent):
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(2).view(1, 512)
    key = torch.arange(64, device=DEV).bfloat16()
    cache = torch.cat([codes, key.view(torch.uint8)[None]], 1).view(1, 1, 640).contiguous()
    scale = torch.full((1, 1), 2.0, device=DEV) ** exponent
    back = A.latent_read(cache, scale, torch.zeros(1, dtype=torch.int64, device=DEV))
    want = codes.view(torch.float8_e4m3fn).double() * 2.0 ** exponent
    want = want.to(torch.bfloat16)  # exact, but for what passes bf16's range
    assert torch.equal(back[0, :512].nan_to_num(nan=-1.0), want[0].nan_to_num(nan=-1.0)) and torch.equal(back[0, 512:], key)


@pytest.mark.parametrize("T", [1, 3, 300])
def test_read_back_and_slots_outside(A, T):
    *_, slots, cache, scale, _ = write(A, T, 256, page=7, seed=T)
    odd = slots.clone()
    odd[::3] = torch.tensor([-1, scale.numel(), 2 ** 40, -2 ** 50], device=DEV).repeat(-(-T // 12))[: odd[::3].numel()]
    wide = torch.full((T, 400), 7.0, dtype=torch.bfloat16, device=DEV)
    back = A.latent_read(cache, scale, odd, out=wide[:, 8:328])
    codes, key = parts(cache, 256)
    want = torch.cat([(codes.float() * scale.view(-1, 1)).bfloat16(), key], 1)[slots]
    want[::3] = 0
    assert torch.equal(back, want) and bool((wide[:, :8] == 7).all()) and bool((wide[:, 328:] == 7).all())


def test_slots_that_write_nothing(A):
    slots = torch.tensor([-1, 5, 48, 2 ** 40], device=DEV)
    kv, *_, cache, scale, _ = write(A, 4, 256, slots=slots, pages=3)
    same = (cache == 0x55).all(2).view(-1)
    assert same.nonzero().flatten().tolist() == [i for i in range(48) if i != 5]


def test_rows_of_zeros_and_values_that_are_not_finite(A):
    g = generator(1)
    kv = torch.randn(5, 320, generator=g, device=DEV).bfloat16()
    kv[0, :256] = 0
    kv[1, 3] = float("nan")
    weight = torch.ones(256, device=DEV)
    weight[7] = float("inf")
    weight[9] = 2.0 ** -120
    table = torch.ones(4, 64, device=DEV)
    slots = torch.arange(5, device=DEV)
    cache, scale = torch.zeros(1, 8, 384, dtype=torch.uint8, device=DEV), torch.zeros(1, 8, device=DEV)
    A.latent_append(kv, weight, EPS, table, torch.zeros(5, dtype=torch.int32, device=DEV), slots, cache, cache_scale=scale)
    back = A.latent_read(cache, scale, slots)[:, :256].float()
    assert bool(back[0, :7].eq(0).all()) and bool(back[0, 7].isnan()) and float(scale[0, 0]) == 1.0  # 0 x inf
    assert bool(back[1].isnan().all())
    finite = torch.arange(256, device=DEV) != 7
    want = normed(kv[2:], torch.ones(256, device=DEV))
    want[:, 9] = 0
    assert bool(back[2:, 7].isnan().all())
    assert bool(((back[2:] - want).abs() <= want.abs() * 0.07 + 2.0 ** -9 * scale[0, 2:5, None])[:, finite].all())


def test_written_and_read_in_a_graph(A):
    kv, weight, table, positions, slots, cache, scale, _ = write(A, 40, 512, seed=9)
    out = torch.empty(40, 576, dtype=torch.bfloat16, device=DEV)

    def step():
        A.latent_append(kv, weight, EPS, table, positions, slots, cache, cache_scale=scale)
        A.latent_read(cache, scale, slots, out=out)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for i in range(3):
        kv.copy_(torch.randn(40, 576, generator=generator(i), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.zero_()
        step()
        assert torch.equal(got, out)


def test_no_rows(A):
    cache, scale = torch.zeros(2, 4, 640, dtype=torch.uint8, device=DEV), torch.zeros(2, 4, device=DEV)
    assert A.latent_read(cache, scale, torch.zeros(0, dtype=torch.int64, device=DEV)).shape == (0, 576)
