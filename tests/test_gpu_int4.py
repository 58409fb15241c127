"""4-bit products against the formula in 64 bits.

Tolerance: a bf16 output is off by at most 2^-8 of its value (fp32: 2^-24).
The sums are fp32 and hold 1.5 + q / 16 per activation, at most 1.94, beside
the 1.5 that is taken away: every addition is off by at most 2^-23 (the matrix
unit may cut) of what has been added so far, at most 3.44 |x| summed over the
group, times 16 and the scale; a group makes 2 additions per column and the
groups are then added up, with a few more for the waves' sums."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def A():
    from routed_expert_int4_amd import attention
    return attention


def weight(N, K, group, seed, extremes=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    if extremes:  # -8 and 7 in turn, of every phase
        codes = torch.tensor([0x78, 0x87, 0x88, 0x77], dtype=torch.uint8, device=DEV)[torch.randint(0, 4, (N, K // 2), generator=g, device=DEV)]
    scale = torch.exp(torch.randn(N, K // group, generator=g, device=DEV) * 0.7 - 4).half()
    return codes, scale


def values(codes, scale):
    low, high = codes.to(torch.int16) & 15, codes.to(torch.int16) >> 4
    q = torch.stack([low, high], 2).flatten(1)
    q = torch.where(q > 7, q - 16, q).double()
    return q * scale.double().repeat_interleave(q.shape[1] // scale.shape[1], 1)


def check(out, x, codes, scale):
    want = x.double() @ values(codes, scale).t()
    K, groups = x.shape[1], scale.shape[1]
    spread = x.abs().double().view(x.shape[0], groups, -1).sum(2) @ scale.double().abs().t()
    half_step = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    bound = half_step * want.abs() + (2 * (K // groups) + groups + 32) * 2.0 ** -23 * 16 * 3.44 * spread
    off = (out.double() - want).abs()
    assert bool((off <= bound * (1 + 2.0 ** -8)).all()), float((off / bound.clamp_min(1e-300)).max())


def inputs(M, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(M, K, generator=g, device=DEV).bfloat16()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 576, 6144), (1, 17, 384), (2, 100, 1152), (5, 333, 640), (16, 48, 2048), (17, 64, 256),
                                   (32, 1000, 512), (33, 130, 896), (64, 64, 128), (100, 2048, 768), (129, 257, 1280), (300, 1500, 512),
                                   (700, 900, 384), (513, 6144, 256)])
def test_against_64_bits(A, M, N, K, group):
    codes, scale = weight(N, K, group, M * 31 + N)
    x = inputs(M, K, K + M)
    check(A.int4_linear(x, codes, scale), x, codes, scale)
    check(A.int4_linear(x, codes, scale, out_dtype=torch.float32), x, codes, scale)


@pytest.mark.parametrize("M", [1, 20, 40, 300, 600])
@pytest.mark.parametrize("K,group", [(32, 32), (64, 32), (96, 32), (64, 64), (192, 64), (160, 32), (1056, 32), (320, 64)])
def test_short_last_segments(A, M, K, group):
    codes, scale = weight(190, K, group, K + M)
    x = inputs(M, K, M)
    check(A.int4_linear(x, codes, scale, out_dtype=torch.float32), x, codes, scale)


@pytest.mark.parametrize("M", [1, 24, 200, 600])
def test_extreme_codes(A, M):
    codes, scale = weight(300, 512, 32, M, extremes=True)
    x = inputs(M, 512, M) * torch.tensor([1.0, 1e4], device=DEV).bfloat16().repeat(256)
    check(A.int4_linear(x, codes, scale, out_dtype=torch.float32), x, codes, scale)


@pytest.mark.parametrize("M", [1, 9, 30, 64, 100, 400])
def test_views(A, M):
    """Rows of wider tensors, an output in a wider one, and what lies beside it."""
    wide = inputs(M, 1024, 3)
    x = wide[:, 256:512]
    codes, scale = weight(200, 1024, 32, 4)
    c, s = codes[3:163, 64:192], scale[3:163, 5:13]
    out = torch.full((M, 200), 7.0, device=DEV, dtype=torch.bfloat16)
    got = A.int4_linear(x, c, s, out=out[:, 13:173])
    assert got.data_ptr() == out[:, 13:].data_ptr()
    check(got, x.contiguous(), c.contiguous(), s.contiguous())
    assert bool((out[:, :13] == 7).all()) and bool((out[:, 173:] == 7).all())


@pytest.mark.parametrize("M", [1, 40, 500])
def test_a_token_that_is_not_finite_keeps_to_itself(A, M):
    codes, scale = weight(150, 512, 32, 5)
    x = inputs(M, 512, 6)
    before = A.int4_linear(x, codes, scale)
    x[M // 2, 77] = float("nan")
    after = A.int4_linear(x, codes, scale)
    others = torch.arange(M, device=DEV) != M // 2
    assert bool(after[M // 2].isnan().all()) and torch.equal(after[others], before[others])


@pytest.mark.parametrize("M", [1, 30, 90, 700])
def test_same_bits_again_and_in_a_graph(A, M):
    codes, scale = weight(700, 1024, 64, 8)
    x = inputs(M, 1024, 9)
    want = A.int4_linear(x, codes, scale)
    out = torch.empty_like(want)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        A.int4_linear(x, codes, scale, out=out)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        A.int4_linear(x, codes, scale, out=out)
    for i in range(3):
        x.copy_(inputs(M, 1024, 20 + i))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, A.int4_linear(x, codes, scale))


def test_no_tokens_and_other_streams(A):
    codes, scale = weight(64, 256, 32, 1)
    assert A.int4_linear(inputs(1, 256, 0)[:0], codes, scale).shape == (0, 64)
    x = inputs(3, 256, 2)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out = A.int4_linear(x, codes, scale, stream=stream)
    stream.synchronize()
    assert torch.equal(out, A.int4_linear(x, codes, scale))


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantized_weights(A, group):
    g = torch.Generator(device=DEV).manual_seed(3)
    w = torch.randn(70, 256, generator=g, device=DEV)
    w[5] = 0
    codes, scale = A.quantize_weight_int4(w, group)
    back = values(codes, scale)
    # half a step of a scale that fp16 has rounded (2^-11 of it), up to 7 steps away
    step = scale.double().repeat_interleave(group, 1)
    assert bool(((back - w.double()).abs() <= step * (0.5 + 7 * 2.0 ** -10)).all())
    assert bool((back[5] == 0).all())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(4000, 2176), (4090, 8448), (4100, 2304), (8192, 8320), (8200, 2432), (1000, 2048), (12288, 256), (12290, 4224),
                                 (7, 16512)])
@pytest.mark.parametrize("M", [3, 16, 17, 32])
def test_forms_for_up_to_32_tokens(A, M, N, K, group):
    """Weight rows that fit one round over the chip in each form, and more;
    inner columns of one turn of a workgroup and of several."""
    codes, scale = weight(N, K, group, M + N + K)
    x = inputs(M, K, M + K)
    check(A.int4_linear(x, codes, scale), x, codes, scale)


@pytest.mark.parametrize("M", [3, 29])
@pytest.mark.parametrize("K,group", [(32, 32), (96, 32), (160, 32), (2080, 32), (4128, 32), (8224, 32), (2112, 64), (8256, 64)])
def test_short_last_stages(A, M, K, group):
    codes, scale = weight(70, K, group, K + M)
    x = inputs(M, K, M)
    check(A.int4_linear(x, codes, scale, out_dtype=torch.float32), x, codes, scale)


@pytest.mark.parametrize("M", [2, 9, 32, 64])
def test_what_lies_behind_the_columns_does_not_count(A, M):
    """Strided operands whose rows go on with values that are not finite."""
    N, K = 100, 544
    codes, scale = weight(N, K, 32, M)
    x = inputs(M, K, M)
    wide_x = torch.full((M, K + 64), float("nan"), device=DEV).bfloat16()
    wide_codes = torch.full((N, K // 2 + 48), 0x77, dtype=torch.uint8, device=DEV)
    wide_scale = torch.full((N, K // 32 + 3), float("inf"), device=DEV).half()
    wide_x[:, :K], wide_codes[:, :K // 2], wide_scale[:, :K // 32] = x, codes, scale
    out = A.int4_linear(wide_x[:, :K], wide_codes[:, :K // 2], wide_scale[:, :K // 32], out_dtype=torch.float32)
    check(out, x, codes, scale)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(40, 200, 8320), (64, 6200, 8448), (130, 4100, 8320), (256, 6144, 8448), (300, 7000, 640), (1025, 6150, 384),
                                   (640, 12300, 128)])
def test_forms_for_more_tokens(A, M, N, K, group):
    """Each shape of tiles, its last tiles cut by either edge, and inner
    columns of one turn of a workgroup and of two."""
    codes, scale = weight(N, K, group, M + N + K)
    x = inputs(M, K, M + K)
    check(A.int4_linear(x, codes, scale), x, codes, scale)
