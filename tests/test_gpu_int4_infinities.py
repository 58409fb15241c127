"""4-bit products of tokens that are not finite: such a token's outputs are NaN
or infinities, all of them, since what is taken away for the weights' offset is
infinite too; those of the other tokens keep their bits.  Every form, by its
number of tokens."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def A():
    from routed_expert_int4_amd import attention
    return attention


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("M,N,K", [(1, 150, 512), (2, 150, 512), (3, 150, 512), (16, 150, 2304), (17, 150, 512), (32, 150, 2304), (29, 4200, 2304),
                                   (9, 12300, 256), (40, 150, 512), (64, 6200, 512), (130, 4100, 512), (256, 6144, 512), (1025, 6150, 384),
                                   (1000, 4100, 384)])
def test_a_token_keeps_to_itself(A, M, N, K, value, out_dtype):
    g = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scale = torch.rand(N, K // 32, generator=g, device=DEV).add(0.1).half()
    before = A.int4_linear(x, codes, scale, out_dtype=out_dtype)
    at = M // 2
    x[at, K - 5] = value
    after = A.int4_linear(x, codes, scale, out_dtype=out_dtype)
    others = torch.arange(M, device=DEV) != at
    assert bool(before.isfinite().all()) and not bool(after[at].isfinite().any())
    assert torch.equal(after[others], before[others])
    if value != value:
        assert bool(after[at].isnan().all())


@pytest.mark.parametrize("M", [1, 2, 16, 32, 64, 600])
def test_two_infinities(A, M):
    """Of either sign, in one group and in two."""
    g = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randn(M, 256, generator=g, device=DEV).bfloat16()
    codes = torch.randint(0, 256, (100, 128), generator=g, device=DEV, dtype=torch.uint8)
    scale = torch.rand(100, 8, generator=g, device=DEV).add(0.1).half()
    x[0, 3], x[0, 4] = float("inf"), -float("inf")
    x[M - 1, 3], x[M - 1, 200] = float("inf"), float("inf")
    out = A.int4_linear(x, codes, scale)
    assert not bool(out[0].isfinite().any()) and not bool(out[M - 1].isfinite().any())
    assert M < 3 or bool(out[1:M - 1].isfinite().all())
