"""Weights in 4 bits as quantize_weight_int4 makes them, on the CPU: any strides,
and which codes the ends of fp16's range leave."""
import pytest

torch = pytest.importorskip("torch")

from routed_expert_int4_amd import attention as A  # noqa: E402


def code(codes, n, k):
    c = int(codes[n, k // 2]) >> 4 * (k % 2) & 15
    return c - 16 if c > 7 else c


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float64])
@pytest.mark.parametrize("view", ["transposed", "columns", "every other column", "one row"])
def test_weights_of_any_strides(view, dtype, group):
    g = torch.Generator().manual_seed(0)
    w = {"transposed": torch.randn(256, 40, generator=g).to(dtype).t(),
         "columns": torch.randn(40, 512, generator=g).to(dtype)[:, 128:384],
         "every other column": torch.randn(40, 512, generator=g).to(dtype)[:, ::2],
         "one row": torch.randn(256, 1, generator=g).to(dtype).t()}[view]
    codes, scale = A.quantize_weight_int4(w, group)
    assert codes.is_contiguous() and scale.is_contiguous() and codes.dtype is torch.uint8 and scale.dtype is torch.float16
    want = A.quantize_weight_int4(w.contiguous(), group)
    assert torch.equal(codes, want[0]) and torch.equal(scale, want[1])


@pytest.mark.parametrize("group", [32, 64, 128])
def test_the_largest_magnitude_gets_code_7(group):
    """Where the scale is a normal fp16 number, 2^-14 to 65504: rounding it moves
    7 by 2^-11 of itself."""
    tops = torch.logspace(-14, 15, 59, base=2.0, dtype=torch.float64).mul(7 * 1.001).float()
    w = torch.rand(59, group, generator=torch.Generator().manual_seed(1)) * 1.8 - 0.9
    w[:, 3] = torch.where(torch.arange(59) % 2 == 0, 1.0, -1.0)
    codes, scale = A.quantize_weight_int4(w * tops[:, None], group)
    assert [code(codes, n, 3) for n in range(59)] == [7, -7] * 29 + [7]
    assert bool((scale >= 2.0 ** -14).all())


def test_ends_of_the_range():
    """Below, the scale is a multiple of 2^-24 (at least that one) and the largest
    code what that leaves, at most 7; above, codes end at 7 times 65504."""
    tops = [2.0 ** -24 * 7 * 1.4, 2.0 ** -24 * 7 * 1.6, 2.0 ** -24 * 3, 0.0, 7 * 70000.0, float("inf")]
    w = torch.zeros(len(tops), 32)
    w[:, 5] = torch.tensor(tops)
    codes, scale = A.quantize_weight_int4(w)
    assert [code(codes, n, 5) for n in range(len(tops))] == [7, 6, 3, 0, 7, 7]
    assert scale[:, 0].tolist() == [2.0 ** -24, 2.0 ** -23, 2.0 ** -24, 2.0 ** -24, 65504.0, 65504.0]
