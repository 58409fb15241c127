"""Weights in 4 bits as quantize_weight_int4 makes them, on the CPU, of any strides."""
import pytest

torch = pytest.importorskip("torch")

from routed_expert_int4_amd import attention as A  # noqa: E402


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
