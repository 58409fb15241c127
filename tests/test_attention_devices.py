"""CPU tests: operands of one call on different devices are refused before
anything runs (routed_expert_int4_amd/attention.py).  There are no GPUs here:
tensors on the CPU that say they are on one stand in for theirs."""
import pytest

torch = pytest.importorskip("torch")

from routed_expert_int4_amd import attention as A  # noqa: E402
from routed_expert_int4_amd import binding as B  # noqa: E402

BF, F32, F8, I32, I64 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32, torch.int64


class On:
    """A tensor that says it is on a device."""

    def __init__(self, tensor, device):
        self.tensor, self.device, self.is_cuda = tensor, torch.device(device), device != "cpu"

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def __getattr__(self, name):
        return getattr(self.tensor, name)


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def norm(p):
    A.add_rmsnorm(p(z(2, 128)), p(z(128)), residual=p(z(2, 128)), sum_out=p(z(2, 128)))


def linear(p):
    A.fp8_linear(p(z(2, 128, dtype=F8)), p(z(2, 1, dtype=F32)), p(z(128, 128, dtype=F8)), p(z(1, 1, dtype=F32)), out=p(z(2, 128)))


def heads(p):
    A.head_linear(p(z(2, 4, 64)), p(z(4, 8, 64)), out=p(z(2, 4, 8)))


def append(p):
    A.latent_append(p(z(2, 320)), p(z(256)), 1e-6, p(z(8, 64, dtype=F32)), p(z(2, dtype=I32)), p(z(2, dtype=I64)),
                    p(z(2, 16, 320)), q_rope=p(z(2, 4, 64)), q_out=p(z(2, 4, 64)))


def latent(p):
    A.latent_attention(p(z(2, 4, 320)), p(z(2, 16, 320)), p(z(2, 1, dtype=I32)), p(z(2, dtype=I32)), 1.0, cu_q=p(z(3, dtype=I32)),
                       max_q=1, tree=p(z(2, dtype=I64)), out=p(z(2, 4, 256)), workspace=p(z(1 << 23, dtype=torch.uint8)))


def prompt(p):
    A.prompt_attention(p(z(2, 4, 128)), p(z(2, 4, 64)), p(z(2, 64)), p(z(2, 4, 64)), 1.0, cu_q=p(z(2, dtype=I32)),
                       cu_k=p(z(2, dtype=I32)), max_q=2, out=p(z(2, 4, 64)))


CALLS = {norm: 4, linear: 5, heads: 3, append: 8, latent: 8, prompt: 7}


class Guard:
    """Stands in for torch.cuda.device."""
    current = [0]

    def __init__(self, device):
        self.device = torch.device(device)

    def __enter__(self):
        Guard.current.append(self.device.index)

    def __exit__(self, *_):
        Guard.current.pop()


@pytest.fixture
def launched(monkeypatch):
    """The calls that got as far as a launch: (current device, stream)."""
    calls, empty = [], torch.empty

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append((Guard.current[-1], args[-1])) or B.MOE_OK

    monkeypatch.setattr(B, "lib", Library)
    monkeypatch.setattr(torch, "empty", lambda *a, device, **k: empty(*a, **k))
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(A, "_device", lambda: Guard.current[-1])
    monkeypatch.setattr(A, "_raw_stream", lambda index: 100 + index)
    return calls


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
@pytest.mark.parametrize("other", ["cuda:1", "cpu"])
def test_one_operand_elsewhere(call, other, launched):
    for odd in range(CALLS[call]):
        count = iter(range(100))
        with pytest.raises(B.MoeError) as e:
            call(lambda t: On(t, other if next(count) == odd else "cuda:0"))
        assert e.value.code == B.MOE_EINVAL and not launched, odd
        assert next(count) <= CALLS[call]


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
@pytest.mark.parametrize("device", [0, 1])
def test_launches_go_to_the_operands_device(call, device, launched):
    call(lambda t: On(t, f"cuda:{device}"))
    assert launched == [(device, 100 + device)] and Guard.current == [0]


def test_a_stream_for_operands_on_the_cpu(launched):
    with pytest.raises(B.MoeError):
        A.quantize(On(z(2, 128), "cpu"), stream=5)
