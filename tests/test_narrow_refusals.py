"""CPU tests of what the 4-bit product, the 8-bit latent cache and attention
with prefixes refuse before anything is launched, and of calls on devices other
than the current one.  There are no GPUs here: tensors on the CPU that say they
are on one stand in for theirs, and the library's own checks get addresses that
nothing reads."""
import pytest

torch = pytest.importorskip("torch")

from routed_expert_int4_amd import attention as A  # noqa: E402
from routed_expert_int4_amd import binding as B  # noqa: E402
from tests.test_attention_devices import Guard, On, launched, z  # noqa: E402, F401

BF, F16, F32, F8, I32, I64, U8 = (torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.int32, torch.int64,
                                  torch.uint8)
P = 1 << 20  # an aligned address that nothing reads: every call here is refused


# ------------------------------------------------------------------ devices
def int4(p):
    A.int4_linear(p(z(2, 128)), p(z(8, 64, dtype=U8)), p(z(8, 4, dtype=F16)), out=p(z(2, 8)))


def append(p):
    A.latent_append(p(z(2, 320)), p(z(256)), 1e-6, p(z(8, 64, dtype=F32)), p(z(2, dtype=I32)), p(z(2, dtype=I64)),
                    p(z(2, 16, 384, dtype=U8)), q_rope=p(z(2, 4, 64)), q_out=p(z(2, 4, 64)), cache_scale=p(z(2, 16, dtype=F32)))


def read(p):
    A.latent_read(p(z(2, 16, 384, dtype=U8)), p(z(2, 16, dtype=F32)), p(z(2, dtype=I64)), out=p(z(2, 320)))


def attend(p):
    prefix = A.SharedPrefix(p(z(2, 1, dtype=I32)), p(z(2, dtype=I32)), 16, p(z(3, dtype=I32)))
    A.latent_attention(p(z(2, 4, 320)), p(z(2, 16, 384, dtype=U8)), p(z(2, 1, dtype=I32)), p(z(2, dtype=I32)), 1.0,
                       cu_q=p(z(3, dtype=I32)), max_q=1, tree=p(z(2, dtype=I64)), out=p(z(2, 4, 256)),
                       workspace=p(z(1 << 23, dtype=U8)), cache_scale=p(z(2, 16, dtype=F32)), prefix=prefix)


CALLS = {int4: 4, append: 9, read: 4, attend: 12}


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
@pytest.mark.parametrize("other", ["cuda:1", "cpu"])
def test_one_operand_elsewhere(call, other, launched):  # noqa: F811
    for odd in range(CALLS[call]):
        count = iter(range(100))
        with pytest.raises(B.MoeError) as e:
            call(lambda t: On(t, other if next(count) == odd else "cuda:0"))
        assert e.value.code == B.MOE_EINVAL and not launched, odd
        assert next(count) <= CALLS[call]


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
@pytest.mark.parametrize("device", [0, 1])
def test_launches_go_to_the_operands_device(call, device, launched):  # noqa: F811
    call(lambda t: On(t, f"cuda:{device}"))
    assert launched == [(device, 100 + device)] and Guard.current == [0]


# ------------------------------------------------------------------ shapes and types
def on0(t):
    return On(t, "cuda:0")


def refused(f):
    with pytest.raises(B.MoeError) as e:
        f()
    assert e.value.code == B.MOE_EINVAL


@pytest.mark.parametrize("x,codes,scale", [
    (z(2, 128), z(8, 32, dtype=U8), z(8, 4, dtype=F16)),                 # columns
    (z(2, 128), z(8, 64, dtype=U8), z(7, 4, dtype=F16)),                 # rows
    (z(2, 128), z(8, 64, dtype=U8), z(8, 8, dtype=F16)),                 # groups of 16
    (z(2, 96), z(8, 48, dtype=U8), z(8, 2, dtype=F16)),                  # groups of 48
    (z(2, 128), z(8, 64, dtype=U8), z(8, 0, dtype=F16)),
    (z(2, 128), z(8, 64, dtype=U8), z(8, 4, dtype=F32)),
    (z(2, 128, dtype=F32), z(8, 64, dtype=U8), z(8, 4, dtype=F16)),
    (z(2, 128), z(8, 64, dtype=I32), z(8, 4, dtype=F16)),
    (z(128, 2).t(), z(8, 64, dtype=U8), z(8, 4, dtype=F16)),
    (z(128), z(8, 64, dtype=U8), z(8, 4, dtype=F16)),
])
def test_int4_operands(x, codes, scale, launched):  # noqa: F811
    refused(lambda: A.int4_linear(on0(x), on0(codes), on0(scale)))
    assert not launched


def test_int4_outputs_and_groups(launched):  # noqa: F811
    ok = on0(z(2, 128)), on0(z(8, 64, dtype=U8)), on0(z(8, 4, dtype=F16))
    refused(lambda: A.int4_linear(*ok, out=on0(z(2, 7))))
    refused(lambda: A.int4_linear(*ok, out=on0(z(2, 8, dtype=F16))))
    refused(lambda: A.int4_linear(*ok, out_dtype=F16))
    refused(lambda: A.quantize_weight_int4(z(4, 128), 16))
    refused(lambda: A.quantize_weight_int4(z(4, 100), 32))
    assert not launched


def test_narrow_cache_operands(launched):  # noqa: F811
    cache, scale, slots = z(2, 16, 384, dtype=U8), z(2, 16, dtype=F32), z(2, dtype=I64)
    for c, s in ((z(2, 16, 384), scale), (cache, z(2, 15, dtype=F32)), (cache, z(2, 16)), (cache[:, ::2], z(2, 8, dtype=F32)),
                 (cache, z(16, 2, dtype=F32).t())):
        refused(lambda: A.latent_read(on0(c), on0(s), on0(slots)))
        refused(lambda: A.latent_append(on0(z(2, 320)), on0(z(256)), 1e-6, on0(z(8, 64, dtype=F32)), on0(z(2, dtype=I32)), on0(slots),
                                        on0(c), cache_scale=on0(s)))
        refused(lambda: A.latent_attention(on0(z(2, 4, 320)), on0(c), on0(z(2, 1, dtype=I32)), on0(z(2, dtype=I32)), 1.0,
                                           cache_scale=on0(s)))
    refused(lambda: A.latent_read(on0(cache), on0(scale), on0(z(2, dtype=I32))))
    refused(lambda: A.latent_read(on0(cache), on0(scale), on0(slots), rope=192))
    refused(lambda: A.latent_read(on0(cache), on0(scale), on0(slots), out=on0(z(2, 321))))
    given = on0(z(2, 320)), on0(z(256)), 1e-6, on0(z(8, 64, dtype=F32)), on0(z(2, dtype=I32))
    refused(lambda: A.latent_append(*given, cache_scale=on0(scale)))                      # no cache
    refused(lambda: A.latent_append(*given, None, on0(cache), cache_scale=on0(scale)))    # no slots
    refused(lambda: A.latent_append(*given, on0(slots), on0(cache)))                      # 8 bits without scales
    refused(lambda: A.latent_append(*given, on0(slots), on0(cache), cache_scale=on0(scale), want_fp8=True))
    refused(lambda: A.latent_append(*given, on0(slots[:1]), on0(cache), cache_scale=on0(scale)))
    assert not launched


def test_prefix_operands(launched):  # noqa: F811
    def call(prefix, **more):
        A.latent_attention(on0(z(2, 4, 320)), on0(z(2, 16, 320)), on0(z(2, 1, dtype=I32)), on0(z(2, dtype=I32)), 1.0, prefix=prefix,
                           workspace=on0(z(1 << 20, dtype=U8)), out=on0(z(2, 4, 256)), **more)
    pages, lens, groups = z(2, 1, dtype=I32), z(2, dtype=I32), z(3, dtype=I32)
    for p in ((z(2, 1), lens, 16, groups), (pages, z(1, dtype=I32), 16, groups), (pages, lens, 16, None), (pages, lens, 16, z(2, dtype=I32)),
              (pages, z(2, dtype=I64), 16, groups), (z(0, 1, dtype=I32), z(0, dtype=I32), 16, None)):
        refused(lambda: call(A.SharedPrefix(*(on0(t) if isinstance(t, torch.Tensor) else t for t in p))))
    assert not launched
    call(A.SharedPrefix(on0(pages[:1]), on0(lens[:1])))
    assert len(launched) == 1


# ------------------------------------------------------------------ the library's own checks
def code(status, what):
    assert status == what, B.last_error()
    assert B.last_error()


def test_int4_abi():
    L = B.lib()

    def call(x=P, x_stride=256, w=P, w_stride=128, scale=P, s_stride=8, group=32, M=4, N=8, K=256, out=P, type_=0, o_stride=8):
        return L.moe_int4_linear(x, x_stride, w, w_stride, scale, s_stride, group, M, N, K, out, type_, o_stride, None)
    for more, what in ((dict(M=-1), B.MOE_EINVAL), (dict(N=0), B.MOE_EINVAL), (dict(K=0), B.MOE_EINVAL), (dict(group=16), B.MOE_EUNSUPPORTED),
                       (dict(K=240), B.MOE_EINVAL), (dict(type_=2), B.MOE_EINVAL), (dict(x=None), B.MOE_EINVAL), (dict(w=None), B.MOE_EINVAL),
                       (dict(scale=None), B.MOE_EINVAL), (dict(out=None), B.MOE_EINVAL), (dict(x_stride=248), B.MOE_EINVAL),
                       (dict(w_stride=112), B.MOE_EINVAL), (dict(s_stride=7), B.MOE_EINVAL), (dict(o_stride=7), B.MOE_EINVAL),
                       (dict(x_stride=260), B.MOE_EUNSUPPORTED), (dict(w_stride=136), B.MOE_EUNSUPPORTED), (dict(x=P + 8), B.MOE_EUNSUPPORTED),
                       (dict(w=P + 8), B.MOE_EUNSUPPORTED), (dict(scale=P + 1), B.MOE_EINVAL), (dict(out=P + 1), B.MOE_EINVAL),
                       (dict(out=P + 2, type_=1), B.MOE_EINVAL), (dict(M=1 << 20, N=1 << 20, o_stride=1 << 20), B.MOE_EUNSUPPORTED), (dict(M=1, N=(1 << 26) + 1, o_stride=1 << 27), B.MOE_EUNSUPPORTED),
                       (dict(x_stride=1 << 22), B.MOE_EUNSUPPORTED), (dict(w_stride=1 << 23), B.MOE_EUNSUPPORTED)):
        code(call(**more), what)
    assert call(M=0, x=None) == B.MOE_OK


def test_read_abi():
    L = B.lib()

    def call(cache=P, scale=P, n=64, rank=256, rope=64, slots=P, T=3, out=P, stride=320):
        return L.moe_latent_read_fp8(cache, scale, n, rank, rope, slots, T, out, stride, None)
    for more, what in ((dict(T=-1), B.MOE_EINVAL), (dict(n=-1), B.MOE_EINVAL), (dict(rank=0), B.MOE_EINVAL), (dict(rope=0), B.MOE_EINVAL),
                       (dict(cache=None), B.MOE_EINVAL), (dict(scale=None), B.MOE_EINVAL), (dict(slots=None), B.MOE_EINVAL),
                       (dict(out=None), B.MOE_EINVAL), (dict(stride=312), B.MOE_EINVAL), (dict(rank=248, stride=320), B.MOE_EUNSUPPORTED),
                       (dict(rope=60), B.MOE_EUNSUPPORTED), (dict(stride=324), B.MOE_EUNSUPPORTED), (dict(out=P + 8), B.MOE_EUNSUPPORTED),
                       (dict(cache=P + 8), B.MOE_EUNSUPPORTED), (dict(slots=P + 4), B.MOE_EINVAL), (dict(scale=P + 2), B.MOE_EINVAL),
                       (dict(rank=4096, stride=8192), B.MOE_EUNSUPPORTED), (dict(rank=2048, T=1 << 30, stride=4096), B.MOE_EUNSUPPORTED)):
        code(call(**more), what)
    assert call(T=0, cache=None) == B.MOE_OK


def test_append_abi():
    L = B.lib()

    def call(cache=P, scale=P, rank=256, T=3, slots=P, n=64):
        return L.moe_latent_append_fp8(P, 576, P, 0, 1e-6, rank, 64, P, 10, P, slots, T, cache, scale, n, None, 0, 0, 0, None, 0, 0,
                                       None, 0, None)
    for more, what in ((dict(cache=None), B.MOE_EINVAL), (dict(scale=None), B.MOE_EINVAL), (dict(slots=None), B.MOE_EINVAL),
                       (dict(rank=248), B.MOE_EUNSUPPORTED), (dict(cache=P + 8), B.MOE_EUNSUPPORTED), (dict(scale=P + 2), B.MOE_EINVAL),
                       (dict(n=-1), B.MOE_EINVAL), (dict(T=-1), B.MOE_EINVAL)):
        code(call(**more), what)
    assert call(T=0, cache=None, scale=None) == B.MOE_OK


def test_attention_abi():
    L = B.lib()

    def call(T=2, heads=64, scale=P, page_stride=64 * 640, B_=2, prefixes=1, p_pages=P, p_stride=4, per=4, p_lens=P, groups=P, p_most=256,
             ws=P, ws_bytes=None, cu_q=None, max_q=1, page=64):
        need = L.moe_latent_attention_shared_workspace(B_, T, max_q, heads, 512, 64, prefixes, max(p_most, 0))
        return L.moe_latent_attention_shared(P, heads * 576, 576, T, heads, 512, 64, P, scale, 64, page, page_stride, P, 4, 4, P, B_, cu_q,
                                             max_q, 64, None, p_pages, p_stride, per, p_lens, groups, prefixes, p_most, 0.1, P, heads * 512,
                                             512, ws, need if ws_bytes is None else ws_bytes, None)
    for more, what in ((dict(prefixes=-1), B.MOE_EINVAL), (dict(per=-1), B.MOE_EINVAL), (dict(p_most=-1), B.MOE_EINVAL),
                       (dict(p_pages=None), B.MOE_EINVAL), (dict(p_lens=None), B.MOE_EINVAL), (dict(prefixes=2, groups=None), B.MOE_EINVAL),
                       (dict(p_stride=3), B.MOE_EINVAL), (dict(prefixes=65536), B.MOE_EUNSUPPORTED), (dict(p_pages=P + 2), B.MOE_EINVAL),
                       (dict(groups=P + 2), B.MOE_EINVAL), (dict(p_lens=P + 1), B.MOE_EINVAL), (dict(scale=P + 2), B.MOE_EINVAL),
                       (dict(page_stride=64 * 640 - 16), B.MOE_EINVAL), (dict(page_stride=64 * 640 + 8), B.MOE_EUNSUPPORTED),
                       (dict(scale=None, page_stride=64 * 575), B.MOE_EINVAL), (dict(ws=None), B.MOE_EINVAL), (dict(ws=P + 128), B.MOE_EINVAL),
                       (dict(ws_bytes=1000), B.MOE_EINVAL), (dict(T=1 << 20, cu_q=P, max_q=1, B_=1), B.MOE_EUNSUPPORTED),
                       (dict(per=1 << 26, p_stride=1 << 26), B.MOE_EUNSUPPORTED)):
        code(call(**more), what)
    assert call(T=0) == B.MOE_OK


def test_workspaces():
    L = B.lib()
    wide = L.moe_latent_attention_workspace(8, 1, 64, 512, 4096)
    assert L.moe_latent_attention_shared_workspace(8, 8, 1, 64, 512, 4096, 0, 0) == wide
    one = L.moe_latent_attention_shared_workspace(8, 8, 1, 64, 512, 4096, 1, 4096)
    assert one >= 2 * 8 * 64 * 514 * 4
    assert L.moe_latent_attention_shared_workspace(8, 8, 1, 64, 512, 4096, 1, -1) == 0
    assert L.moe_latent_attention_shared_workspace(8, 0, 1, 64, 512, 4096, 1, 64) == 0
