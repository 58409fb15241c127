"""Token bounds that decrease, with a prefix: which rows have it.

cu_q = [4, 0, 2, 6, 6] over six tokens names none in the first sequence and the
last, tokens 0 and 1 in the second and 2 to 5 in the third.  The prefix belongs
to sequences 0 to 2, whose tokens start at cu_q[0] = 4 and end at cu_q[3] = 6: so
tokens 4 and 5 have it, and the others their own rows alone."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from tests.test_gpu_shared_prefix import D, U, Case, ints  # noqa: E402


@pytest.fixture(scope="module")
def A():
    from routed_expert_int4_amd import attention
    return attention


@pytest.mark.parametrize("narrow", [False, True])
def test_bounds_that_decrease_and_a_prefix(A, narrow):
    c = Case([20, 65, 30, 40], [0, 2, 0, 4], 512, 16, 16, narrow, [100], [0, 3])
    out = torch.full((6, 16, 512), 7.0, dtype=torch.bfloat16, device=c.q.device)
    A.latent_attention(c.q, c.cache, c.pages, ints(c.lens), c.softmax_scale, max_len=65, cu_q=ints([4, 0, 2, 6, 6]), max_q=6, out=out,
                       cache_scale=c.scale_of if narrow else None, prefix=c.prefix(A))
    before, _ = c.rows(c.prefix_pages[0], 100)
    for t, (b, i, new) in enumerate([(1, 0, 2), (1, 1, 2), (2, 0, 4), (2, 1, 4), (2, 2, 4), (2, 3, 4)]):
        own, _ = c.rows(c.pages[b], c.lens[b])
        kv = torch.cat([before[:100 if t >= 4 else 0], own[:c.lens[b] - new + i + 1]])
        w = torch.softmax(c.q[t].to(D) @ kv.t() * c.softmax_scale, 1)
        ref, mag = w @ kv[:, :512], w @ kv[:, :512].abs()
        over = (out[t].to(D) - ref).abs() - U * (ref.abs() + mag) - len(kv) * 448 * 2.0 ** -126  # as for bounds that do not decrease
        assert bool(out[t].isfinite().all()) and float(over.max()) <= 0, (t, float(over.max()))
