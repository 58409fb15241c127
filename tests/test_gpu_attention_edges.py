"""GPU tests of the attention half at edges of its calls
(routed_expert_int4_amd/attention.py): empty operands, bounds, and the loops
that only longer inputs enter.  References in 64 bits and tolerances are those
of test_gpu_attention.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_int4_amd import attention as A  # noqa: E402
from test_gpu_attention import BF, D, DEV, U, close, cumulative, gen, latent_case, latent_ref, normal  # noqa: E402


@pytest.mark.parametrize("heads,nq", [(4, 1), (64, 3)])
def test_latent_attention_without_pages(heads, nq):
    g = gen(1)
    q = normal(g, 2 * nq, heads, 320)
    lens = torch.tensor([5, 0], dtype=torch.int32, device=DEV)
    pages = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    pool = normal(g, 4, 16, 320)
    for cache, table in ((pool[:0], pages), (pool, pages[:, :0].contiguous()), (pool[:0], pages[:, :0].contiguous())):
        out = A.latent_attention(q, cache, table, lens, 0.07)
        assert out.shape == (2 * nq, heads, 256) and (out == 0).all()


def test_latent_attention_with_a_loose_bound_of_tokens():
    # max_q only bounds: the launch that joins the parts of a sequence is sized by the tokens there are
    g = gen(2)
    nq, lens = [2, 3], [700, 300]
    q, cache, pages, dl = latent_case(g, lens, nq, 64, 512, 64)
    ref, mag = latent_ref(q, cache, pages, lens, nq, 0.07, 512)
    for max_q in (3, 5, 1 << 24):
        out = A.latent_attention(q, cache, pages, dl, 0.07, max_len=700, cu_q=cumulative(nq), max_q=max_q)
        close(out, ref, U * ref.abs() + U * mag, f"max_q {max_q}")
