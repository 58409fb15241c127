"""GPU tests of the attention half at edges of its calls
(routed_expert_int4_amd/attention.py): empty operands, bounds, and the loops
that only longer inputs enter.  References in 64 bits and tolerances are those
of test_gpu_attention.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from routed_expert_int4_amd import attention as A  # noqa: E402
from test_gpu_attention import BF, D, DEV, U, close, cumulative, gen, latent_case, latent_ref, normal, prompt_ref  # noqa: E402


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


@pytest.mark.parametrize("bounds", [[0, 6, 0, 6], [0, 6, 5, 9], [3, 6, 0, 6]])
def test_latent_attention_bounds_that_overlap(bounds):
    # together they name more tokens than there are: nothing is computed
    g = gen(3)
    lens = [700, 300, 90]
    q, cache, pages, dl = latent_case(g, lens, [2, 2, 2], 64, 512, 64)
    cu = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    out = torch.full((6, 64, 512), -7.0, dtype=BF, device=DEV)
    A.latent_attention(q, cache, pages, dl, 0.07, max_len=700, cu_q=cu, max_q=6, out=out)
    assert (out == -7.0).all()


def test_latent_attention_many_sequences_with_bounds():
    # more sequences than lanes, some without tokens, and rows of q in no sequence
    g = gen(4)
    nq = [(i * 7) % 4 for i in range(150)]
    lens = [max(n, (i * 37) % 260 + 1) for i, n in enumerate(nq)]
    q, cache, pages, dl = latent_case(g, lens, nq, 16, 256, 32)
    ref, mag = latent_ref(q, cache, pages, lens, nq, 0.07, 256)
    T = sum(nq)
    wide = torch.cat([normal(g, 5, 16, 320), q, normal(g, 3, 16, 320)])
    out = torch.full((T + 8, 16, 256), -7.0, dtype=BF, device=DEV)
    A.latent_attention(wide, cache, pages, dl, 0.07, max_len=260, cu_q=cumulative(nq) + 5, max_q=3, out=out)
    close(out[5:T + 5], ref, U * ref.abs() + U * mag)
    assert (out[:5] == -7.0).all() and (out[T + 5:] == -7.0).all()


def test_prompt_attention_rows_in_no_sequence():
    g = gen(5)
    q, k, v, kr = normal(g, 40, 2, 128), normal(g, 40, 2, 64), normal(g, 40, 2, 64), normal(g, 40, 64)
    cu = torch.tensor([3, 20, 33], dtype=torch.int32, device=DEV)
    out = torch.full((40, 2, 64), -7.0, dtype=BF, device=DEV)
    A.prompt_attention(q, k, kr, v, 0.08, cu_q=cu, cu_k=cu, max_q=17, out=out)
    ref, mag = prompt_ref(q[3:33], k[3:33], kr[3:33], v[3:33], [17, 13], [17, 13], 0.08)
    close(out[3:33], ref, U * ref.abs() + U * mag)
    assert (out[:3] == -7.0).all() and (out[33:] == -7.0).all()
