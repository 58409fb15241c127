"""Host-side checks of the attention half of the C ABI (no GPU needed): what
is refused before anything is launched."""
from routed_expert_int4_amd import binding as B

P = 1 << 20  # an aligned address that nothing reads: every call here is refused


def latent(T=2, heads=64, B_=1, max_q=2, max_len=64, cu_q=P, per_seq=4):
    L = B.lib()
    ws = L.moe_latent_attention_workspace(B_, max_q, heads, 512, max_len)
    return L.moe_latent_attention(P, heads * 576, 576, T, heads, 512, 64, P, 8, 64, 64 * 576, P, per_seq, per_seq, P, B_, cu_q,
                                  max_q, max_len, None, 0.1, P, heads * 512, 512, P, ws, None)


def test_latent_attention_rows_that_a_launch_cannot_count():
    assert latent(T=1 << 20, max_q=1 << 20) == B.MOE_EUNSUPPORTED and "2^26" in B.last_error()
    assert latent(T=1 << 20, max_q=1 << 20, cu_q=None) == B.MOE_EUNSUPPORTED
