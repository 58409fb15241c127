"""The attention half of a decoder block: what stands between two routed
layers of a model with latent attention, as calls on torch tensors.

    add_rmsnorm       residual addition and root-mean-square norm, bf16 and / or 8-bit output
    fp8_linear        8-bit product with a scale per 128 columns (activations) and 128 x 128 block (weights)
    head_linear       one product per head (queries into the latent space, outputs back out)
    latent_append     norm, rotation and write of new rows of the latent cache
    latent_attention  attention over the paged latent cache (single tokens, chunks, trees of drafted tokens)
    prompt_attention  the same attention with keys and values expanded per head, for prompts

Every step runs in the HIP kernels behind include/moe.h; this module checks
shapes and types, allocates outputs where none are given, and passes pointers
and strides.  Calls run on torch's current stream unless `stream` is given,
return at once, and can be captured in a graph.  There is no CPU fallback.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding as B

_BF16, _F32, _FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_TYPES = {_BF16: 0, _F32: 1}  # MOE_BF16, MOE_F32
GROUP = 128                   # columns (and weight rows) that share a scale


class NormOut(NamedTuple):
    """Outputs of add_rmsnorm; None where not asked for."""
    sum: torch.Tensor | None    # x + residual, in the residual's type
    y: torch.Tensor | None      # bf16
    q: torch.Tensor | None      # 8-bit
    scale: torch.Tensor | None  # fp32 [T, ceil(H / 128)]


class AppendOut(NamedTuple):
    """Outputs of latent_append; None where not asked for."""
    q_rope: torch.Tensor | None  # rotated position part of the queries
    q: torch.Tensor | None       # the normed latent in 8 bits
    scale: torch.Tensor | None
    key: torch.Tensor | None     # rotated position part of the keys


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise B.MoeError(B.MOE_EINVAL, what)


def _rows(t: torch.Tensor, name: str, dims: int, dtypes) -> None:
    """A device tensor of `dims` dimensions with a contiguous last one."""
    if t.dim() != dims or t.dtype not in dtypes or not t.is_cuda or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise B.MoeError(B.MOE_EINVAL, f"{name}: a device tensor of {dims} dimensions, contiguous in the last, of type "
                                       f"{' or '.join(str(d) for d in dtypes)} is needed, got {t.dtype} {tuple(t.shape)} "
                                       f"with strides {t.stride()} on {t.device}")


def _scales(T: int, H: int, device) -> torch.Tensor:
    """[T, groups] stored group by group, the order fp8_linear reads fastest."""
    return torch.empty_strided((T, (H + GROUP - 1) // GROUP), (1, T), dtype=_F32, device=device)


def _codes(T: int, H: int, device) -> torch.Tensor:
    """[T, H] of 8-bit codes, rows a multiple of 16 bytes apart."""
    pad = -(-H // 16) * 16
    return torch.empty_strided((T, H), (pad, 1), dtype=_FP8, device=device)


def add_rmsnorm(x, weight, eps: float = 1e-6, residual=None, out: str = "bf16", sum_out=None, want_sum: bool = True,
                stream=None) -> NormOut:
    """h = x + residual and its root-mean-square norm times weight.

    x [T, H] bf16 or fp32, weight [H], residual [T, H] or None.  out: "bf16",
    "fp8" (codes and one scale per 128 columns) or "both".  h is returned in
    the residual's type (sum_out, which may be the residual itself, receives
    it in place; want_sum=False leaves it out)."""
    _rows(x, "x", 2, (_BF16, _F32))
    _rows(weight, "weight", 1, (_BF16, _F32))
    T, H = x.shape
    _need(weight.shape[0] == H, f"weight has {weight.shape[0]} values, x {H} columns")
    r_stride, r_type, sum_type = 0, 0, x.dtype
    if residual is not None:
        _rows(residual, "residual", 2, (_BF16, _F32))
        _need(residual.shape == x.shape, f"residual {tuple(residual.shape)}, x {tuple(x.shape)}")
        r_stride, sum_type = residual.stride(0) if T > 1 else H, residual.dtype
        r_type = _TYPES[sum_type]
    dev = x.device
    if sum_out is not None:
        _rows(sum_out, "sum_out", 2, (sum_type,))
        _need(sum_out.shape == x.shape, f"sum_out {tuple(sum_out.shape)}, x {tuple(x.shape)}")
    elif want_sum and residual is not None:
        sum_out = torch.empty((T, H), dtype=sum_type, device=dev)
    _need(out in ("bf16", "fp8", "both"), f"out: {out!r}")
    y = torch.empty((T, H), dtype=_BF16, device=dev) if out != "fp8" else None
    q = scale = None
    if out != "bf16":
        q, scale = _codes(T, H, dev), _scales(T, H, dev)
    B.check(B.lib().moe_add_rmsnorm(
        x.data_ptr(), _TYPES[x.dtype], x.stride(0) if T > 1 else H, residual.data_ptr() if residual is not None else None,
        r_type, r_stride, weight.data_ptr(), _TYPES[weight.dtype], T, H, eps,
        sum_out.data_ptr() if sum_out is not None else None, sum_out.stride(0) if sum_out is not None and T > 1 else H,
        y.data_ptr() if y is not None else None, H, q.data_ptr() if q is not None else None,
        q.stride(0) if q is not None else H, scale.data_ptr() if scale is not None else None, 1, T,
        B._stream_handle(stream)))
    return NormOut(sum_out, y, q, scale)


def fp8_linear(a, a_scale, w, w_scale, out_dtype=_BF16, out=None, stream=None) -> torch.Tensor:
    """a [M, K] 8-bit with a_scale [M, ceil(K / 128)] times the transpose of
    w [N, K] 8-bit with w_scale [ceil(N / 128), ceil(K / 128)]: [M, N] in
    out_dtype (bf16 or fp32).  K is a multiple of 16; a_scale may have any
    strides (add_rmsnorm's are the fastest)."""
    _rows(a, "a", 2, (_FP8,))
    _rows(w, "w", 2, (_FP8,))
    _rows(w_scale, "w_scale", 2, (_F32,))
    (M, K), N = a.shape, w.shape[0]
    kb = (K + GROUP - 1) // GROUP
    _need(w.shape[1] == K, f"a has {K} inner columns, w {w.shape[1]}")
    _need(a_scale.dtype == _F32 and a_scale.is_cuda and tuple(a_scale.shape) == (M, kb),
          f"a_scale: fp32 {(M, kb)} on the device is needed, got {a_scale.dtype} {tuple(a_scale.shape)}")
    _need(tuple(w_scale.shape) == ((N + GROUP - 1) // GROUP, kb),
          f"w_scale {tuple(w_scale.shape)}, {((N + GROUP - 1) // GROUP, kb)} is needed")
    if out is None:
        _need(out_dtype in _TYPES, f"out_dtype {out_dtype}: bf16 or fp32")
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    else:
        _rows(out, "out", 2, (_BF16, _F32))
        _need(tuple(out.shape) == (M, N), f"out {tuple(out.shape)}, {(M, N)} is needed")
    B.check(B.lib().moe_fp8_linear(
        a.data_ptr(), a.stride(0) if M > 1 else -(-K // 16) * 16, a_scale.data_ptr(), a_scale.stride(0),
        a_scale.stride(1), w.data_ptr(), w.stride(0) if N > 1 else -(-K // 16) * 16, w_scale.data_ptr(),
        w_scale.stride(0) if w_scale.shape[0] > 1 else kb, M, N, K, out.data_ptr(), _TYPES[out.dtype],
        out.stride(0) if M > 1 else N, B._stream_handle(stream)))
    return out


def head_linear(x, w, out=None, stream=None) -> torch.Tensor:
    """x [T, heads, K] times the transpose of w [heads, N, K], head by head:
    [T, heads, N], all bf16.  x and out may be strided views (of a wider
    query, say)."""
    _rows(x, "x", 3, (_BF16,))
    _rows(w, "w", 3, (_BF16,))
    T, heads, K = x.shape
    N = w.shape[1]
    _need(w.shape[0] == heads and w.shape[2] == K and w.is_contiguous(),
          f"w: contiguous {(heads, 'N', K)} is needed, got {tuple(w.shape)} with strides {w.stride()}")
    if out is None:
        out = torch.empty((T, heads, N), dtype=_BF16, device=x.device)
    else:
        _rows(out, "out", 3, (_BF16,))
        _need(tuple(out.shape) == (T, heads, N), f"out {tuple(out.shape)}, {(T, heads, N)} is needed")
    B.check(B.lib().moe_head_linear(x.data_ptr(), x.stride(0), x.stride(1), w.data_ptr(), T, heads, K, N,
                                    out.data_ptr(), out.stride(0), out.stride(1), B._stream_handle(stream)))
    return out


def latent_append(kv, weight, eps, table, positions, slots=None, cache=None, q_rope=None, q_out=None,
                  want_fp8: bool = False, want_key: bool = False, stream=None) -> AppendOut:
    """Norms the latents and rotates the position parts of new tokens and
    writes them to their rows of the cache.

    kv [T, rank + rope] bf16, weight [rank], table fp32 [positions, rope]
    (cosines, then sines), positions int32 [T], slots int64 [T] (row of the
    cache, page * page_size + place; negative: not written), cache [pages,
    page_size, rank + rope] contiguous.  q_rope [T, heads, rope] is rotated
    into q_out (given, the view itself for in place, or new).  want_fp8: the
    normed latent in 8 bits too; want_key: the rotated key part too."""
    _rows(kv, "kv", 2, (_BF16,))
    _rows(weight, "weight", 1, (_BF16, _F32))
    _rows(table, "table", 2, (_F32,))
    _rows(positions, "positions", 1, (torch.int32,))
    T, rank, rope = kv.shape[0], weight.shape[0], table.shape[1]
    _need(kv.shape[1] == rank + rope, f"kv has {kv.shape[1]} columns, weight and table {rank} + {rope}")
    _need(positions.shape[0] == T and table.is_contiguous(), "positions: one per token; table: contiguous")
    cache_p = slots_p = None
    n_slots = 0
    if cache is not None:
        _need(cache.dtype == _BF16 and cache.is_cuda and cache.is_contiguous() and cache.shape[-1] == rank + rope,
              f"cache: contiguous bf16 rows of {rank + rope} are needed, got {cache.dtype} {tuple(cache.shape)}")
        _need(slots is not None, "a cache needs slots")
        _rows(slots, "slots", 1, (torch.int64,))
        _need(slots.shape[0] == T, f"{slots.shape[0]} slots for {T} tokens")
        cache_p, slots_p, n_slots = cache.data_ptr(), slots.data_ptr(), cache.numel() // (rank + rope)
    heads, qs, qo, qp, qop = 0, (0, 0), (0, 0), None, None
    if q_rope is not None:
        _rows(q_rope, "q_rope", 3, (_BF16,))
        _need(q_rope.shape[0] == T and q_rope.shape[2] == rope, f"q_rope {tuple(q_rope.shape)}, {(T, 'heads', rope)} is needed")
        heads = q_rope.shape[1]
        if q_out is None:
            q_out = torch.empty((T, heads, rope), dtype=_BF16, device=kv.device)
        else:
            _rows(q_out, "q_out", 3, (_BF16,))
            _need(q_out.shape == q_rope.shape, f"q_out {tuple(q_out.shape)}, q_rope {tuple(q_rope.shape)}")
        qs, qo, qp, qop = q_rope.stride(), q_out.stride(), q_rope.data_ptr(), q_out.data_ptr()
    q = scale = key = None
    if want_fp8:
        q, scale = _codes(T, rank, kv.device), _scales(T, rank, kv.device)
    if want_key:
        key = torch.empty((T, rope), dtype=_BF16, device=kv.device)
    B.check(B.lib().moe_latent_append(
        kv.data_ptr(), kv.stride(0) if T > 1 else rank + rope, weight.data_ptr(), _TYPES[weight.dtype], eps, rank, rope,
        table.data_ptr(), table.shape[0], positions.data_ptr(), slots_p, T, cache_p, n_slots, qp, heads, qs[0], qs[1],
        qop, qo[0], qo[1], q.data_ptr() if q is not None else None, q.stride(0) if q is not None else 0,
        scale.data_ptr() if scale is not None else None, 1, T, key.data_ptr() if key is not None else None, rope,
        B._stream_handle(stream)))
    return AppendOut(q_out if q_rope is not None else None, q, scale, key)


def latent_attention(q, cache, pages, lens, scale: float, max_len: int | None = None, cu_q=None,
                     max_q: int | None = None, tree=None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention over the paged latent cache, heads absorbed into the queries.

    q [T, heads, rank + rope] bf16; cache [pages, page_size, rank + rope];
    pages int32 [B, pages per sequence]; lens int32 [B] (rows of each
    sequence, its new tokens included).  New tokens: T / B per sequence, or
    with cu_q (int32 [B + 1]) rows cu_q[b] .. cu_q[b + 1] of q, at most max_q
    each.  max_len bounds lens (the page table's reach if None; a tighter
    bound makes short calls faster).  A token sees the context and the new
    tokens up to itself, or those set in its mask (tree, int64 [T], bit j for
    the sequence's j-th new token, itself included if set).  Returns
    [T, heads, rank] bf16.  workspace: uint8 of
    moe_latent_attention_workspace() bytes (allocated per call if None)."""
    _rows(q, "q", 3, (_BF16,))
    _rows(cache, "cache", 3, (_BF16,))
    _rows(pages, "pages", 2, (torch.int32,))
    _rows(lens, "lens", 1, (torch.int32,))
    T, heads, width = q.shape
    n_pages, page_size = cache.shape[0], cache.shape[1]
    nb, per_seq = pages.shape
    rope = 64
    rank = width - rope
    _need(cache.shape[2] == width and (page_size == 1 or cache.stride(1) == width),
          f"cache: rows of {width} one after another in a page are needed, got {tuple(cache.shape)} with strides {cache.stride()}")
    _need(lens.shape[0] == nb, f"{lens.shape[0]} lengths for {nb} page rows")
    if cu_q is not None:
        _rows(cu_q, "cu_q", 1, (torch.int32,))
        _need(cu_q.shape[0] == nb + 1, f"cu_q has {cu_q.shape[0]} entries for {nb} sequences")
        _need(max_q is not None, "cu_q needs max_q")
    else:
        max_q = T // nb if nb else 0
    if max_len is None:
        max_len = per_seq * page_size
    if tree is not None:
        _rows(tree, "tree", 1, (torch.int64,))
        _need(tree.shape[0] == T, f"tree has {tree.shape[0]} masks for {T} tokens")
    if out is None:
        out = torch.empty((T, heads, rank), dtype=_BF16, device=q.device)
    else:
        _rows(out, "out", 3, (_BF16,))
        _need(tuple(out.shape) == (T, heads, rank), f"out {tuple(out.shape)}, {(T, heads, rank)} is needed")
    L = B.lib()
    if workspace is None:
        workspace = torch.empty(L.moe_latent_attention_workspace(nb, max_q, heads, rank, max_len), dtype=torch.uint8,
                                device=q.device)
    B.check(L.moe_latent_attention(
        q.data_ptr(), q.stride(0), q.stride(1), T, heads, rank, rope, cache.data_ptr(), n_pages, page_size,
        cache.stride(0) if n_pages > 1 else page_size * width, pages.data_ptr(), pages.stride(0) if nb > 1 else per_seq,
        per_seq, lens.data_ptr(), nb, cu_q.data_ptr() if cu_q is not None else None, max_q, max_len,
        tree.data_ptr() if tree is not None else None, scale, out.data_ptr(), out.stride(0), out.stride(1),
        workspace.data_ptr(), workspace.numel(), B._stream_handle(stream)))
    return out


def prompt_attention(q, k, k_rope, v, scale: float, cu_q=None, cu_k=None, max_q: int | None = None,
                     max_k: int | None = None, causal: bool = True, out=None, stream=None) -> torch.Tensor:
    """Attention with keys and values expanded per head, for prompts.

    q [Tq, heads, nope + rope], k [Tk, heads, nope], k_rope [Tk, rope] shared
    by the heads, v [Tk, heads, vdim], all bf16 (k and v may be views of one
    expansion).  Sequence b has queries cu_q[b] .. cu_q[b + 1] and keys
    cu_k[b] .. cu_k[b + 1] (int32 [B + 1]; None: one sequence); its queries
    are its last positions.  max_q bounds the queries of a sequence; max_k is
    not needed.  Returns [Tq, heads, vdim] bf16."""
    _rows(q, "q", 3, (_BF16,))
    _rows(k, "k", 3, (_BF16,))
    _rows(k_rope, "k_rope", 2, (_BF16,))
    _rows(v, "v", 3, (_BF16,))
    Tq, heads, width = q.shape
    Tk, rope, vdim = k.shape[0], k_rope.shape[1], v.shape[2]
    _need(k.shape[1] == heads and v.shape[1] == heads and v.shape[0] == Tk and k_rope.shape[0] == Tk
          and k.shape[2] + rope == width,
          f"q {tuple(q.shape)}, k {tuple(k.shape)}, k_rope {tuple(k_rope.shape)}, v {tuple(v.shape)} do not go together")
    _need((cu_q is None) == (cu_k is None), "cu_q and cu_k go together")
    if cu_q is None:
        cu_q = torch.tensor([0, Tq], dtype=torch.int32, device=q.device)
        cu_k = torch.tensor([0, Tk], dtype=torch.int32, device=q.device)
        max_q = Tq
    _rows(cu_q, "cu_q", 1, (torch.int32,))
    _rows(cu_k, "cu_k", 1, (torch.int32,))
    _need(cu_q.shape == cu_k.shape and cu_q.shape[0] >= 1 and max_q is not None,
          "cu_q and cu_k: one more entry than sequences each, and max_q")
    if out is None:
        out = torch.empty((Tq, heads, vdim), dtype=_BF16, device=q.device)
    else:
        _rows(out, "out", 3, (_BF16,))
        _need(tuple(out.shape) == (Tq, heads, vdim), f"out {tuple(out.shape)}, {(Tq, heads, vdim)} is needed")
    B.check(B.lib().moe_prompt_attention(
        q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), k.stride(0), k.stride(1), k_rope.data_ptr(),
        k_rope.stride(0), v.data_ptr(), v.stride(0), v.stride(1), Tq, Tk, heads, k.shape[2], rope, vdim,
        cu_q.data_ptr(), cu_k.data_ptr(), cu_q.shape[0] - 1, max_q, int(bool(causal)), scale, out.data_ptr(),
        out.stride(0), out.stride(1), B._stream_handle(stream)))
    return out
