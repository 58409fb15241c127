"""The attention half of a decoder block: what stands between two routed
layers of a model with latent attention, as calls on torch tensors.

    add_rmsnorm       residual addition and root-mean-square norm, bf16 and / or 8-bit output
    quantize          8-bit codes and scales alone
    fp8_linear        8-bit product with a scale per 128 columns (activations) and 128 x 128 block (weights)
    head_linear       one product per head (queries into the latent space, outputs back out)
    latent_append     norm, rotation and write of new rows of the latent cache
    latent_attention  attention over the paged latent cache (single tokens, chunks, trees of drafted tokens)
    prompt_attention  the same attention with keys and values expanded per head, for prompts

Every step runs in the HIP kernels behind include/moe.h; this module checks
shapes and types, allocates outputs where none are given, and passes pointers
and strides.  Calls run on torch's current stream, or on `stream` as if under
torch.cuda.stream(stream) (outputs and workspaces belong to it, and it has to
be behind whatever makes the inputs), return at once, and can be captured in a
graph.  There is no CPU fallback.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding as B

_BF16, _F32, _FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_TYPES = {_BF16: 0, _F32: 1}  # MOE_BF16, MOE_F32
_WIDE, _BF16_ONLY, _FP8_ONLY, _F32_ONLY = (_BF16, _F32), (_BF16,), (_FP8,), (_F32,)
_I32_ONLY, _I64_ONLY = (torch.int32,), (torch.int64,)
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
    key: torch.Tensor | None     # rotated position part of the keys (a view of rows)
    rows: torch.Tensor | None    # the cache rows, one after another


_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(stream, f, *args):
    """f(*args) on `stream` (torch's, or a handle; None: the current one) of
    the first operand's device, as the current device (a launch goes to that
    one, whatever device its stream belongs to).  What f allocates belongs to
    that stream, and memory of the inputs is not used again before a stream of
    torch's has passed the call (a handle's owner sees to that)."""
    device = args[0].device
    _need(device.type == "cuda", f"a tensor on a GPU is needed, got one on {device}")
    if isinstance(stream, torch.cuda.Stream):
        _need(stream.device == device, f"a stream of {stream.device} and operands on {device}")
        with torch.cuda.stream(stream):
            out = f(*args)
        for t in args:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
        return out
    if stream is None:
        with torch.cuda.device(device):
            return f(*args)
    handle = B._stream_handle(stream)
    with torch.cuda.stream(torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)):
        return f(*args)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise B.MoeError(B.MOE_EINVAL, what)


def _rows(t: torch.Tensor, name: str, dims: int, dtypes, on: int):
    """Shape and strides of a tensor of `dims` dimensions with a contiguous
    last one on GPU `on`, that of the call's first operand."""
    shape, stride = t.shape, t.stride()
    if len(stride) == dims and t.dtype in dtypes and t.get_device() == on and (stride[-1] == 1 or shape[-1] <= 1):
        return shape, stride
    raise B.MoeError(B.MOE_EINVAL, f"{name}: a tensor of {dims} dimensions, contiguous in the last, of type "
                                   f"{' or '.join(str(d) for d in dtypes)} on cuda:{on} is needed, got {t.dtype} "
                                   f"{tuple(shape)} with strides {stride} on {t.device}")


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

    x [T, H] bf16 or fp32, weight [H] (None: no norm, the addition and the
    conversion alone), residual [T, H] or None.  out: "bf16",
    "fp8" (codes and one scale per 128 columns) or "both".  h is returned in
    the residual's type (sum_out, which may be the residual itself, receives
    it in place; want_sum=False leaves it out)."""
    on = x.get_device()
    if stream is not None or on < 0 or on != _device():
        return _elsewhere(stream, add_rmsnorm, x, weight, eps, residual, out, sum_out, want_sum)
    shape, strides = _rows(x, "x", 2, _WIDE, on)
    T, H = shape
    weight_p, w_type = None, 0
    if weight is not None:
        wide, _ = _rows(weight, "weight", 1, _WIDE, on)
        if wide[0] != H:
            _need(False, f"weight has {wide[0]} values, x {H} columns")
        weight_p, w_type = weight.data_ptr(), _TYPES[weight.dtype]
    x_type = _TYPES[x.dtype]
    residual_p, r_stride, r_type, sum_type = None, 0, 0, x.dtype
    if residual is not None:
        r_shape, r_strides = _rows(residual, "residual", 2, _WIDE, on)
        if r_shape != shape:
            _need(False, f"residual {tuple(r_shape)}, x {tuple(shape)}")
        residual_p, r_stride, sum_type = residual.data_ptr(), r_strides[0] if T > 1 else H, residual.dtype
        r_type = _TYPES[sum_type]
    sum_p, s_stride = None, H
    if sum_out is not None:
        s_shape, s_strides = _rows(sum_out, "sum_out", 2, (sum_type,), on)
        _need(s_shape == shape, f"sum_out {tuple(s_shape)}, x {tuple(shape)}")
        sum_p, s_stride = sum_out.data_ptr(), s_strides[0] if T > 1 else H
    elif want_sum and residual is not None:
        sum_out = torch.empty(shape, dtype=sum_type, device=on)
        sum_p = sum_out.data_ptr()
    y = q = scale = y_p = q_p = scale_p = None
    pad = -(-H // 16) * 16
    if out != "fp8":
        _need(out in ("bf16", "both"), f"out: {out!r}")
        y = torch.empty(shape, dtype=_BF16, device=on)
        y_p = y.data_ptr()
    if out != "bf16":
        q, scale = _codes(T, H, on), _scales(T, H, on)
        q_p, scale_p = q.data_ptr(), scale.data_ptr()
    B.check(B.lib().moe_add_rmsnorm(x.data_ptr(), x_type, strides[0] if T > 1 else H, residual_p, r_type, r_stride,
                                    weight_p, w_type, T, H, eps, sum_p, s_stride, y_p, H, q_p, pad,
                                    scale_p, 1, T, _raw_stream(on)))
    return NormOut(sum_out, y, q, scale)


def quantize(x, stream=None):
    """x [T, H] bf16 or fp32 in 8 bits: (codes, scales [T, ceil(H / 128)])."""
    r = add_rmsnorm(x, None, 0.0, out="fp8", stream=stream)
    return r.q, r.scale


def quantize_weight(w):
    """A weight [N, K] in 8 bits with one scale per 128 x 128 block, as
    fp8_linear reads it.  Done once when a model is loaded, in torch."""
    N, K = w.shape
    nb, kb = -(-N // GROUP), -(-K // GROUP)
    wide = torch.nn.functional.pad(w.float(), (0, kb * GROUP - K, 0, nb * GROUP - N))
    blocks = wide.view(nb, GROUP, kb, GROUP)
    scale = (blocks.abs().amax((1, 3)) / 448.0).clamp_min(1e-12)
    codes = (blocks / scale[:, None, :, None]).clamp(-448.0, 448.0).view(nb * GROUP, kb * GROUP)[:N, :K]
    return codes.to(_FP8).contiguous(), scale.contiguous()


def fp8_linear(a, a_scale, w, w_scale, out_dtype=_BF16, out=None, stream=None) -> torch.Tensor:
    """a [M, K] 8-bit with a_scale [M, ceil(K / 128)] times the transpose of
    w [N, K] 8-bit with w_scale [ceil(N / 128), ceil(K / 128)]: [M, N] in
    out_dtype (bf16 or fp32).  K is a multiple of 16; a_scale may have any
    strides (add_rmsnorm's are the fastest)."""
    on = a.get_device()
    if stream is not None or on < 0 or on != _device():
        return _elsewhere(stream, fp8_linear, a, a_scale, w, w_scale, out_dtype, out)
    (M, K), a_strides = _rows(a, "a", 2, _FP8_ONLY, on)
    (N, wk), w_strides = _rows(w, "w", 2, _FP8_ONLY, on)
    ws_shape, ws_strides = _rows(w_scale, "w_scale", 2, _F32_ONLY, on)
    kb, nb = (K + GROUP - 1) // GROUP, (N + GROUP - 1) // GROUP
    as_shape, as_strides = a_scale.shape, a_scale.stride()
    if (wk != K or a_scale.dtype is not _F32 or a_scale.get_device() != on or tuple(as_shape) != (M, kb)
            or tuple(ws_shape) != (nb, kb)):
        _need(False, f"a {(M, K)} and w {(N, wk)} need scales of fp32 {(M, kb)} and {(nb, kb)} on cuda:{on}, got "
                     f"{a_scale.dtype} {tuple(as_shape)} on {a_scale.device} and {tuple(ws_shape)}, and the same inner width")
    if out is None:
        _need(out_dtype in _TYPES, f"out_dtype {out_dtype}: bf16 or fp32")
        out, o_stride = torch.empty((M, N), dtype=out_dtype, device=on), N
    else:
        o_shape, o_strides = _rows(out, "out", 2, _WIDE, on)
        _need(tuple(o_shape) == (M, N), f"out {tuple(o_shape)}, {(M, N)} is needed")
        out_dtype, o_stride = out.dtype, o_strides[0] if M > 1 else N
    pad = -(-K // 16) * 16  # the stride of a single row says nothing
    B.check(B.lib().moe_fp8_linear(a.data_ptr(), a_strides[0] if M > 1 else pad, a_scale.data_ptr(), as_strides[0],
                                   as_strides[1], w.data_ptr(), w_strides[0] if N > 1 else pad, w_scale.data_ptr(),
                                   ws_strides[0] if nb > 1 else kb, M, N, K, out.data_ptr(), _TYPES[out_dtype], o_stride,
                                   _raw_stream(on)))
    return out


def head_linear(x, w, out=None, stream=None) -> torch.Tensor:
    """x [T, heads, K] times the transpose of w [heads, N, K], head by head:
    [T, heads, N], all bf16.  x and out may be strided views (of a wider
    query, say)."""
    on = x.get_device()
    if stream is not None or on < 0 or on != _device():
        return _elsewhere(stream, head_linear, x, w, out)
    (T, heads, K), xs = _rows(x, "x", 3, _BF16_ONLY, on)
    w_shape, _ = _rows(w, "w", 3, _BF16_ONLY, on)
    N = w_shape[1]
    if w_shape[0] != heads or w_shape[2] != K or not w.is_contiguous():
        _need(False, f"w: contiguous {(heads, 'N', K)} is needed, got {tuple(w_shape)} with strides {w.stride()}")
    if out is None:
        out, os = torch.empty((T, heads, N), dtype=_BF16, device=on), (heads * N, N)
    else:
        o_shape, os = _rows(out, "out", 3, _BF16_ONLY, on)
        _need(tuple(o_shape) == (T, heads, N), f"out {tuple(o_shape)}, {(T, heads, N)} is needed")
    B.check(B.lib().moe_head_linear(x.data_ptr(), xs[0], xs[1], w.data_ptr(), T, heads, K, N, out.data_ptr(), os[0], os[1],
                                    _raw_stream(on)))
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
    on = kv.get_device()
    if stream is not None or on < 0 or on != _device():
        return _elsewhere(stream, latent_append, kv, weight, eps, table, positions, slots, cache, q_rope, q_out,
                          want_fp8, want_key)
    (T, width), kvs = _rows(kv, "kv", 2, _BF16_ONLY, on)
    (rank,), _ = _rows(weight, "weight", 1, _WIDE, on)
    (n_positions, rope), _ = _rows(table, "table", 2, _F32_ONLY, on)
    (n,), _ = _rows(positions, "positions", 1, _I32_ONLY, on)
    if width != rank + rope or n != T or not table.is_contiguous():
        _need(False, f"kv has {width} columns, weight and table {rank} + {rope}; {n} positions for {T} tokens; table "
                     "contiguous")
    cache_p = slots_p = None
    n_slots = 0
    if cache is not None:
        if cache.dtype is not _BF16 or cache.get_device() != on or not cache.is_contiguous() or cache.shape[-1] != width:
            _need(False, f"cache: contiguous bf16 rows of {width} on cuda:{on} are needed, got {cache.dtype} "
                         f"{tuple(cache.shape)} on {cache.device}")
        _need(slots is not None, "a cache needs slots")
        (n,), _ = _rows(slots, "slots", 1, _I64_ONLY, on)
        _need(n == T, f"{n} slots for {T} tokens")
        cache_p, slots_p, n_slots = cache.data_ptr(), slots.data_ptr(), cache.numel() // width
    heads, qs, qo, qp, qop = 0, (0, 0), (0, 0), None, None
    if q_rope is not None:
        q_shape, qs = _rows(q_rope, "q_rope", 3, _BF16_ONLY, on)
        if q_shape[0] != T or q_shape[2] != rope:
            _need(False, f"q_rope {tuple(q_shape)}, {(T, 'heads', rope)} is needed")
        heads = q_shape[1]
        if q_out is None:
            q_out, qo = torch.empty(q_shape, dtype=_BF16, device=on), (heads * rope, rope)
        else:
            qo_shape, qo = _rows(q_out, "q_out", 3, _BF16_ONLY, on)
            _need(qo_shape == q_shape, f"q_out {tuple(qo_shape)}, q_rope {tuple(q_shape)}")
        qp, qop = q_rope.data_ptr(), q_out.data_ptr()
    q = scale = rows = q_p = scale_p = rows_p = None
    if want_fp8:
        q, scale = _codes(T, rank, on), _scales(T, rank, on)
        q_p, scale_p = q.data_ptr(), scale.data_ptr()
    if want_key:
        rows = torch.empty((T, width), dtype=_BF16, device=on)
        rows_p = rows.data_ptr()
    B.check(B.lib().moe_latent_append(
        kv.data_ptr(), kvs[0] if T > 1 else width, weight.data_ptr(), _TYPES[weight.dtype], eps, rank, rope,
        table.data_ptr(), n_positions, positions.data_ptr(), slots_p, T, cache_p, n_slots, qp, heads, qs[0], qs[1],
        qop, qo[0], qo[1], q_p, -(-rank // 16) * 16, scale_p, 1, T, rows_p, width, _raw_stream(on)))
    return AppendOut(q_out if q_rope is not None else None, q, scale, rows[:, rank:] if want_key else None, rows)


def latent_attention(q, cache, pages, lens, scale: float, max_len: int | None = None, cu_q=None,
                     max_q: int | None = None, tree=None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention over the paged latent cache, heads absorbed into the queries.

    q [T, heads, rank + rope] bf16; cache [pages, page_size, rank + rope];
    pages int32 [B, pages per sequence]; lens int32 [B] (rows of each
    sequence, its new tokens included).  New tokens: T / B per sequence, or
    with cu_q (int32 [B + 1], not decreasing) rows cu_q[b] .. cu_q[b + 1] of q,
    at most max_q each (rows of q in no sequence have no output: what out held
    there stays, and a new one holds anything).  max_len bounds lens (the page table's reach if None; a tighter
    bound makes short calls faster).  A token sees the context and the new
    tokens up to itself, or those set in its mask (tree, int64 [T], bit j for
    the sequence's j-th new token, itself included if set).  Returns
    [T, heads, rank] bf16.  workspace: uint8 of
    moe_latent_attention_workspace() bytes (allocated per call if None)."""
    on = q.get_device()
    if stream is not None or on < 0 or on != _device():
        return _elsewhere(stream, latent_attention, q, cache, pages, lens, scale, max_len, cu_q, max_q, tree, out,
                          workspace)
    (T, heads, width), qs = _rows(q, "q", 3, _BF16_ONLY, on)
    (n_pages, page_size, c_width), cs = _rows(cache, "cache", 3, _BF16_ONLY, on)
    (nb, per_seq), ps = _rows(pages, "pages", 2, _I32_ONLY, on)
    (n,), _ = _rows(lens, "lens", 1, _I32_ONLY, on)
    rope = 64
    rank = width - rope
    if c_width != width or (page_size > 1 and cs[1] != width) or n != nb:
        _need(False, f"cache: rows of {width} one after another in a page are needed, got {tuple(cache.shape)} with strides "
                     f"{cs}; {n} lengths for {nb} page rows")
    cu_p = tree_p = None
    if cu_q is not None:
        (n,), _ = _rows(cu_q, "cu_q", 1, _I32_ONLY, on)
        _need(n == nb + 1 and max_q is not None, f"cu_q has {n} entries for {nb} sequences; it needs max_q")
        cu_p = cu_q.data_ptr()
    else:
        max_q = T // nb if nb else 0
    if max_len is None:
        max_len = per_seq * page_size
    if tree is not None:
        (n,), _ = _rows(tree, "tree", 1, _I64_ONLY, on)
        _need(n == T, f"tree has {n} masks for {T} tokens")
        tree_p = tree.data_ptr()
    if out is None:
        out, os = torch.empty((T, heads, rank), dtype=_BF16, device=on), (heads * rank, rank)
    else:
        o_shape, os = _rows(out, "out", 3, _BF16_ONLY, on)
        _need(tuple(o_shape) == (T, heads, rank), f"out {tuple(o_shape)}, {(T, heads, rank)} is needed")
    L = B.lib()
    if workspace is None:
        n = L.moe_latent_attention_workspace(nb, max_q, heads, rank, max_len)
        workspace = torch.empty(n, dtype=torch.uint8, device=on)
    else:
        if workspace.get_device() != on or not workspace.is_contiguous():
            _need(False, f"workspace: contiguous memory of cuda:{on} is needed, got strides {workspace.stride()} on "
                         f"{workspace.device}")
        n = workspace.numel() * workspace.element_size()
    B.check(L.moe_latent_attention(
        q.data_ptr(), qs[0], qs[1], T, heads, rank, rope, cache.data_ptr(), n_pages, page_size,
        cs[0] if n_pages > 1 else page_size * width, pages.data_ptr(), ps[0] if nb > 1 else per_seq, per_seq,
        lens.data_ptr(), nb, cu_p, max_q, max_len, tree_p, scale, out.data_ptr(), os[0], os[1], workspace.data_ptr(), n,
        _raw_stream(on)))
    return out


def prompt_attention(q, k, k_rope, v, scale: float, cu_q=None, cu_k=None, max_q: int | None = None,
                     max_k: int | None = None, causal: bool = True, out=None, stream=None) -> torch.Tensor:
    """Attention with keys and values expanded per head, for prompts.

    q [Tq, heads, nope + rope], k [Tk, heads, nope], k_rope [Tk, rope] shared
    by the heads, v [Tk, heads, vdim], all bf16 (k and v may be views of one
    expansion).  Sequence b has queries cu_q[b] .. cu_q[b + 1] and keys
    cu_k[b] .. cu_k[b + 1] (int32 [B + 1]; None: one sequence); its queries
    are its last positions.  max_q bounds the queries of a sequence (rows past
    it or in no sequence have no output); max_k is not needed.  Returns [Tq, heads, vdim] bf16."""
    on = q.get_device()
    if stream is not None or on < 0 or on != _device():
        return _elsewhere(stream, prompt_attention, q, k, k_rope, v, scale, cu_q, cu_k, max_q, max_k, causal, out)
    (Tq, heads, width), qs = _rows(q, "q", 3, _BF16_ONLY, on)
    (Tk, k_heads, nope), ks = _rows(k, "k", 3, _BF16_ONLY, on)
    (r_rows, rope), rs = _rows(k_rope, "k_rope", 2, _BF16_ONLY, on)
    (v_rows, v_heads, vdim), vs = _rows(v, "v", 3, _BF16_ONLY, on)
    if k_heads != heads or v_heads != heads or v_rows != Tk or r_rows != Tk or nope + rope != width:
        _need(False, f"q {tuple(q.shape)}, k {tuple(k.shape)}, k_rope {tuple(k_rope.shape)}, v {tuple(v.shape)} do not go "
                     "together")
    _need((cu_q is None) == (cu_k is None), "cu_q and cu_k go together")
    if cu_q is None:
        ends = torch.arange(2, dtype=torch.int32, device=on)
        cu_q, cu_k = ends * Tq, ends * Tk
        max_q = Tq
    (n,), _ = _rows(cu_q, "cu_q", 1, _I32_ONLY, on)
    (n_k,), _ = _rows(cu_k, "cu_k", 1, _I32_ONLY, on)
    _need(n == n_k and n >= 1 and max_q is not None, "cu_q and cu_k: one more entry than sequences each, and max_q")
    if out is None:
        out, os = torch.empty((Tq, heads, vdim), dtype=_BF16, device=on), (heads * vdim, vdim)
    else:
        o_shape, os = _rows(out, "out", 3, _BF16_ONLY, on)
        _need(tuple(o_shape) == (Tq, heads, vdim), f"out {tuple(o_shape)}, {(Tq, heads, vdim)} is needed")
    B.check(B.lib().moe_prompt_attention(
        q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], k_rope.data_ptr(), rs[0], v.data_ptr(), vs[0], vs[1], Tq,
        Tk, heads, nope, rope, vdim, cu_q.data_ptr(), cu_k.data_ptr(), n - 1, max_q, int(causal), scale, out.data_ptr(),
        os[0], os[1], _raw_stream(on)))
    return out
