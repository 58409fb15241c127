"""The attention half of a decoder block: what stands between two routed
layers of a model with latent attention, as calls on torch tensors.

    add_rmsnorm       residual addition and root-mean-square norm, bf16 and / or 8-bit output
    quantize          8-bit codes and scales alone
    fp8_linear        8-bit product with a scale per 128 columns (activations) and 128 x 128 block (weights)
    int4_linear       product with 4-bit weights and a scale per group of 32, 64 or 128 columns
    head_linear       one product per head (queries into the latent space, outputs back out)
    latent_append     norm, rotation and write of new rows of the latent cache (bf16, or 8 bits)
    latent_read       rows of an 8-bit latent cache as bf16
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
_U8_ONLY, _F16_ONLY = (torch.uint8,), (torch.float16,)
_I32_ONLY, _I64_ONLY = (torch.int32,), (torch.int64,)
GROUP = 128                   # columns (and weight rows) that share a scale
_GROUPS = (32, 64, 128)       # columns that share a scale of 4-bit weights


class NormOut(NamedTuple):
    """Outputs of add_rmsnorm; None where not asked for."""
    sum: torch.Tensor | None    # x + residual, in the residual's type
    y: torch.Tensor | None      # bf16
    q: torch.Tensor | None      # 8-bit
    scale: torch.Tensor | None  # fp32 [T, ceil(H / 128)]


class SharedPrefix(NamedTuple):
    """Rows that several sequences have before their own, for latent_attention."""
    pages: torch.Tensor           # int32 [prefixes, pages per prefix], of the sequences' pool
    lens: torch.Tensor            # int32 [prefixes], their rows
    max_len: int | None = None    # bounds lens (the pages' reach if None)
    groups: torch.Tensor | None = None  # int32 [prefixes + 1]: i belongs to sequences groups[i] .. groups[i + 1] (None: one for all)


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
        for t in (u for arg in args for u in (arg if isinstance(arg, tuple) else (arg,))):
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


def quantize_weight_int4(w, group: int = 32):
    """A weight [N, K] in 4 bits with one fp16 scale per `group` (32, 64 or
    128) columns of a row, as int4_linear reads it: (codes uint8 [N, K / 2],
    scales [N, K / group]), both contiguous.  The largest magnitude of a group
    gets code 7 or -7 where a seventh of it is a normal fp16 number; below, the
    scale is a multiple of 2^-24, and weights over 7 x 65504 are cut.  Done once
    when a model is loaded, in torch."""
    N, K = w.shape
    _need(group in _GROUPS and K % group == 0, f"groups of {group} columns (32, 64 or 128) in rows of {K}")
    blocks = w.float().view(N, K // group, group)
    scale = (blocks.abs().amax(2) / 7).clamp_(2.0 ** -24, 65504.0).half().contiguous()  # finite, and not zero
    q = (blocks / scale.float()[:, :, None]).round_().clamp_(-8, 7).view(N, K).to(torch.int32)
    return ((q[:, 0::2] & 15) | (q[:, 1::2] & 15) << 4).to(torch.uint8).contiguous(), scale


def int4_linear(x, codes, scale, out_dtype=_BF16, out=None, stream=None) -> torch.Tensor:
    """x [M, K] bf16 times the transpose of a 4-bit weight: codes uint8
    [N, K / 2] (two's complement nibbles, the even column in the low one) with
    scale fp16 [N, K / group], group 32, 64 or 128: [M, N] in out_dtype (bf16
    or fp32).  Rows of x and codes start on 16 bytes."""
    on = x.get_device()
    if stream is not None or on < 0 or on != _device():
        return _elsewhere(stream, int4_linear, x, codes, scale, out_dtype, out)
    (M, K), x_strides = _rows(x, "x", 2, _BF16_ONLY, on)
    (N, half), w_strides = _rows(codes, "codes", 2, _U8_ONLY, on)
    (rows, groups), s_strides = _rows(scale, "scale", 2, _F16_ONLY, on)
    group = K // groups if groups else 0
    if half * 2 != K or rows != N or group not in _GROUPS or group * groups != K:
        _need(False, f"x {(M, K)} needs codes (N, {K // 2}) and scales (N, {K} / 32, 64 or 128), got {(N, half)} and "
                     f"{(rows, groups)}")
    if out is None:
        if out_dtype not in _TYPES:
            _need(False, f"out_dtype {out_dtype}: bf16 or fp32")
        out, o_stride = torch.empty_strided((M, N), (N, 1), dtype=out_dtype, device=on), N  # (0.4 us quicker than empty)
    else:
        o_shape, o_strides = _rows(out, "out", 2, _WIDE, on)
        if tuple(o_shape) != (M, N):
            _need(False, f"out {tuple(o_shape)}, {(M, N)} is needed")
        out_dtype, o_stride = out.dtype, o_strides[0] if M > 1 else N
    # the stride of a single row says nothing
    B.check(B.lib().moe_int4_linear(x.data_ptr(), x_strides[0] if M > 1 else K, codes.data_ptr(),
                                    w_strides[0] if N > 1 else -(-half // 16) * 16, scale.data_ptr(),
                                    s_strides[0] if N > 1 else groups, group, M, N, K, out.data_ptr(), _TYPES[out_dtype],
                                    o_stride, _raw_stream(on)))
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
                  want_fp8: bool = False, want_key: bool = False, stream=None, cache_scale=None) -> AppendOut:
    """Norms the latents and rotates the position parts of new tokens and
    writes them to their rows of the cache.

    kv [T, rank + rope] bf16, weight [rank], table fp32 [positions, rope]
    (cosines, then sines), positions int32 [T], slots int64 [T] (row of the
    cache, page * page_size + place; negative: not written), cache [pages,
    page_size, rank + rope] contiguous.  q_rope [T, heads, rope] is rotated
    into q_out (given, the view itself for in place, or new).  want_fp8: the
    normed latent in 8 bits too; want_key: the rotated key part too.

    With cache_scale (fp32, contiguous, one value per row of the cache) the
    cache holds 8 bits: uint8 [pages, page_size, rank + 2 rope], a row being
    rank E4M3 codes and the rotated part's bf16 bytes, and cache_scale
    receives the row's power of two (want_fp8 is not for this cache; want_key's
    rows are those before their rounding to codes)."""
    on = kv.get_device()
    if stream is not None or on < 0 or on != _device():
        return _elsewhere(stream, latent_append, kv, weight, eps, table, positions, slots, cache, q_rope, q_out,
                          want_fp8, want_key, None, cache_scale)
    (T, width), kvs = _rows(kv, "kv", 2, _BF16_ONLY, on)
    (rank,), _ = _rows(weight, "weight", 1, _WIDE, on)
    (n_positions, rope), _ = _rows(table, "table", 2, _F32_ONLY, on)
    (n,), _ = _rows(positions, "positions", 1, _I32_ONLY, on)
    if width != rank + rope or n != T or not table.is_contiguous():
        _need(False, f"kv has {width} columns, weight and table {rank} + {rope}; {n} positions for {T} tokens; table "
                     "contiguous")
    cache_p = slots_p = None
    n_slots = 0
    if cache_scale is not None:
        _need(cache is not None and slots is not None and not want_fp8, "cache_scale goes with a cache of 8 bits and slots, "
              "and without want_fp8")
        n_slots = _narrow_rows(cache, cache_scale, width + rope, on)
    elif cache is not None:
        if cache.dtype is not _BF16 or cache.get_device() != on or not cache.is_contiguous() or cache.shape[-1] != width:
            _need(False, f"cache: contiguous bf16 rows of {width} on cuda:{on} are needed, got {cache.dtype} "
                         f"{tuple(cache.shape)} on {cache.device}")
        _need(slots is not None, "a cache needs slots")
        n_slots = cache.numel() // width
    if cache is not None:
        (n,), _ = _rows(slots, "slots", 1, _I64_ONLY, on)
        if n != T:
            _need(False, f"{n} slots for {T} tokens")
        cache_p, slots_p = cache.data_ptr(), slots.data_ptr()
    heads, qs, qo, qp, qop = 0, (0, 0), (0, 0), None, None
    if q_rope is not None:
        q_shape, qs = _rows(q_rope, "q_rope", 3, _BF16_ONLY, on)
        if q_shape[0] != T or q_shape[2] != rope:
            _need(False, f"q_rope {tuple(q_shape)}, {(T, 'heads', rope)} is needed")
        heads = q_shape[1]
        if q_out is None:
            qo = (heads * rope, rope)
            q_out = torch.empty_strided(q_shape, (*qo, 1), dtype=_BF16, device=on)
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
    if cache_scale is not None:
        B.check(B.lib().moe_latent_append_fp8(
            kv.data_ptr(), kvs[0] if T > 1 else width, weight.data_ptr(), _TYPES[weight.dtype], eps, rank, rope,
            table.data_ptr(), n_positions, positions.data_ptr(), slots_p, T, cache_p, cache_scale.data_ptr(), n_slots, qp,
            heads, qs[0], qs[1], qop, qo[0], qo[1], rows_p, width, _raw_stream(on)))
        return AppendOut(q_out if q_rope is not None else None, None, None, rows[:, rank:] if want_key else None, rows)
    B.check(B.lib().moe_latent_append(
        kv.data_ptr(), kvs[0] if T > 1 else width, weight.data_ptr(), _TYPES[weight.dtype], eps, rank, rope,
        table.data_ptr(), n_positions, positions.data_ptr(), slots_p, T, cache_p, n_slots, qp, heads, qs[0], qs[1],
        qop, qo[0], qo[1], q_p, -(-rank // 16) * 16, scale_p, 1, T, rows_p, width, _raw_stream(on)))
    return AppendOut(q_out if q_rope is not None else None, q, scale, rows[:, rank:] if want_key else None, rows)


def _narrow_rows(cache, cache_scale, row: int, on: int) -> int:
    """Rows of a cache of 8 bits with `row` bytes each and its scales."""
    if (cache.dtype is not torch.uint8 or cache.get_device() != on or not cache.is_contiguous() or cache.shape[-1] != row
            or cache_scale.dtype is not _F32 or cache_scale.get_device() != on or not cache_scale.is_contiguous()
            or cache_scale.numel() * row != cache.numel()):
        _need(False, f"a cache of 8 bits: contiguous uint8 rows of {row} and an fp32 scale for each, on cuda:{on}, are "
                     f"needed, got {cache.dtype} {tuple(cache.shape)} on {cache.device} and {cache_scale.dtype} "
                     f"{tuple(cache_scale.shape)} on {cache_scale.device}")
    return cache_scale.numel()


def latent_read(cache, cache_scale, slots, rope: int = 64, out=None, stream=None) -> torch.Tensor:
    """Rows slots (int64 [T]) of a cache of 8 bits (uint8 [pages, page_size,
    rank + 2 rope] with cache_scale) as bf16 [T, rank + rope], which holds
    their values exactly; a slot outside the cache reads as zeros.  Scales are
    read as powers of two, by their exponents alone, here and in attention."""
    on = cache.get_device()
    if stream is not None or on < 0 or on != _device():
        return _elsewhere(stream, latent_read, cache, cache_scale, slots, rope, out)
    n_slots = _narrow_rows(cache, cache_scale, cache.shape[-1], on)
    (T,), _ = _rows(slots, "slots", 1, _I64_ONLY, on)
    width = cache.shape[-1] - rope
    if not width > rope > 0:
        _need(False, f"rows of {cache.shape[-1]} bytes do not hold {rope} position values and codes")
    if out is None:
        out, o_stride = torch.empty_strided((T, width), (width, 1), dtype=_BF16, device=on), width
    else:
        o_shape, o_strides = _rows(out, "out", 2, _BF16_ONLY, on)
        if tuple(o_shape) != (T, width):
            _need(False, f"out {tuple(o_shape)}, {(T, width)} is needed")
        o_stride = o_strides[0] if T > 1 else width
    B.check(B.lib().moe_latent_read_fp8(cache.data_ptr(), cache_scale.data_ptr(), n_slots, width - rope, rope, slots.data_ptr(),
                                        T, out.data_ptr(), o_stride, _raw_stream(on)))
    return out


def latent_attention(q, cache, pages, lens, scale: float, max_len: int | None = None, cu_q=None,
                     max_q: int | None = None, tree=None, out=None, workspace=None, stream=None, cache_scale=None,
                     prefix: SharedPrefix | None = None) -> torch.Tensor:
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
    moe_latent_attention_workspace() bytes (allocated per call if None).

    cache_scale (fp32 [pages, page_size], contiguous): the cache holds 8 bits,
    as latent_append leaves it (a scale that is no power of two counts as the
    one with its exponent).  prefix: rows that sequences share, seen by
    their tokens before all of these (pages, lens, max_len and trees are of
    each sequence's own rows then); they are read once for all tokens on them
    (workspace: moe_latent_attention_shared_workspace() bytes, which grow with
    the tokens: 8 heads (rank + 2) each)."""
    on = q.get_device()
    if stream is not None or on < 0 or on != _device():
        return _elsewhere(stream, latent_attention, q, cache, pages, lens, scale, max_len, cu_q, max_q, tree, out,
                          workspace, None, cache_scale, prefix)
    (T, heads, width), qs = _rows(q, "q", 3, _BF16_ONLY, on)
    narrow = cache_scale is not None
    (n_pages, page_size, c_width), cs = _rows(cache, "cache", 3, _U8_ONLY if narrow else _BF16_ONLY, on)
    (nb, per_seq), ps = _rows(pages, "pages", 2, _I32_ONLY, on)
    (n,), _ = _rows(lens, "lens", 1, _I32_ONLY, on)
    rope = 64
    rank = width - rope
    row = width + rope if narrow else width
    if c_width != row or (page_size > 1 and cs[1] != row) or n != nb:
        _need(False, f"cache: rows of {row} one after another in a page are needed, got {tuple(cache.shape)} with strides "
                     f"{cs}; {n} lengths for {nb} page rows")
    if narrow:
        s_shape, _ = _rows(cache_scale, "cache_scale", 2, _F32_ONLY, on)
        if tuple(s_shape) != (n_pages, page_size) or not cache_scale.is_contiguous():
            _need(False, f"cache_scale: contiguous {(n_pages, page_size)} is needed, got {tuple(s_shape)} with strides "
                         f"{cache_scale.stride()}")
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
    prefixes = most = per_prefix = p_stride = 0
    p_pages = p_lens = p_groups = None
    if prefix is not None:
        (prefixes, per_prefix), pps = _rows(prefix.pages, "prefix.pages", 2, _I32_ONLY, on)
        (n,), _ = _rows(prefix.lens, "prefix.lens", 1, _I32_ONLY, on)
        _need(n == prefixes > 0, f"prefix: {n} lengths for {prefixes} page rows")
        if prefix.groups is not None:
            (n,), _ = _rows(prefix.groups, "prefix.groups", 1, _I32_ONLY, on)
            _need(n == prefixes + 1, f"prefix.groups has {n} entries for {prefixes} prefixes")
            p_groups = prefix.groups.data_ptr()
        _need(prefixes == 1 or p_groups, f"{prefixes} prefixes need groups")
        p_stride = pps[0] if prefixes > 1 else per_prefix
        p_pages, p_lens = prefix.pages.data_ptr(), prefix.lens.data_ptr()
        most = per_prefix * page_size if prefix.max_len is None else prefix.max_len
    L = B.lib()
    if workspace is None:
        n = L.moe_latent_attention_shared_workspace(nb, T, max_q, heads, rank, max_len, prefixes, most)
        workspace = torch.empty(n, dtype=torch.uint8, device=on)
    else:
        if workspace.get_device() != on or not workspace.is_contiguous():
            _need(False, f"workspace: contiguous memory of cuda:{on} is needed, got strides {workspace.stride()} on "
                         f"{workspace.device}")
        n = workspace.numel() * workspace.element_size()
    if narrow or prefixes:
        B.check(L.moe_latent_attention_shared(
            q.data_ptr(), qs[0], qs[1], T, heads, rank, rope, cache.data_ptr(), cache_scale.data_ptr() if narrow else None,
            n_pages, page_size, cs[0] if n_pages > 1 else page_size * row, pages.data_ptr(), ps[0] if nb > 1 else per_seq,
            per_seq, lens.data_ptr(), nb, cu_p, max_q, max_len, tree_p, p_pages, p_stride, per_prefix, p_lens, p_groups,
            prefixes, most, scale, out.data_ptr(), os[0], os[1], workspace.data_ptr(), n, _raw_stream(on)))
        return out
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
