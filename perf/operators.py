"""The attention half of a decoder block around the routed MoE layer: cases that are measured.

Five operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and, with `own` true, as calls of this
repository's package:

  norm    residual addition, root-mean-square norm, 8-bit output with a scale per 128 columns
  linear  product of 8-bit activations (a scale per 128 columns) with 8-bit weights (a scale per 128 x 128 block)
  heads   one product per head, between a head's own and the shared latent dimensions
  append  norm of the latent, rotation of the position part, write into the paged cache, rotation of the queries
  latent  attention over a paged cache of one latent vector per token, heads absorbed into the queries
          (single tokens, causal chunks, trees of drafted tokens)
  prompt  the same attention with keys and values expanded per head, causal, sequences packed one after another

(latent and prompt are the two forms of one operator.)  Sizes: hidden 6144,
64 heads and a cache row of 512 + 64 values are this repository's own; the
head widths 128 + 64 (queries, keys) and 128 (values), and a query rank of
2048, are generic.
"""
import math

import torch

own = False

HIDDEN, HEADS, RANK, ROPE, NOPE, VDIM = 6144, 64, 512, 64, 128, 128
EPS = 1e-6
FP8_MAX = 448.0
DEV = "cuda:0"


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token between the two halves of a block: latency only
        {"name": "norm decode", "op": "norm", "T": 1, "H": HIDDEN, "x": "f32", "out": "fp8"},
        # a large prefill chunk: the MoE output (fp32) joins the bf16 residual
        {"name": "norm prefill", "op": "norm", "T": 8192, "H": HIDDEN, "x": "f32", "out": "fp8"},
        # one token through the key/value down-projection (576 rows: not a multiple of 128)
        {"name": "linear decode", "op": "linear", "M": 1, "N": RANK + ROPE, "K": HIDDEN, "out": "bf16"},
        # a prefill chunk through the output projection
        {"name": "linear prefill", "op": "linear", "M": 4096, "N": HIDDEN, "K": HEADS * VDIM, "out": "bf16"},
        # one token's queries into the latent space
        {"name": "heads decode", "op": "heads", "T": 1, "heads": HEADS, "K": NOPE, "N": RANK},
        # attention outputs of a chunk back out of the latent space
        {"name": "heads chunk", "op": "heads", "T": 1024, "heads": HEADS, "K": RANK, "N": VDIM},
        # one decoded token enters the cache
        {"name": "append decode", "op": "append", "T": 1, "heads": HEADS, "page": 64},
        # a prefill chunk enters the cache
        {"name": "append prefill", "op": "append", "T": 8192, "heads": HEADS, "page": 64},
        # one sequence, one new token, a short odd context: latency
        {"name": "latent decode", "op": "latent", "B": 1, "nq": 1, "heads": HEADS, "len": 1013, "page": 64, "ragged": False, "tree": False},
        # a batch of 32 sequences that verify trees of 4 drafted tokens over ragged long contexts
        {"name": "latent verify", "op": "latent", "B": 32, "nq": 4, "heads": HEADS, "len": 16384, "page": 64, "ragged": True, "tree": True},
        # three short ragged prompts in one call
        {"name": "prompt short", "op": "prompt", "B": 3, "heads": HEADS, "nq": 257, "past": 0},
        # one long prompt
        {"name": "prompt long", "op": "prompt", "B": 1, "heads": HEADS, "nq": 8192, "past": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "heads", "append", "latent", "latent", "prompt"])
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 8192), "H": rng.choice([HIDDEN, 2048, RANK, 1000, 4104]),
                "x": rng.choice(["f32", "bf16"]), "out": rng.choice(["fp8", "bf16"])}
    if op == "linear":
        N, K = rng.choice([(2048, HIDDEN), (RANK + ROPE, HIDDEN), (HEADS * (NOPE + ROPE), 2048), (HEADS * (NOPE + VDIM), RANK),
                           (HIDDEN, HEADS * VDIM), (_log(rng, 100, 4000), 16 * _log(rng, 9, 400))])
        return {"op": op, "M": _log(rng, 1, 4096 * 6144 * 8192 // max(N * K, 6144 * 8192)), "N": N, "K": K, "out": "bf16"}
    if op == "heads":
        K, N = rng.choice([(NOPE, RANK), (RANK, VDIM)])
        return {"op": op, "T": _log(rng, 1, 1024), "heads": rng.choice([16, 64]), "K": K, "N": N}
    if op == "append":
        return {"op": op, "T": _log(rng, 1, 8192), "heads": rng.choice([16, 64]), "page": rng.choice([16, 64, 100])}
    if op == "latent":
        B, nq, heads = _log(rng, 1, 64), rng.choice([1, 1, 2, 3, 7, 16]), rng.choice([16, 64, 128])
        most = max(256, min(32768, 32 * 4 * 64 * 8192 // (B * nq * heads)))
        return {"op": op, "B": B, "nq": nq, "heads": heads, "len": _log(rng, max(nq, 100), most), "page": rng.choice([16, 64, 100]),
                "ragged": rng.random() < 0.6, "tree": nq > 1 and rng.random() < 0.5}
    B, heads = _log(rng, 1, 8), rng.choice([16, 64])
    nq = _log(rng, 1, 8192 // B)
    past = rng.choice([0, 0, _log(rng, 1, 2048)])
    return {"op": "prompt", "B": B, "heads": heads, "nq": nq, "past": min(past, 8192 - nq)}


# -------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g


def _lengths(case):
    """Query and key counts of each sequence of an attention case: the case's own, so that every pass of it is the same work."""
    g = torch.Generator()
    g.manual_seed(case["B"] * 1009 + case["nq"])
    B = case["B"]
    u = torch.rand(B, generator=g).tolist()
    if case["op"] == "latent":
        nq = [case["nq"]] * B
        # contexts from a sixteenth of the longest up, the longest among them
        nk = [max(case["nq"], int(case["len"] * (1 / 16 + 15 / 16 * x))) if case["ragged"] else case["len"] for x in u]
        nk[0] = max(case["len"], case["nq"])
    else:
        nq = [max(1, int(case["nq"] * (1 / 4 + 3 / 4 * x))) for x in u]
        nq[0] = case["nq"]
        nk = [n + case["past"] for n in nq]
    return nq, nk


def _trees(nq, count, g):
    """For each drafted token the bits of itself and its ancestors, in trees of nq tokens."""
    rows = []
    for _ in range(count):
        masks = []
        for j in range(nq):
            parent = int(torch.randint(-1, j, (1,), generator=g)) if j else -1
            masks.append((masks[parent] if parent >= 0 else 0) | 1 << j)
        rows += masks
    return torch.tensor(rows, dtype=torch.int64, device=DEV)


def _cumulative(counts):
    c = [0]
    for n in counts:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=DEV)


def _quantized(x, scale, rows, cols):
    """x in 8 bits with the given scales, one per rows x cols block."""
    full = scale.repeat_interleave(rows, 0)[: x.shape[0]].repeat_interleave(cols, 1)[:, : x.shape[1]]
    return (x / full).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def prepare(case, seed):
    g = _gen(seed)
    bf = torch.bfloat16

    def normal(*shape, std=1.0, dtype=bf):
        return torch.empty(*shape, device=DEV, dtype=torch.float32).normal_(0.0, std, generator=g).to(dtype)

    s = {"case": case, "op": case["op"]}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s["x"] = normal(T, H, std=0.5, dtype=torch.float32 if case["x"] == "f32" else bf)
        s["residual"] = normal(T, H, std=2.0)
        s["weight"] = normal(H, std=0.2).abs_().add_(0.5)
        s["out"] = case["out"]
    elif case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        kb, nb = -(-K // 128), -(-N // 128)
        # activations as the norm leaves them: each group of 128 scaled to its largest value; stored group by group
        x = normal(M, K, std=1.0, dtype=torch.float32)
        pad = torch.nn.functional.pad(x, (0, kb * 128 - K)).view(M, kb, 128)
        a_scale = (pad.abs().amax(2) / FP8_MAX).clamp_min_(1e-12)
        s["a"] = _quantized(x, a_scale, 1, 128)
        s["a_scale"] = a_scale.t().contiguous().t()
        w = normal(N, K, std=K ** -0.5, dtype=torch.float32)
        top = torch.nn.functional.pad(w, (0, kb * 128 - K, 0, nb * 128 - N)).view(nb, 128, kb, 128).abs().amax((1, 3))
        s["w_scale"] = (top / FP8_MAX).contiguous()
        s["w"] = _quantized(w, s["w_scale"], 128, 128)
    elif case["op"] == "heads":
        s["x"] = normal(case["T"], case["heads"], case["K"])
        s["w"] = normal(case["heads"], case["N"], case["K"], std=case["K"] ** -0.5)
    elif case["op"] == "append":
        T, page = case["T"], case["page"]
        pages = -(-T // page) + 3
        s["kv"] = normal(T, RANK + ROPE, std=1.5)
        s["weight"] = normal(RANK, std=0.2).abs_().add_(0.5)
        # cosines, then sines, of position * 10000^(-2 i / width), from 64 bits
        rate = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=DEV) / ROPE)
        angle = torch.arange(T + 1000, dtype=torch.float64, device=DEV)[:, None] * rate
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["positions"] = torch.arange(T, device=DEV, dtype=torch.int32) + 777
        order = torch.randperm(pages, device=DEV, generator=g)
        at = torch.arange(T, device=DEV)
        s["slots"] = order[at // page] * page + at % page
        s["cache"] = torch.zeros(pages, page, RANK + ROPE, dtype=bf, device=DEV)
        s["q"] = normal(T, case["heads"], NOPE + ROPE)
    elif case["op"] == "latent":
        B, page = case["B"], case["page"]
        nq, nk = _lengths(case)
        width = -(-max(nk) // page)
        used = [-(-n // page) for n in nk]
        order = torch.randperm(sum(used) + 5, device=DEV, generator=g).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(used):
            table[b, :n] = order[at:at + n]
            at += n
        s["pages"] = table
        # the latents share a direction, as a norm's weighted outputs do
        s["cache"] = (normal(sum(used) + 5, page, RANK + ROPE) + normal(RANK + ROPE, std=0.5)).contiguous()
        s["lens"] = torch.tensor(nk, dtype=torch.int32, device=DEV)
        s["max_len"] = max(nk)
        s["q"] = normal(sum(nq), case["heads"], RANK + ROPE)
        host = torch.Generator()
        host.manual_seed(seed)
        s["tree"] = _trees(case["nq"], B, host) if case["tree"] else None
        s["scale"] = (NOPE + ROPE) ** -0.5
    else:
        nq, nk = _lengths(case)
        heads = case["heads"]
        s["q"] = normal(sum(nq), heads, NOPE + ROPE)
        # keys and values as one product leaves them: head by head, the key part before the value
        both = normal(sum(nk), heads, NOPE + VDIM)
        s["k"], s["v"] = both[..., :NOPE], both[..., NOPE:]
        s["k_rope"] = normal(sum(nk), ROPE)
        s["cu_q"], s["cu_k"], s["max_q"], s["max_k"] = _cumulative(nq), _cumulative(nk), max(nq), max(nk)
        s["scale"] = (NOPE + ROPE) ** -0.5
    return s


# --------------------------------------------------------------- plain forms
def _norm_plain(x, residual, weight, out):
    total = x.float() + residual.float()
    y = total * torch.rsqrt((total * total).mean(1, keepdim=True) + EPS) * weight.float()
    if out == "bf16":
        return {"sum": total.to(residual.dtype), "y": y.to(torch.bfloat16)}
    T, H = y.shape
    kb = -(-H // 128)
    groups = torch.nn.functional.pad(y, (0, kb * 128 - H)).view(T, kb, 128)
    scale = (groups.abs().amax(2) / FP8_MAX).clamp_min(1e-12)
    q = (groups / scale[:, :, None]).clamp(-FP8_MAX, FP8_MAX).view(T, kb * 128)[:, :H].to(torch.float8_e4m3fn)
    return {"sum": total.to(residual.dtype), "q": q, "scale": scale}


def _linear_plain(a, a_scale, w, w_scale):
    N, K = w.shape
    x = a.float() * a_scale.repeat_interleave(128, 1)[:, :K]
    full = w_scale.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return (x @ (w.float() * full).t()).to(torch.bfloat16)


def _heads_plain(x, w):
    return torch.bmm(x.float().transpose(0, 1).contiguous(), w.float().transpose(1, 2).contiguous()).transpose(0, 1).to(torch.bfloat16)


def _rotated(x, cos, sin):
    even, odd = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack([even * cos - odd * sin, even * sin + odd * cos], -1).flatten(-2).to(torch.bfloat16)


def _append_plain(s):
    kv, q = s["kv"], s["q"]
    c = kv[:, :RANK].float()
    c = c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS) * s["weight"].float()
    row = s["table"][s["positions"].long()]
    cos, sin = row[:, : ROPE // 2], row[:, ROPE // 2:]
    rows = torch.cat([c.to(torch.bfloat16), _rotated(kv[:, RANK:], cos, sin)], 1)
    s["cache"].view(-1, RANK + ROPE)[s["slots"]] = rows
    return {"cache": s["cache"], "q": _rotated(q[..., NOPE:], cos[:, None], sin[:, None])}


def _softmax_product(scores, visible, values):
    """softmax over the visible scores times the values; rows that see nothing give zero."""
    scores = scores.masked_fill(~visible, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return torch.matmul(p / p.sum(-1, keepdim=True).clamp_min(1e-30), values)


def _latent_plain(s):
    q, lens, pages, cache = s["q"], s["lens"].long(), s["pages"].long(), s["cache"]
    page, B = cache.shape[1], lens.shape[0]
    T, heads, width = q.shape
    nq = T // B
    at = torch.arange(s["max_len"], device=q.device)
    rows = pages.clamp_min(0)[:, at // page] * page + at % page
    kv = cache.view(-1, width)[rows].float()
    scores = torch.matmul(q.view(B, nq * heads, width).float(), kv.transpose(1, 2).contiguous()).view(B, nq, heads, -1) * s["scale"]
    draft = at[None, :] - (lens - nq)[:, None]  # the place among the new tokens, negative for the context
    own_place = torch.arange(nq, device=q.device)
    if s["tree"] is None:
        visible = draft[:, None, :] <= own_place[None, :, None]
    else:
        bit = (s["tree"].view(B, nq, 1) >> draft.clamp(0, 63)[:, None, :]) & 1
        visible = (draft < 0)[:, None, :] | ((bit == 1) & (draft < nq)[:, None, :])
    out = _softmax_product(scores.view(B, nq * heads, -1), visible.repeat_interleave(heads, 1), kv[..., :RANK])
    return out.view(T, heads, RANK).to(torch.bfloat16)


def _prompt_plain(s):
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    iq, ik = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    rows_q = (cu_q[:-1, None] + iq).clamp_max(s["q"].shape[0] - 1)
    rows_k = (cu_k[:-1, None] + ik).clamp_max(s["k"].shape[0] - 1)
    heads = s["q"].shape[1]
    k = torch.cat([s["k"], s["k_rope"][:, None].expand(-1, heads, -1)], 2)
    q, k, v = (x[r].float().transpose(1, 2).contiguous() for x, r in ((s["q"], rows_q), (k, rows_k), (s["v"], rows_k)))
    visible = ik[None, None, :] <= iq[None, :, None] + (nk - nq)[:, None, None]
    out = _softmax_product(torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"], visible[:, None], v)
    return out.transpose(1, 2)[iq[None] < nq[:, None]].to(torch.bfloat16)


def run(s):
    op = s["op"]
    if own:
        from routed_expert_int4_amd import attention as A
        if op == "norm":
            r = A.add_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], out=s["out"])
            return {"sum": r.sum, "y": r.y} if s["out"] == "bf16" else {"sum": r.sum, "q": r.q, "scale": r.scale}
        if op == "linear":
            return A.fp8_linear(s["a"], s["a_scale"], s["w"], s["w_scale"])
        if op == "heads":
            return A.head_linear(s["x"], s["w"])
        if op == "append":
            q = A.latent_append(s["kv"], s["weight"], EPS, s["table"], s["positions"], s["slots"], s["cache"], q_rope=s["q"][..., NOPE:])
            return {"cache": s["cache"], "q": q.q_rope}
        if op == "latent":
            return A.latent_attention(s["q"], s["cache"], s["pages"], s["lens"], s["scale"], max_len=s["max_len"], tree=s["tree"])
        return A.prompt_attention(s["q"], s["k"], s["k_rope"], s["v"], s["scale"], cu_q=s["cu_q"], cu_k=s["cu_k"], max_q=s["max_q"], max_k=s["max_k"])
    if op == "norm":
        return _norm_plain(s["x"], s["residual"], s["weight"], s["out"])
    if op == "linear":
        return _linear_plain(s["a"], s["a_scale"], s["w"], s["w_scale"])
    if op == "heads":
        return _heads_plain(s["x"], s["w"])
    if op == "append":
        return _append_plain(s)
    return _latent_plain(s) if op == "latent" else _prompt_plain(s)


# ----------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        read = T * H * ((4 if case["x"] == "f32" else 2) + 2) + 2 * H
        wrote = T * H * 2 + (T * H * 2 if case["out"] == "bf16" else T * H + 4 * T * -(-H // 128))
        return {"bytes": read + wrote, "flops": 6 * T * H}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // 128)
        return {"bytes": M * K + 4 * M * kb + N * K + 4 * kb * -(-N // 128) + 2 * M * N, "flops": 2 * M * N * K}
    if op == "heads":
        T, h, K, N = case["T"], case["heads"], case["K"], case["N"]
        return {"bytes": 2 * h * (T * K + N * K + T * N), "flops": 2 * T * h * N * K}
    if op == "append":
        T, h = case["T"], case["heads"]
        return {"bytes": T * (4 * (RANK + ROPE) + 4 * ROPE + 12 + 4 * h * ROPE) + 2 * RANK, "flops": T * (6 * RANK + 3 * ROPE * (h + 1))}
    nq, nk = _lengths(case)
    h = case["heads"]
    if op == "latent":
        pairs = sum(q * k for q, k in zip(nq, nk))
        return {"bytes": 2 * sum(nk) * (RANK + ROPE) + 2 * sum(nq) * h * (2 * RANK + ROPE), "flops": 2 * pairs * h * (2 * RANK + ROPE)}
    pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(nq, nk))
    return {"bytes": 2 * sum(nq) * h * (NOPE + ROPE + VDIM) + 2 * sum(nk) * (h * (NOPE + VDIM) + ROPE), "flops": 2 * pairs * h * (NOPE + ROPE + VDIM)}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """From the definitions, in 64 bits, sequence by sequence and head by head."""
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "norm":
        h = s["x"].to(d) + s["residual"].to(d)
        y = h / ((h ** 2).sum(1, keepdim=True) / case["H"] + EPS).sqrt() * s["weight"].to(d)
        if case["out"] == "bf16":
            return {"sum": h, "y": y}
        scale = torch.stack([part.abs().max(1).values for part in y.split(128, 1)], 1) / FP8_MAX
        # the values that the 8-bit outputs stand for, before their rounding
        q = torch.cat([part / scale[:, i:i + 1] for i, part in enumerate(y.split(128, 1))], 1)
        return {"sum": h, "q": q, "scale": scale}
    if case["op"] == "linear":
        out = torch.zeros(case["M"], case["N"], dtype=d, device=DEV)
        for i, (a, w) in enumerate(zip(s["a"].to(d).split(128, 1), s["w"].to(d).split(128, 1))):
            rows = s["w_scale"][:, i].to(d)[torch.arange(case["N"], device=DEV) // 128]
            out += (a @ w.t()) * s["a_scale"][:, i:i + 1].to(d) * rows
        return out
    if case["op"] == "heads":
        return torch.stack([s["x"][:, h].to(d) @ s["w"][h].to(d).t() for h in range(case["heads"])], 1)
    if case["op"] == "append":
        c = s["kv"][:, :RANK].to(d)
        c = c / ((c ** 2).sum(1, keepdim=True) / RANK + EPS).sqrt() * s["weight"].to(d)
        row = s["table"][s["positions"].long()].to(d)
        turn = torch.complex(row[:, : ROPE // 2], row[:, ROPE // 2:])
        key = torch.view_as_real(torch.view_as_complex(s["kv"][:, RANK:].to(d).view(case["T"], -1, 2)) * turn).flatten(1)
        q = torch.view_as_complex(s["q"][..., NOPE:].to(d).reshape(case["T"], case["heads"], -1, 2)) * turn[:, None]
        cache = torch.zeros(s["cache"].shape, dtype=d, device=DEV)
        cache.view(-1, RANK + ROPE)[s["slots"]] = torch.cat([c, key], 1)
        return {"cache": cache, "q": torch.view_as_real(q).flatten(2)}
    if work(case)["flops"] > 4e12:
        return None
    out = []
    if case["op"] == "latent":
        page, n = case["page"], case["nq"]
        for b, length in enumerate(s["lens"].tolist()):
            kv = torch.cat([s["cache"][p] for p in s["pages"][b, : -(-length // page)].tolist()])[:length].to(d)
            for j in range(n):
                t = b * n + j
                keep = torch.ones(length, dtype=torch.bool, device=DEV)
                for i in range(n):
                    keep[length - n + i] = bool(int(s["tree"][t]) >> i & 1) if case["tree"] else i <= j
                p = torch.softmax(((s["q"][t].to(d) @ kv.t()) * s["scale"])[:, keep], 1)
                out.append(p @ kv[keep, :RANK])
        return torch.stack(out)
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for q0, q1, k0, k1 in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        hidden = torch.ones(q1 - q0, k1 - k0, dtype=torch.bool, device=DEV).triu(1 + (k1 - k0) - (q1 - q0))
        rope = s["k_rope"][k0:k1].to(d)
        per_head = []
        for h in range(case["heads"]):
            q = s["q"][q0:q1, h].to(d)
            scores = (q[:, :NOPE] @ s["k"][k0:k1, h].to(d).t() + q[:, NOPE:] @ rope.t()) * s["scale"]
            per_head.append(torch.softmax(scores.masked_fill_(hidden, float("-inf")), 1) @ s["v"][k0:k1, h].to(d))
        out.append(torch.stack(per_head, 1))
    return torch.cat(out)
