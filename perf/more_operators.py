"""Serving a decoder block at few bits and over shared contexts: cases that are measured.

Four operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and, with `own` true, as calls of this
repository's package:

  int4    product of bf16 activations with 4-bit weights (two's complement, an fp16 scale per group of input columns)
  store   new rows into a latent cache of 8 bits (codes, one power of two per row, position part in bf16), and the
          same rows read back
  latent  attention over that cache (single tokens, causal chunks, trees of drafted tokens)
  shared  attention of sequences that share a long prefix, over a cache of 16 or 8 bits

Sizes: hidden 6144, 64 heads and 512 + 64 values per token are this
repository's own; the head widths 128 + 64 (queries, keys) and 128 (values),
and a query rank of 2048, are generic.
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
        # one token through the key/value down-projection: latency only
        {"name": "int4 decode", "op": "int4", "M": 1, "N": RANK + ROPE, "K": HIDDEN, "group": 32},
        # one token through the output projection: 25 MB of weights
        {"name": "int4 decode wide", "op": "int4", "M": 1, "N": HIDDEN, "K": HEADS * VDIM, "group": 32},
        # a few sequences' drafted tokens through the query projection, odd
        {"name": "int4 verify", "op": "int4", "M": 29, "N": HEADS * (NOPE + ROPE), "K": 2048, "group": 64},
        # a prefill chunk through the output projection
        {"name": "int4 prefill", "op": "int4", "M": 2048, "N": HIDDEN, "K": HEADS * VDIM, "group": 32},
        # one decoded token into the cache and out of it
        {"name": "store decode", "op": "store", "T": 1, "heads": HEADS, "page": 64},
        # a prefill chunk
        {"name": "store prefill", "op": "store", "T": 8192, "heads": HEADS, "page": 64},
        # one sequence, one new token, a short odd context: latency
        {"name": "latent decode", "op": "latent", "B": 1, "nq": 1, "heads": HEADS, "len": 1013, "page": 64, "ragged": False, "tree": False},
        # 32 sequences of long contexts, one token each
        {"name": "latent batch", "op": "latent", "B": 32, "nq": 1, "heads": HEADS, "len": 16384, "page": 64, "ragged": False, "tree": False},
        # trees of drafted tokens over ragged contexts
        {"name": "latent verify", "op": "latent", "B": 11, "nq": 5, "heads": HEADS, "len": 9001, "page": 64, "ragged": True, "tree": True},
        # two sequences on a short common prompt: latency
        {"name": "shared short", "op": "shared", "bits": 16, "B": 2, "nq": 1, "heads": HEADS, "prefix": 517, "groups": 1, "len": 40, "page": 64, "ragged": True, "tree": False},
        # 32 sequences on one long document, one token each
        {"name": "shared batch", "op": "shared", "bits": 16, "B": 32, "nq": 1, "heads": HEADS, "prefix": 16384, "groups": 1, "len": 500, "page": 64, "ragged": True, "tree": False},
        # two system prompts, 8 sequences on each that verify drafted trees, 8 bits
        {"name": "shared verify", "op": "shared", "bits": 8, "B": 16, "nq": 4, "heads": HEADS, "prefix": 8192, "groups": 2, "len": 700, "page": 64, "ragged": True, "tree": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["int4", "int4", "store", "latent", "latent", "shared", "shared"])
    if op == "int4":
        group = rng.choice([32, 32, 64, 128])
        N, K = rng.choice([(2048, HIDDEN), (RANK + ROPE, HIDDEN), (HEADS * (NOPE + ROPE), 2048), (HIDDEN, HEADS * VDIM),
                           (_log(rng, 100, 8000), group * _log(rng, 2, 6000 // group))])
        most = 2048 * 6144 * 8192 // max(N * K, 6144 * 8192)
        return {"op": op, "M": rng.choice([_log(rng, 1, 16), _log(rng, 1, most)]), "N": N, "K": K, "group": group}
    if op == "store":
        return {"op": op, "T": _log(rng, 1, 8192), "heads": rng.choice([16, 64]), "page": rng.choice([16, 64, 100])}
    page, nq, heads = rng.choice([16, 64, 100]), rng.choice([1, 1, 2, 3, 7, 16]), rng.choice([16, 64, 128])
    tree = nq > 1 and rng.random() < 0.5
    if op == "latent":
        B = _log(rng, 1, 64)
        most = max(256, min(32768, 32 * 64 * 16384 // (B * nq * heads)))
        return {"op": op, "B": B, "nq": nq, "heads": heads, "len": _log(rng, max(nq, 100), most), "page": page,
                "ragged": rng.random() < 0.6, "tree": tree}
    groups = rng.choice([1, 1, 2])
    B = groups * _log(rng, 1, 48 // groups)
    most = max(256, min(32768, 32 * 64 * 16384 // (B * nq * heads)))
    return {"op": op, "bits": rng.choice([8, 16]), "B": B, "nq": nq, "heads": heads, "prefix": _log(rng, 100, most), "groups": groups,
            "len": _log(rng, nq, max(nq, min(1500, most))), "page": page, "ragged": rng.random() < 0.6, "tree": tree}


# -------------------------------------------------------------------- inputs
def _lengths(case):
    """Rows of each sequence's own, and of each prefix: the case's own, so that every pass of it is the same work."""
    g = torch.Generator()
    g.manual_seed(case["B"] * 1009 + case["nq"])
    u = torch.rand(case["B"], generator=g).tolist()
    # from a sixteenth of the longest up, the longest among them
    own_rows = [max(case["nq"], int(case["len"] * (1 / 16 + 15 / 16 * x))) if case["ragged"] else case["len"] for x in u]
    own_rows[0] = max(case["len"], case["nq"])
    prefix = [case["prefix"] - i * (case["prefix"] // 5) for i in range(case["groups"])] if case["op"] == "shared" else []
    return own_rows, prefix


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


def _page_table(rows, page, order, at):
    """Page lists of sequences with the given rows, from order[at] on; and where they end."""
    used = [-(-n // page) for n in rows]
    table = torch.full((len(rows), max(used)), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return table, at


def _rows_of_8_bits(rows):
    """bf16 rows as codes (with the position part's bytes behind them) and a power of two per row."""
    latent = rows[..., :RANK].float()
    scale = _power(latent.abs().amax(-1))
    codes = (latent / scale[..., None]).to(torch.float8_e4m3fn)
    return torch.cat([codes.view(torch.uint8), rows[..., RANK:].contiguous().view(torch.uint8)], -1), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    bf = torch.bfloat16

    def normal(*shape, std=1.0, dtype=bf):
        return torch.empty(*shape, device=DEV, dtype=torch.float32).normal_(0.0, std, generator=g).to(dtype)

    s = {"case": case, "op": case["op"]}
    if case["op"] == "int4":
        M, N, K, group = case["M"], case["N"], case["K"], case["group"]
        s["x"] = normal(M, K)
        w = normal(N, K, std=K ** -0.5, dtype=torch.float32).view(N, K // group, group)
        s["scale"] = (w.abs().amax(2) / 7).half()
        q = (w / s["scale"].float()[:, :, None]).round_().clamp_(-8, 7).view(N, K).to(torch.int32)
        s["codes"] = ((q[:, 0::2] & 15) | (q[:, 1::2] & 15) << 4).to(torch.uint8)
        return s
    page = case["page"]
    if case["op"] == "store":
        T = case["T"]
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
        s["cache"] = torch.zeros(pages, page, RANK + 2 * ROPE, dtype=torch.uint8, device=DEV)
        s["cache_scale"] = torch.ones(pages, page, device=DEV)
        s["q"] = normal(T, case["heads"], NOPE + ROPE)
        return s
    own_rows, prefix = _lengths(case)
    total = sum(-(-n // page) for n in own_rows + prefix) + 5
    order = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    s["pages"], at = _page_table(own_rows, page, order, 0)
    # the latents share a direction, as a norm's weighted outputs do
    cache = (normal(total, page, RANK + ROPE) + normal(RANK + ROPE, std=0.5)).contiguous()
    s["cache"], s["cache_scale"] = _rows_of_8_bits(cache) if case["op"] == "latent" or case["bits"] == 8 else (cache, None)
    s["lens"] = torch.tensor(own_rows, dtype=torch.int32, device=DEV)
    s["max_len"] = max(own_rows)
    if prefix:
        s["prefix_pages"], at = _page_table(prefix, page, order, at)
        s["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device=DEV)
        s["prefix_max_len"] = max(prefix)
        each = case["B"] // case["groups"]
        s["groups"] = torch.arange(case["groups"] + 1, dtype=torch.int32, device=DEV) * each
    s["q"] = normal(case["B"] * case["nq"], case["heads"], RANK + ROPE)
    host = torch.Generator()
    host.manual_seed(seed)
    s["tree"] = _trees(case["nq"], case["B"], host) if case["tree"] else None
    s["scale"] = (NOPE + ROPE) ** -0.5
    return s


# --------------------------------------------------------------- plain forms
def _power(top):
    """The least power of two that brings magnitudes up to `top` into the codes' range, from 2^-100 on."""
    mantissa, exponent = torch.frexp(top / FP8_MAX)
    return torch.ldexp(torch.ones_like(top), (exponent - (mantissa == 0.5).int()).clamp_min(-100))


def _int4_plain(x, codes, scale):
    N, K = codes.shape[0], 2 * codes.shape[1]
    nibbles = torch.stack([codes & 15, codes >> 4], 2).view(N, K).float()
    w = torch.where(nibbles > 7, nibbles - 16, nibbles).view(N, scale.shape[1], -1) * scale.float()[:, :, None]
    return (x.float() @ w.view(N, K).t()).to(torch.bfloat16)


def _rotated(x, cos, sin):
    even, odd = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack([even * cos - odd * sin, even * sin + odd * cos], -1).flatten(-2).to(torch.bfloat16)


def _values(cache, cache_scale):
    """Cache rows of either width as 32-bit values."""
    if cache_scale is None:
        return cache.float()
    latent = cache[..., :RANK].contiguous().view(torch.float8_e4m3fn).float() * cache_scale[..., None]
    return torch.cat([latent, cache[..., RANK:].contiguous().view(torch.bfloat16).float()], -1)


def _store_plain(s):
    kv, q, width = s["kv"], s["q"], RANK + 2 * ROPE
    c = kv[:, :RANK].float()
    c = c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS) * s["weight"].float()
    row = s["table"][s["positions"].long()]
    cos, sin = row[:, : ROPE // 2], row[:, ROPE // 2:]
    scale = _power(c.abs().amax(1))
    key = _rotated(kv[:, RANK:], cos, sin)
    codes = (c / scale[:, None]).to(torch.float8_e4m3fn)
    s["cache"].view(-1, width)[s["slots"]] = torch.cat([codes.view(torch.uint8), key.view(torch.uint8)], 1)
    s["cache_scale"].view(-1)[s["slots"]] = scale
    back = _values(s["cache"].view(-1, width)[s["slots"]], s["cache_scale"].view(-1)[s["slots"]])
    return {"rows": back.to(torch.bfloat16), "q": _rotated(q[..., NOPE:], cos[:, None], sin[:, None])}


def _gathered(s, pages, most):
    """The first `most` rows of each page list, as values."""
    page, width = s["cache"].shape[1:]
    at = torch.arange(most, device=DEV)
    rows = pages.long().clamp_min(0)[:, at // page] * page + at % page
    scale = s["cache_scale"]
    return _values(s["cache"].view(-1, width)[rows], None if scale is None else scale.view(-1)[rows])


def _scores(q, kv, scale):
    return torch.matmul(q, kv.transpose(1, 2).contiguous()) * scale


def _attention_plain(s):
    q, lens = s["q"], s["lens"].long()
    T, heads, width = q.shape
    B = lens.shape[0]
    nq = T // B
    kv = _gathered(s, s["pages"], s["max_len"])
    at = torch.arange(s["max_len"], device=DEV)
    draft = at[None, :] - (lens - nq)[:, None]  # the place among the new tokens, negative for the context
    if s["tree"] is None:
        visible = draft[:, None, :] <= torch.arange(nq, device=DEV)[None, :, None]
    else:
        bit = (s["tree"].view(B, nq, 1) >> draft.clamp(0, 63)[:, None, :]) & 1
        visible = (draft < 0)[:, None, :] | ((bit == 1) & (draft < nq)[:, None, :])
    hidden = ~visible.repeat_interleave(heads, 1)
    scores = _scores(q.view(B, nq * heads, width).float(), kv, s["scale"]).masked_fill(hidden, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    if s["op"] == "shared":
        G = s["prefix_lens"].shape[0]
        before = _gathered(s, s["prefix_pages"], s["prefix_max_len"])
        past = torch.arange(s["prefix_max_len"], device=DEV) >= s["prefix_lens"][:, None]
        first = _scores(q.view(G, -1, width).float(), before, s["scale"]).masked_fill(past[:, None], float("-inf"))
        top = torch.maximum(top, first.amax(-1).view(B, -1, 1))
    p = torch.exp(scores - top)
    total, out = p.sum(-1, keepdim=True), torch.matmul(p, kv[..., :RANK])
    if s["op"] == "shared":
        p = torch.exp(first - top.view(G, -1, 1))
        total = total + p.sum(-1).view(B, -1, 1)
        out = out + torch.matmul(p, before[..., :RANK]).view(B, -1, RANK)
    return (out / total).view(T, heads, RANK).to(torch.bfloat16)


def run(s):
    op = s["op"]
    if own:
        from routed_expert_int4_amd import attention as A
        if op == "int4":
            return A.int4_linear(s["x"], s["codes"], s["scale"])
        if op == "store":
            new = A.latent_append(s["kv"], s["weight"], EPS, s["table"], s["positions"], s["slots"], s["cache"],
                                  q_rope=s["q"][..., NOPE:], cache_scale=s["cache_scale"])
            return {"rows": A.latent_read(s["cache"], s["cache_scale"], s["slots"]), "q": new.q_rope}
        prefix = None
        if op == "shared":
            prefix = A.SharedPrefix(s["prefix_pages"], s["prefix_lens"], s["prefix_max_len"], s["groups"])
        return A.latent_attention(s["q"], s["cache"], s["pages"], s["lens"], s["scale"], max_len=s["max_len"], tree=s["tree"],
                                  cache_scale=s["cache_scale"], prefix=prefix)
    if op == "int4":
        return _int4_plain(s["x"], s["codes"], s["scale"])
    return _store_plain(s) if op == "store" else _attention_plain(s)


# ----------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "int4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K // 2 + 2 * N * K // case["group"] + 2 * M * N, "flops": 2 * M * N * K}
    narrow = RANK + 2 * ROPE + 4
    if op == "store":
        T, h = case["T"], case["heads"]
        return {"bytes": T * (4 * (RANK + ROPE) + 2 * narrow + 4 * ROPE + 20 + 4 * h * ROPE) + 2 * RANK, "flops": T * (8 * RANK + 3 * ROPE * (h + 1))}
    own_rows, prefix = _lengths(case)
    nq, h, B = case["nq"], case["heads"], case["B"]
    wide = narrow if op == "latent" or case["bits"] == 8 else 2 * (RANK + ROPE)
    pairs = nq * (sum(own_rows) + sum(n * (B // case["groups"]) for n in prefix))
    return {"bytes": wide * (sum(own_rows) + sum(prefix)) + 2 * B * nq * h * (2 * RANK + ROPE), "flops": 2 * pairs * h * (2 * RANK + ROPE)}


# ------------------------------------------------------------------ in 64 bits
def _row64(s, page_list, n):
    """The first n rows on a list of pages, taken page by page."""
    page = s["cache"].shape[1]
    parts = []
    for p in page_list[: -(-n // page)]:
        if s["cache_scale"] is None:
            parts.append(s["cache"][p].double())
            continue
        codes, key = s["cache"][p].split([RANK, 2 * ROPE], 1)
        latent = torch.einsum("rc,r->rc", codes.clone().view(torch.float8_e4m3fn).double(), s["cache_scale"][p].double())
        parts.append(torch.hstack([latent, key.clone().view(torch.bfloat16).double()]))
    return torch.vstack(parts)[:n]


def exact(case, seed):
    """From the definitions, in 64 bits, group by group and sequence by sequence."""
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "int4":
        out = torch.zeros(case["M"], case["N"], dtype=d, device=DEV)
        group = case["group"]
        for i in range(case["K"] // group):
            byte = s["codes"][:, i * group // 2:(i + 1) * group // 2].to(torch.int16)
            low, high = (byte % 16 + 8) % 16 - 8, (byte // 16 + 8) % 16 - 8
            x = s["x"][:, i * group:(i + 1) * group].to(d)
            part = x[:, 0::2] @ low.t().to(d) + x[:, 1::2] @ high.t().to(d)
            out += part * s["scale"][:, i].to(d)
        return out
    if case["op"] == "store":
        c = s["kv"][:, :RANK].to(d)
        c = c / ((c ** 2).sum(1, keepdim=True) / RANK + EPS).sqrt() * s["weight"].to(d)
        row = s["table"][s["positions"].long()].to(d)
        turn = torch.complex(row[:, : ROPE // 2], row[:, ROPE // 2:])
        key = torch.view_as_real(torch.view_as_complex(s["kv"][:, RANK:].to(d).view(case["T"], -1, 2)) * turn).flatten(1)
        q = torch.view_as_complex(s["q"][..., NOPE:].to(d).reshape(case["T"], case["heads"], -1, 2)) * turn[:, None]
        # what the cache holds is by definition rounded to codes: 4 bits of significand from 2^-6 on, steps of 2^-9 below
        scale = 2.0 ** (c.abs().max(1, keepdim=True).values / FP8_MAX).log2().ceil()
        c = c / scale
        step = 2.0 ** (c.abs().clamp_min(2.0 ** -6).log2().floor() - 3)
        return {"rows": torch.cat([torch.round(c / step) * step * scale, key], 1), "q": torch.view_as_real(q).flatten(2)}
    out = []
    n, B = case["nq"], case["B"]
    table, lens = s["pages"].tolist(), s["lens"].tolist()
    if case["op"] == "shared":
        before = [_row64(s, p, m) for p, m in zip(s["prefix_pages"].tolist(), s["prefix_lens"].tolist())]
    for b in range(B):
        kv = _row64(s, table[b], lens[b])
        for j in range(n):
            t = b * n + j
            keep = list(range(lens[b] - n))
            keep += [lens[b] - n + i for i in range(n) if (int(s["tree"][t]) >> i & 1 if case["tree"] else i <= j)]
            seen = kv[torch.tensor(keep, device=DEV)]
            if case["op"] == "shared":
                seen = torch.vstack([before[b * case["groups"] // B], seen])
            p = torch.softmax(s["q"][t].to(d) @ seen.t() * s["scale"], 1)
            out.append(p @ seen[:, :RANK])
    return torch.stack(out)
