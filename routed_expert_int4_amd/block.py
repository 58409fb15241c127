"""One decoder block: latent attention and the routed MoE layer.

    python -m routed_expert_int4_amd.block            # a prompt, then decoded tokens, timed

Per token (colibri summary, "Principales fonctionnalites": q/kv-LoRA, partial
interleaved rotary positions, one latent vector per token in the cache):

    h      = residual + delta;  x = norm(h)                          add_rmsnorm, 8-bit out
    q      = W_qb norm(W_qa x);  c | k_r = W_kva x                   fp8_linear, add_rmsnorm
    cache <- norm(c) | rotate(k_r);  q_r = rotate(q_r)               latent_append
    prompt:  k = W_uk c, v = W_uv c per head, attention over them    head_linear, prompt_attention
    decode:  q_c = q W_uk per head, attention over the cache,        head_linear, latent_attention,
             o = W_uv o_c per head                                   head_linear
    delta  = W_o o                                                   quantize, fp8_linear
    h      = h + delta;  delta = MoE(norm(h))                        add_rmsnorm, DeviceLayer.forward

The latents stay in bf16 in both forms (rounding them to 8 bits for the
prompt's expansion would give a prompt other keys and values than the tokens
decoded after it), so the expansions W_uk and W_uv are bf16 and per head, as
given.

The block holds its weights (8-bit projections, bf16 expansions, the keys' one
in both orders) and the table of angles; the cache belongs to the caller, and
the residual stream and the MoE output go from block to block.
"""
from __future__ import annotations

from contextlib import contextmanager
from dataclasses import dataclass
from itertools import accumulate

import torch

from . import attention as A


@dataclass(frozen=True)
class BlockConfig:
    hidden: int = 6144
    heads: int = 64
    q_rank: int = 2048
    rank: int = 512
    rope: int = 64
    nope: int = 128
    vdim: int = 128
    page: int = 64
    eps: float = 1e-6

    @property
    def scale(self) -> float:
        return (self.nope + self.rope) ** -0.5


def rope_table(n: int, rope: int, base: float = 10000.0, device: str = "cuda:0"):
    """Cosines, then sines, of position * base^(-2 i / rope), from 64 bits."""
    angle = torch.arange(n, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, rope, 2, dtype=torch.float64) / rope)
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def random_weights(cfg: BlockConfig, seed: int, device: str = "cuda:0") -> dict:
    """bf16 weights of the block's shapes (there are no checkpoints here)."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(n, k):
        return (torch.randn(n, k, generator=g, device=device) * k ** -0.5).bfloat16()

    def gain(n):
        return (1.0 + 0.1 * torch.randn(n, generator=g, device=device)).bfloat16()

    head = cfg.nope + cfg.rope
    return {"norm_in": gain(cfg.hidden), "norm_q": gain(cfg.q_rank), "norm_kv": gain(cfg.rank), "norm_moe": gain(cfg.hidden),
            "q_a": normal(cfg.q_rank, cfg.hidden), "q_b": normal(cfg.heads * head, cfg.q_rank),
            "kv_a": normal(cfg.rank + cfg.rope, cfg.hidden), "kv_b": normal(cfg.heads * (cfg.nope + cfg.vdim), cfg.rank),
            "o": normal(cfg.hidden, cfg.heads * cfg.vdim)}


class LatentCache:
    """Pages of one block's latent cache and the page lists of its sequences."""

    def __init__(self, cfg: BlockConfig, n_pages: int, max_seqs: int, max_len: int, device: str = "cuda:0"):
        self.cfg, self.max_len = cfg, max_len
        self.pool = torch.zeros(n_pages, cfg.page, cfg.rank + cfg.rope, dtype=torch.bfloat16, device=device)
        self.pages = torch.full((max_seqs, -(-max_len // cfg.page)), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(max_seqs, dtype=torch.int32, device=device)
        self.host_lens = [0] * max_seqs
        self._drafted = [0] * max_seqs  # rows at the end of a sequence that accept() has to decide on
        self._lists = [[] for _ in range(max_seqs)]
        self._free = list(range(n_pages))[::-1]

    def _slot(self, b: int, p: int) -> int:
        """Cache row of place p of sequence b."""
        return self._lists[b][p // self.cfg.page] * self.cfg.page + p % self.cfg.page

    def _check(self, counts) -> None:
        """Refuses counts that extend() could not place."""
        if len(counts) > len(self.host_lens):
            raise ValueError(f"{len(counts)} sequences, the cache holds {len(self.host_lens)}")
        pages = 0
        for b, n in enumerate(counts):
            rows = self.host_lens[b] + n
            if n and self._drafted[b]:
                raise ValueError(f"sequence {b} ends with {self._drafted[b]} drafted tokens: accept() some of them first")
            if n < 0 or rows > self.max_len:
                raise ValueError(f"sequence {b}: {n} new rows after {self.host_lens[b]}, the cache holds {self.max_len} per "
                                 "sequence")
            pages += -(-rows // self.cfg.page) - len(self._lists[b])
        if pages > len(self._free):
            raise ValueError(f"{pages} more pages are needed, the latent cache has {len(self._free)} free ones")

    def extend(self, counts, drafted: bool = False):
        """Makes room for counts[b] new rows of sequence b.  Returns their
        positions (int32) and cache rows (int64), sequence after sequence.
        What does not fit is refused as a whole: nothing has changed then.
        drafted: the rows are drafts, on which accept() decides before their
        sequences go on."""
        self._check(counts)
        positions, slots, dev = [], [], self.pool.device
        for b, n in enumerate(counts):
            have, pages = self.host_lens[b], self._lists[b]
            held = len(pages)
            while len(pages) * self.cfg.page < have + n:
                pages.append(self._free.pop())
            if len(pages) > held:
                self.pages[b, held:len(pages)] = torch.tensor(pages[held:], dtype=torch.int32)
            positions += range(have, have + n)
            slots += [self._slot(b, p) for p in range(have, have + n)]
            self.host_lens[b] = have + n
            if drafted:
                self._drafted[b] += n
        self.lens.copy_(torch.tensor(self.host_lens, dtype=torch.int32))
        return (torch.tensor(positions, dtype=torch.int32).to(dev), torch.tensor(slots, dtype=torch.int64).to(dev))

    def _cut(self, lens) -> None:
        """Keeps the first lens[b] rows of sequence b and frees the pages after them."""
        for b, n in enumerate(lens):
            keep = -(-n // self.cfg.page)
            self._free += self._lists[b][keep:][::-1]
            del self._lists[b][keep:]
            self.host_lens[b] = n
        self.lens.copy_(torch.tensor(self.host_lens, dtype=torch.int32))

    @contextmanager
    def step(self, counts, drafted: bool = False):
        """extend() around the calls that fill the rows: if one of them is
        refused, the rows are taken back."""
        before, drafts = list(self.host_lens), list(self._drafted)
        rows = self.extend(counts, drafted)
        try:
            yield rows
        except BaseException:
            self._cut(before)
            self._drafted = drafts
            raise

    def accept(self, kept) -> None:
        """Ends a step of drafted tokens.  kept[b] names those of sequence b's
        drafts that stay (0 the first; a branch is all of its tokens from the
        root on): their rows move together behind the context, all others go,
        and their pages are free again.  A sequence past the end of kept keeps
        none."""
        kept = [list(k) for k in kept] + [[]] * (len(self.host_lens) - len(kept))
        if len(kept) > len(self.host_lens):
            raise ValueError(f"{len(kept)} sequences, the cache holds {len(self.host_lens)}")
        lens, moved = [], []
        for b, keep in enumerate(kept):
            if len(set(keep)) < len(keep) or any(not 0 <= j < self._drafted[b] for j in keep):
                raise ValueError(f"sequence {b}: {keep} of {self._drafted[b]} drafted tokens")
            first = self.host_lens[b] - self._drafted[b]
            moved += [(self._slot(b, first + i), self._slot(b, first + j)) for i, j in enumerate(keep) if i != j]
            lens.append(first + len(keep))
        if moved:
            to, source = torch.tensor(moved, dtype=torch.int64).t().contiguous().to(self.pool.device)
            rows = self.pool.view(-1, self.pool.shape[2])
            rows[to] = rows[source]  # read whole before the first is written
        self._cut(lens)
        self._drafted = [0] * len(lens)

    def truncate(self, b: int, length: int = 0) -> None:
        """Shortens sequence b to its first `length` rows (0 ends it); what
        is left counts as accepted, and pages no longer needed are free."""
        if not 0 <= length <= self.host_lens[b]:
            raise ValueError(f"sequence {b}: {length} of {self.host_lens[b]} rows")
        lens = list(self.host_lens)
        lens[b] = length
        self._cut(lens)
        self._drafted[b] = 0


class _Weights(dict):
    """The block's 8-bit projections by name, each (values, scales per 128 x
    128 block).  "kv_b" is held per head and in bf16, as its products take it:
    asked for here, it is put together again, with scales of one."""

    def __init__(self, projections, w_uk, w_uv):
        super().__init__(projections)
        self._kv_b = w_uk, w_uv

    def __missing__(self, name):
        if name != "kv_b":
            raise KeyError(name)
        w = torch.cat(self._kv_b, 1).flatten(0, 1)
        return w, torch.ones(-(-w.shape[0] // A.GROUP), -(-w.shape[1] // A.GROUP), device=w.device)


class DecoderBlock:
    """The attention half around a DeviceLayer (or None: attention only)."""

    def __init__(self, cfg: BlockConfig, weights: dict, moe=None, max_positions: int = 4096, device: str = "cuda:0"):
        self.cfg, self.moe = cfg, moe
        self.norms = {k: weights[k] for k in ("norm_in", "norm_q", "norm_kv", "norm_moe")}
        # the per-head expansions, for the absorbed form with the keys'
        # transposed (queries go the other way)
        full = weights["kv_b"].reshape(cfg.heads, cfg.nope + cfg.vdim, cfg.rank)
        self.w_uk = full[:, :cfg.nope].bfloat16().contiguous()
        self.w_uk_t = self.w_uk.transpose(1, 2).contiguous()
        self.w_uv = full[:, cfg.nope:].bfloat16().contiguous()
        self.lin = _Weights({k: A.quantize_weight(weights[k]) for k in ("q_a", "q_b", "kv_a", "o")}, self.w_uk, self.w_uv)
        self.table = rope_table(max_positions, cfg.rope, device=device)

    def _linear(self, x, name):
        return A.fp8_linear(x[0], x[1], *self.lin[name])

    def _queries(self, delta, residual):
        cfg = self.cfg
        n = A.add_rmsnorm(delta, self.norms["norm_in"], cfg.eps, residual=residual, out="fp8")
        x = (n.q, n.scale)
        qa = A.add_rmsnorm(self._linear(x, "q_a"), self.norms["norm_q"], cfg.eps, out="fp8")
        q = self._linear((qa.q, qa.scale), "q_b").view(-1, cfg.heads, cfg.nope + cfg.rope)
        return n.sum, q, self._linear(x, "kv_a")

    def _finish(self, o, h):
        """Output projection, second norm and the MoE layer: the residual and
        the next delta."""
        delta = self._linear(A.quantize(o.flatten(1)), "o")
        if self.moe is None:
            return h, delta
        n = A.add_rmsnorm(delta, self.norms["norm_moe"], self.cfg.eps, residual=h, out="bf16", sum_out=h)
        return h, self.moe.forward(n.y)[0]

    def _known(self, last: int) -> None:
        """Refuses text positions that the table of angles does not hold."""
        if last >= self.table.shape[0]:
            raise ValueError(f"position {last}: the block has a table of {self.table.shape[0]} (max_positions)")

    def _starts(self, counts):
        """Where each sequence's tokens start, and the last one's end."""
        return torch.tensor([0, *accumulate(counts)], dtype=torch.int32).to(self.table.device)

    def prompt(self, delta, residual, cache: LatentCache, counts):
        """Prompts of counts[b] tokens, one after another in delta and
        residual [T, hidden], for sequences that have no rows yet."""
        cfg = self.cfg
        if any(n and have for n, have in zip(counts, cache.host_lens)):
            raise ValueError("prompt() starts sequences; decode() continues them")
        self._known(max(counts, default=0) - 1)
        with cache.step(counts) as (positions, slots):
            h, q, kv = self._queries(delta, residual)
            new = A.latent_append(kv, self.norms["norm_kv"], cfg.eps, self.table, positions, slots, cache.pool,
                                  q_rope=q[..., cfg.nope:], q_out=q[..., cfg.nope:], want_key=True)
            latents = new.rows[:, None, :cfg.rank].expand(-1, cfg.heads, -1)  # every head reads the same
            k, v = A.head_linear(latents, self.w_uk), A.head_linear(latents, self.w_uv)
            cu = self._starts(counts)
            o = A.prompt_attention(q, k, new.key, v, cfg.scale, cu_q=cu, cu_k=cu, max_q=max(counts))
            return self._finish(o, h)

    def decode(self, delta, residual, cache: LatentCache, count=1, tree=None, positions=None):
        """`count` new tokens of every sequence, or count[b] of sequence b
        (0: it sits out), one sequence after another in delta and residual
        [T, hidden]: one decoded token, a causal chunk, or with tree (int64
        masks [T]) up to 64 drafted tokens, whose positions in the text the
        caller gives (a list, or int32 [T] on the device, which is not looked
        at here: a position outside the table makes NaN of its token; siblings
        share one).  After drafted tokens cache.accept() says which of them
        stay; until then their sequences do not go on."""
        cfg, seqs = self.cfg, len(cache.host_lens)
        counts = [count] * seqs if isinstance(count, int) else [*count, *[0] * (seqs - len(count))]
        running = [b for b, n in enumerate(counts) if n]
        most = max(counts)
        if tree is not None and most > 64:
            raise ValueError(f"{most} drafted tokens in a sequence: a mask has 64 bits")
        if positions is None:
            self._known(max((have + n - 1 for have, n in zip(cache.host_lens, counts) if n), default=0))
        elif not isinstance(positions, torch.Tensor):
            if min(positions, default=0) < 0:
                raise ValueError(f"position {min(positions)}")
            self._known(max(positions, default=0))
            positions = torch.tensor(positions, dtype=torch.int32).to(self.table.device)
        with cache.step(counts, drafted=tree is not None) as (following, slots):
            h, q, kv = self._queries(delta, residual)
            ql = torch.empty(q.shape[0], cfg.heads, cfg.rank + cfg.rope, dtype=torch.bfloat16, device=q.device)
            A.latent_append(kv, self.norms["norm_kv"], cfg.eps, self.table, following if positions is None else positions,
                            slots, cache.pool, q_rope=q[..., cfg.nope:], q_out=ql[..., cfg.rank:])
            A.head_linear(q[..., :cfg.nope], self.w_uk_t, out=ql[..., :cfg.rank])
            cu = None if min(counts) == most else self._starts(counts)
            o = A.latent_attention(ql, cache.pool, cache.pages, cache.lens, cfg.scale, cu_q=cu, max_q=most, tree=tree,
                                   max_len=max((cache.host_lens[b] for b in running), default=0))
            return self._finish(A.head_linear(o, self.w_uv), h)


def main() -> None:
    """A GLM-shaped block on synthetic weights: one prompt of 2048 tokens, then
    single tokens and trees of 4 drafted tokens for 8 sequences."""
    import time

    cfg = BlockConfig()
    block = DecoderBlock(cfg, random_weights(cfg, 0))
    cache = LatentCache(cfg, n_pages=8 * 40, max_seqs=8, max_len=2400)

    def timed(what, call, n):
        call()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            call()
        torch.cuda.synchronize()
        print(f"{what}: {(time.perf_counter() - t) / n * 1e6:.1f} us", flush=True)

    def inputs(T):
        return torch.randn(T, cfg.hidden, device="cuda:0"), torch.randn(T, cfg.hidden, device="cuda:0").bfloat16()

    counts = [2048] + [2048 - 64 * b for b in range(1, 8)]
    x, r = inputs(sum(counts))
    block.prompt(x, r, cache, counts)
    x, r = inputs(8)
    timed("one token for each of 8 sequences, attention half", lambda: block.decode(x, r, cache), 20)
    x4, r4 = inputs(32)
    tree = torch.tensor([1, 3, 5, 11] * 8, dtype=torch.int64, device="cuda:0")  # branches 0 1 3 and 0 2

    def verify():
        at = [n + d for n in cache.host_lens for d in (0, 1, 1, 2)]
        block.decode(x4, r4, cache, 4, tree=tree, positions=at)
        cache.accept([[0, 2]] * 8)

    timed("a tree of 4 drafted tokens for each, two of them accepted, attention half", verify, 20)


if __name__ == "__main__":
    main()
