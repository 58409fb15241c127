"""One decoder block: latent attention and the routed MoE layer.

    python -m routed_expert_int4_amd.block            # a prompt, then decoded tokens, timed

Per token (colibri summary, "Principales fonctionnalites": q/kv-LoRA, partial
interleaved rotary positions, one latent vector per token in the cache):

    h      = residual + delta;  x = norm(h)                          add_rmsnorm, 8-bit out (bf16 for 4-bit weights)
    q      = W_qb norm(W_qa x);  c | k_r = W_kva x                   fp8_linear or int4_linear, add_rmsnorm
    cache <- norm(c) | rotate(k_r);  q_r = rotate(q_r)               latent_append
    prompt:  k = W_uk c, v = W_uv c per head, attention over them    (latent_read,) head_linear, prompt_attention
    decode:  q_c = q W_uk per head, attention over the cache,        head_linear, latent_attention,
             o = W_uv o_c per head                                   head_linear
    delta  = W_o o                                                   quantize, fp8_linear, or int4_linear
    h      = h + delta;  delta = MoE(norm(h))                        add_rmsnorm, DeviceLayer.forward

The latents are the cache's in both forms: bf16 rows as they are written, or
rows of 8 bits, which a prompt reads back before it expands them (with any
other rounding a prompt would have other keys and values than the tokens
decoded after it).  The expansions W_uk and W_uv are bf16 and per head, as
given.

The block holds its weights (8-bit or 4-bit projections, bf16 expansions, the
keys' one in both orders) and the table of angles; the cache belongs to the
caller, and the residual stream and the MoE output go from block to block.  A
cache can make one sequence's rows the prefix of all its sequences: a long
common context is then held, and read in each step, once.
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
    weight_bits: int = 8   # of the projections: 8 (a scale per 128 x 128 block) or 4 (a scale per 32 columns)
    cache_bits: int = 16   # of the cached latents: 16, or 8 with a power of two per row

    def __post_init__(self):
        if self.weight_bits not in (4, 8) or self.cache_bits not in (8, 16):
            raise ValueError(f"{self.weight_bits}-bit weights, {self.cache_bits}-bit cache: 4 or 8, and 8 or 16 are there")

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
        narrow = cfg.cache_bits == 8
        self.pool = torch.zeros(n_pages, cfg.page, cfg.rank + (2 if narrow else 1) * cfg.rope,
                                dtype=torch.uint8 if narrow else torch.bfloat16, device=device)
        self.scale = torch.ones(n_pages, cfg.page, device=device) if narrow else None  # of rows of 8 bits
        self.prefix, self.prefix_len = None, 0  # rows before every sequence's own: share()
        self.pages = torch.full((max_seqs, -(-max_len // cfg.page)), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(max_seqs, dtype=torch.int32, device=device)
        self.host_lens = [0] * max_seqs
        self._drafted = [0] * max_seqs  # rows at the end of a sequence that accept() has to decide on
        self._lists = [[] for _ in range(max_seqs)]
        self._free = list(range(n_pages))[::-1]
        self._prefix_list = []

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
        positions (int32; a prefix comes first) and cache rows (int64),
        sequence after sequence.  What does not fit is refused as a whole: nothing has changed then.
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
            positions += range(self.prefix_len + have, self.prefix_len + have + n)
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
            if self.scale is not None:
                scale = self.scale.view(-1)
                scale[to] = scale[source]
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


    def share(self, b: int) -> None:
        """Makes the rows of sequence b the prefix of all sequences: they are
        before each one's own rows from now on, b's own being none.  All other
        sequences have to be empty, and b without undecided drafts.  It is held
        once.  Steps on a long one take less time than with its pages in every
        sequence's own list where a token has fewer than 64 heads (32 sequences
        on 16384 rows, 16 heads: 51 against 93 us); with 64, or after a few
        thousand rows, as much or up to a fifth more."""
        if self.prefix is not None:
            raise ValueError("there is a prefix already: drop_prefix() first")
        others = [n for i, n in enumerate(self.host_lens) if i != b]
        if self._drafted[b] or not self.host_lens[b] or any(others):
            raise ValueError(f"sequence {b} has {self.host_lens[b]} rows ({self._drafted[b]} drafted), the others {others}: "
                             "rows of one sequence alone, accepted, are needed")
        dev = self.pool.device
        self.prefix_len, self._prefix_list = self.host_lens[b], self._lists[b]
        self.prefix = A.SharedPrefix(torch.tensor([self._prefix_list], dtype=torch.int32).to(dev),
                                     torch.tensor([self.prefix_len], dtype=torch.int32).to(dev), self.prefix_len)
        self._lists[b] = []
        self._cut([0] * len(self.host_lens))

    def drop_prefix(self) -> None:
        """Ends the prefix and frees its pages; all sequences have to be empty."""
        if any(self.host_lens):
            raise ValueError(f"sequences of {self.host_lens} rows follow the prefix: truncate() them first")
        self._free += self._prefix_list[::-1]
        self._prefix_list, self.prefix, self.prefix_len = [], None, 0


class _Weights(dict):
    """The block's projections by name, each (values, scales): of 8 bits with a
    scale per 128 x 128 block, or 4-bit codes with one per 32 columns.  "kv_b" is held per head and in bf16, as its products take it:
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
        pack = A.quantize_weight if cfg.weight_bits == 8 else A.quantize_weight_int4
        self.lin = _Weights({k: pack(weights[k]) for k in ("q_a", "q_b", "kv_a", "o")}, self.w_uk, self.w_uv)
        self.table = rope_table(max_positions, cfg.rope, device=device)

    def _linear(self, x, name):
        """x as _norm leaves it: (codes, scales) for 8-bit weights, bf16 for
        4-bit ones."""
        if self.cfg.weight_bits == 4:
            return A.int4_linear(x, *self.lin[name])
        return A.fp8_linear(x[0], x[1], *self.lin[name])

    def _norm(self, x, name, residual=None):
        """The sum, and its norm as _linear takes it."""
        wide = self.cfg.weight_bits == 4
        n = A.add_rmsnorm(x, self.norms[name], self.cfg.eps, residual=residual, out="bf16" if wide else "fp8")
        return n.sum, n.y if wide else (n.q, n.scale)

    def _queries(self, delta, residual):
        cfg = self.cfg
        h, x = self._norm(delta, "norm_in", residual)
        _, qa = self._norm(self._linear(x, "q_a"), "norm_q")
        q = self._linear(qa, "q_b").view(-1, cfg.heads, cfg.nope + cfg.rope)
        return h, q, self._linear(x, "kv_a")

    def _finish(self, o, h):
        """Output projection, second norm and the MoE layer: the residual and
        the next delta."""
        delta = self._linear(o.flatten(1) if self.cfg.weight_bits == 4 else A.quantize(o.flatten(1)), "o")
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
        residual [T, hidden], for sequences that have no rows yet and no
        prefix (decode() takes a whole prompt as one chunk after either; behind
        a prefix each of its tokens takes 8 heads (rank + 2) bytes of workspace,
        540 MB for 2048 at 64 heads and rank 512, so long ones go in several)."""
        cfg = self.cfg
        if cache.prefix is not None or any(n and have for n, have in zip(counts, cache.host_lens)):
            raise ValueError("prompt() starts sequences; decode() continues them")
        self._known(max(counts, default=0) - 1)
        with cache.step(counts) as (positions, slots):
            h, q, kv = self._queries(delta, residual)
            new = A.latent_append(kv, self.norms["norm_kv"], cfg.eps, self.table, positions, slots, cache.pool,
                                  q_rope=q[..., cfg.nope:], q_out=q[..., cfg.nope:], want_key=cache.scale is None,
                                  cache_scale=cache.scale)
            rows = new.rows if cache.scale is None else A.latent_read(cache.pool, cache.scale, slots, cfg.rope)
            latents = rows[:, None, :cfg.rank].expand(-1, cfg.heads, -1)  # every head reads the same
            k, v = A.head_linear(latents, self.w_uk), A.head_linear(latents, self.w_uv)
            cu = self._starts(counts)
            o = A.prompt_attention(q, k, rows[:, cfg.rank:], v, cfg.scale, cu_q=cu, cu_k=cu, max_q=max(counts))
            return self._finish(o, h)

    def decode(self, delta, residual, cache: LatentCache, count=1, tree=None, positions=None):
        """`count` new tokens of every sequence, or count[b] of sequence b
        (0: it sits out), one sequence after another in delta and residual
        [T, hidden]: one decoded token, a causal chunk, or with tree (int64
        masks [T]) up to 64 drafted tokens, whose positions in the text the
        caller gives (a list, or int32 [T] on the device, which is not looked
        at here: a position outside the table makes NaN of its token; siblings
        share one, and a prefix's rows count).  After drafted tokens cache.accept() says which of them
        stay; until then their sequences do not go on."""
        cfg, seqs = self.cfg, len(cache.host_lens)
        counts = [count] * seqs if isinstance(count, int) else [*count, *[0] * (seqs - len(count))]
        running = [b for b, n in enumerate(counts) if n]
        most = max(counts)
        if tree is not None and most > 64:
            raise ValueError(f"{most} drafted tokens in a sequence: a mask has 64 bits")
        if positions is None:
            self._known(max((cache.prefix_len + have + n - 1 for have, n in zip(cache.host_lens, counts) if n), default=0))
        elif not isinstance(positions, torch.Tensor):
            if min(positions, default=0) < 0:
                raise ValueError(f"position {min(positions)}")
            self._known(max(positions, default=0))
            positions = torch.tensor(positions, dtype=torch.int32).to(self.table.device)
        with cache.step(counts, drafted=tree is not None) as (following, slots):
            h, q, kv = self._queries(delta, residual)
            ql = torch.empty(q.shape[0], cfg.heads, cfg.rank + cfg.rope, dtype=torch.bfloat16, device=q.device)
            A.latent_append(kv, self.norms["norm_kv"], cfg.eps, self.table, following if positions is None else positions,
                            slots, cache.pool, q_rope=q[..., cfg.nope:], q_out=ql[..., cfg.rank:], cache_scale=cache.scale)
            A.head_linear(q[..., :cfg.nope], self.w_uk_t, out=ql[..., :cfg.rank])
            cu = None if min(counts) == most else self._starts(counts)
            o = A.latent_attention(ql, cache.pool, cache.pages, cache.lens, cfg.scale, cu_q=cu, max_q=most, tree=tree,
                                   max_len=max((cache.host_lens[b] for b in running), default=0), cache_scale=cache.scale,
                                   prefix=cache.prefix)
            return self._finish(A.head_linear(o, self.w_uv), h)


def main() -> None:
    """A GLM-shaped block on synthetic weights: one prompt of 2048 tokens, then
    single tokens and trees of 4 drafted tokens for 8 sequences, and 8 sequences
    after 2048 tokens that they share; the same with 4-bit projections and an
    8-bit cache."""
    for cfg in (BlockConfig(), BlockConfig(weight_bits=4, cache_bits=8)):
        demo(cfg)


def demo(cfg: BlockConfig) -> None:
    import time

    print(f"{cfg.weight_bits}-bit projections, {cfg.cache_bits}-bit cache", flush=True)
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

    common = LatentCache(cfg, n_pages=8 * 40, max_seqs=8, max_len=2400)
    block.prompt(*inputs(2048), common, [2048])
    common.share(0)
    timed("one token for each of 8 sequences after 2048 common ones, attention half", lambda: block.decode(x, r, common), 20)


if __name__ == "__main__":
    main()
