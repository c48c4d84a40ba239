"""The operators of one sparse-attention decode step, used together.

`DecodeCache` holds the private caches of a batch of requests that share a
prefix: keys, values and index keys by slot, each slot's position and running
attention mass.  A step appends the new tokens, lets the indexer choose slots
(idx_topk), covers every segment of the slots with a witness (witness_merge),
attends to the prefix and the chosen slots (attn_shared, which adds the weights
to the masses), and trims the caches to their budget by mass (cache_evict, which
moves keys, values and index keys alike).  The work is enqueued on the current
stream.

The segments are equal shares of a request's filled slots.  Until the first trim
slots are positions, and a segment is a stretch of the context.  A trim moves
rows into freed slots, out of the order of their positions: from then on a
segment is a share of what is kept, and its witness still one of its slots.

The caches, the chosen ids, the output and what a trim returns are allocated
once, the workspace with the first step.  The problems of a step are described
anew each time, because its queries are other tensors.

`PagedCache` holds the same batch's keys and values in pages of one pool, taken
as the requests grow and given back when they end.  It takes the projections'
rows as they are: a prompt or a step normalises and rotates queries, keys and the
indexer's rows and writes them where they belong in one launch (paged_append),
lets the indexer choose slots (idx_topk, witness_merge) and attends to them, or
to every slot, through the page table (attn_paged).
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import binding as B


class DecodeCache:
    def __init__(self, requests: int, slots: int, q_heads: int, kv_heads: int, dim: int, index_dim: int, top_k: int,
                 prefix_k: Optional[torch.Tensor] = None, prefix_v: Optional[torch.Tensor] = None,
                 dtype=torch.bfloat16, device="cuda", index_dtype=torch.bfloat16):
        """dtype (bfloat16 or float16): of keys, values and queries; index_dtype
        (bfloat16 or float32): of the indexer's keys and queries."""
        z = lambda *s, dt=dtype: torch.zeros(s, dtype=dt, device=device)  # noqa: E731
        self.k, self.v = z(requests, slots, kv_heads, dim), z(requests, slots, kv_heads, dim)
        self.index_k = z(requests, slots, index_dim, dt=index_dtype)
        self.lens = z(requests, 1, dt=torch.int32)
        self.pos = torch.full((requests, 1, slots), -1, dtype=torch.int32, device=device)
        self.mass = z(requests, 1, slots, dt=torch.float32)
        self.cur = z(requests, dt=torch.int32)            # positions seen so far
        self.filled = 0                                   # slots of the longest request, known to the host
        self.prefix_k, self.prefix_v = prefix_k, prefix_v
        self.top_k = top_k
        self.ids = z(requests, top_k, dt=torch.int32)
        self.out = z(requests, 1, q_heads, dim)
        self.key_off = torch.arange(requests, dtype=torch.int64, device=device) * slots
        self.rows = torch.arange(requests, device=device)
        self.src = z(requests * slots, dt=torch.int32)    # where a trim takes each slot from
        self.ws: Optional[torch.Tensor] = None

    def fill(self, k: torch.Tensor, v: torch.Tensor, index_k: torch.Tensor,
             lens: Optional[Sequence[int]] = None) -> None:
        """The prompts, into empty caches: k, v [B, n, kv_heads, dim], index_k
        [B, n, index_dim]; request b has lens[b] <= n tokens (n without lens)."""
        requests, slots = self.index_k.shape[:2]
        n = k.shape[1]
        lens = [n] * requests if lens is None else [int(x) for x in lens]
        if n > slots or len(lens) != requests or any(x < 0 or x > n for x in lens):
            raise ValueError(f"prompts of {n} tokens, lens {lens}: {requests} requests of {slots} slots")
        self.k[:, :n], self.v[:, :n], self.index_k[:, :n] = k, v, index_k
        self.lens[:, 0] = torch.tensor(lens, dtype=torch.int32).to(self.lens.device)
        self.cur.copy_(self.lens[:, 0])
        at = torch.arange(self.pos.shape[2], dtype=torch.int32, device=self.pos.device)
        self.pos[:, 0] = torch.where(at < self.lens, at, -1)
        self.mass.zero_()
        self.filled = max(lens, default=0)

    def append(self, k: torch.Tensor, v: torch.Tensor, index_k: torch.Tensor) -> None:
        """One token of every request: k, v [B, kv_heads, dim], index_k [B, index_dim].
        Full caches are refused: trim them first."""
        slots = self.index_k.shape[1]
        if self.filled >= slots:
            raise ValueError(f"append: a request's {slots} slots are full")
        # The count is the host's.  Lengths that were changed past it must not index
        # out of the caches: the kernels then report the length itself.
        at = self.lens[:, 0].long().clamp(0, slots - 1)
        self.k[self.rows, at], self.v[self.rows, at], self.index_k[self.rows, at] = k, v, index_k
        self.pos[self.rows, 0, at] = self.cur
        self.lens += 1
        self.cur += 1
        self.filled += 1

    def step(self, q: torch.Tensor, index_q: torch.Tensor, index_w: torch.Tensor, segments: int = 16) -> torch.Tensor:
        """q [B, 1, q_heads, dim]; index_q [B, H, index_dim], index_w [B, H] of the
        indexer.  Returns the attention output; its buffer is reused."""
        requests, slots = self.index_k.shape[:2]
        lens = self.lens.view(-1)
        p = B.Problem(index_q, index_w, self.index_k.view(requests * slots, -1), lens, slots, self.key_off)
        a = B.AttnProblem(q, q.shape[-1] ** -0.5, self.k, self.v, self.lens, self.prefix_k, self.prefix_v,
                          ids=self.ids.view(requests, 1, -1))
        need = max(B.idx_topk_workspace_size(p, self.top_k), B.attn_shared_workspace_size(a, True))
        if self.ws is None or self.ws.numel() < need:
            self.ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        B.idx_topk(p, self.top_k, self.ids, None, self.ws)
        B.witness_merge(self.ids, lens, max(self.top_k - segments, 0), segments, segments)
        B.attn_shared(a, self.out, None, self.mass, self.ws)
        return self.out

    def trim(self, n_keep: int, n_first: int, n_last: int) -> torch.Tensor:
        """Evicts every request down to n_keep slots.  Returns the slot that each
        new slot came from, [B, 1, n_keep] int32, -1 behind the new length; its
        buffer is reused."""
        requests, _, slots = self.mass.shape
        if not 0 < n_keep <= slots:
            raise ValueError(f"trim: n_keep={n_keep} of {slots} slots")
        p = B.EvictProblem(self.mass, self.lens, n_keep, n_first, n_last, self.pos, self.cur,
                           (self.k, self.v, self.index_k))
        src = self.src[: requests * n_keep].view(requests, 1, n_keep)
        B.cache_evict(p, src, self.lens, self.pos, self.mass)
        self.filled = min(self.filled, n_keep)
        return src


class PagedCache:
    def __init__(self, requests: int, max_len: int, n_pages: int, page_size: int, q_heads: int, kv_heads: int, dim: int,
                 index_heads: int = 0, index_dim: int = 128, top_k: Optional[int] = None, rot: Optional[int] = None,
                 index_rot: int = 64, base: float = 10000.0, eps: float = 1e-6, norms: Optional[dict] = None,
                 interleaved: bool = False, dtype=torch.bfloat16, device="cuda", index_dtype=torch.bfloat16):
        """max_len: slots that a request can grow to; n_pages pages of page_size slots
        for all of them.  dtype (bfloat16 or float16): of keys, values and queries;
        index_dtype (bfloat16 or float32): of the indexer's rows.  norms: float32 weights
        by name ("q", "k", "index_q", "index_k") of the rows that are normalised.
        index_heads 0: no indexer, every step attends to all slots; else to the top_k best
        and their witnesses.  The indexer's keys are read in one piece and stay by request
        and slot."""
        if not 0 < page_size or not 0 < max_len or n_pages < 0 or (index_heads > 0) != (top_k is not None):
            raise ValueError(f"max_len={max_len}, {n_pages} pages of {page_size}, {index_heads} index heads, top_k={top_k}")
        self._check_kinds(q_heads, kv_heads, dim, dim if rot is None else rot, dtype, eps)
        if index_heads:
            self._check_indexer(index_heads, index_dim, index_rot, index_dtype, top_k)
        for name, w in (norms or {}).items():
            n = {"q": dim, "k": dim, "index_q": index_dim, "index_k": index_dim}.get(name)
            if n is None or tuple(w.shape) != (n,) or w.dtype != torch.float32:
                raise ValueError(f"norms: {name!r}, {tuple(w.shape)} {w.dtype}")
        z = lambda *s, dt=dtype: torch.zeros(s, dtype=dt, device=device)  # noqa: E731
        self.page_size, self.max_len, self.cols = page_size, max_len, -(-max_len // page_size)
        self.k, self.v = z(n_pages, page_size, kv_heads, dim), z(n_pages, page_size, kv_heads, dim)
        self.table = torch.full((requests, self.cols), -1, dtype=torch.int32, device=device)
        self.lens, self.slot = z(requests, dt=torch.int32), torch.full((requests,), -1, dtype=torch.int32, device=device)
        self.live = z(requests, dt=torch.int32)           # 1: a step adds a token
        self.free = list(range(n_pages - 1, -1, -1))
        self.pages = [[] for _ in range(requests)]        # of each request, and how long the host knows it to be
        self.known = [0] * requests
        self.eps, self.norms, self.interleaved = eps, norms or {}, interleaved
        f = lambda n: B.rope_frequencies(n, base, device=device) if n else None  # noqa: E731
        self.freq = f(dim if rot is None else rot)
        self.q, self.out = z(requests, 1, q_heads, dim), z(requests, 1, q_heads, dim)
        self.top_k = top_k
        if index_heads:
            slots = self.cols * page_size
            self.index_freq = f(index_rot)
            self.index_k = z(requests, slots, index_dim, dt=index_dtype)
            self.index_q = z(requests, index_heads, index_dim, dt=index_dtype)
            self.index_table = torch.arange(requests * self.cols, dtype=torch.int32, device=device).view(requests, -1)
            self.key_off = torch.arange(requests, dtype=torch.int64, device=device) * slots
            self.ids = z(requests, 1, top_k, dt=torch.int32)
        self.ws: Optional[torch.Tensor] = None

    # What every step would be refused for: head rows, attention and the indexer each
    # take less than all sizes and types.
    @staticmethod
    def _check_kinds(q_heads, kv_heads, dim, rot, dtype, eps):
        if kv_heads < 1 or q_heads < 1 or q_heads % kv_heads or dim not in (64, 128):
            raise ValueError(f"{q_heads} query heads over {kv_heads} KV heads of {dim} (64 or 128)")
        if not 0 <= rot <= dim or rot % 16:
            raise ValueError(f"rot={rot}: a multiple of 16, at most {dim}")
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"dtype {dtype} (bfloat16 or float16)")
        if not 0 <= eps < float("inf"):
            raise ValueError(f"eps={eps}")

    @staticmethod
    def _check_indexer(heads, dim, rot, dtype, top_k):
        if not 0 < heads <= 128 or dim not in (32, 64, 128, 256) or heads * dim > 16384:
            raise ValueError(f"{heads} index heads of {dim}: at most 128, and 16384 elements, of 32, 64, 128 or 256")
        if not 0 <= rot <= dim or rot % 16:
            raise ValueError(f"index_rot={rot}: a multiple of 16, at most {dim}")
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"index_dtype {dtype} (bfloat16 or float32)")
        if not 0 < top_k <= B.IDX_MAX_K:
            raise ValueError(f"top_k={top_k} outside [1, {B.IDX_MAX_K}]")

    def _take(self, grow: dict) -> dict:
        """Pages for the requests (index -> length), all of them or none.  Returns how
        many each got."""
        want = {}
        for b, n in grow.items():
            if n > self.max_len:
                raise ValueError(f"request {b}: {n} slots of at most {self.max_len}")
            want[b] = max(0, -(-n // self.page_size) - len(self.pages[b]))
        if sum(want.values()) > len(self.free):
            raise ValueError(f"{sum(want.values())} pages wanted, {len(self.free)} are free")
        for b, n in want.items():
            if n:
                at = len(self.pages[b])
                self.pages[b] += [self.free.pop() for _ in range(n)]
                self.table[b, at: at + n] = torch.tensor(self.pages[b][at:], dtype=torch.int32).to(self.table.device)
        return want

    def _append(self, p: B.AppendProblem, grow: dict) -> None:
        """The rows of a described call into the caches of requests that become that
        long, on pages taken for it.  Where the library refuses it they go back."""
        took = self._take(grow)
        try:
            B.paged_append(p)
        except Exception:
            for b, n in reversed(took.items()):
                for _ in range(n):
                    self.free.append(self.pages[b].pop())
                self.table[b, len(self.pages[b]): len(self.pages[b]) + n] = -1
            raise
        for b, n in grow.items():
            self.known[b] = n

    def _check(self, b: int) -> None:
        if not 0 <= b < len(self.known):
            raise ValueError(f"request {b} of {len(self.known)}")

    def release(self, b: int) -> None:
        """Request b has ended: its pages are free again, later steps pass it by."""
        self._check(b)
        self.free += reversed(self.pages[b])
        self.pages[b], self.known[b] = [], 0
        self.table[b].fill_(-1)
        self.lens[b], self.live[b] = 0, 0

    def _planes(self, k, v, index_k, q=None, index_q=None):
        def plane(name, src, dst, freq, table=None):
            w = self.norms.get(name)
            return B.HeadPlane(src, dst, weight=w, eps=None if w is None else self.eps, freq=freq,
                               interleaved=self.interleaved, table=table)

        p = [plane("k", k, self.k, self.freq, self.table), B.HeadPlane(v, self.v, table=self.table)]
        if self.top_k is not None:
            if index_k is None or (q is not None and index_q is None):
                raise ValueError("the indexer's rows are missing")
            pool = self.index_k.view(-1, self.page_size, 1, self.index_k.shape[2])
            p.append(plane("index_k", index_k.unsqueeze(1), pool, self.index_freq, self.index_table))
        if q is not None:
            p.append(plane("q", q, self.q.squeeze(1), self.freq))
            if self.top_k is not None:
                p.append(plane("index_q", index_q, self.index_q, self.index_freq))
        return p

    def prompt(self, b: int, k: torch.Tensor, v: torch.Tensor, index_k: Optional[torch.Tensor] = None) -> None:
        """Request b begins, or goes on, with n tokens: k, v [n, kv_heads, dim],
        index_k [n, index_dim], not yet normalised and rotated."""
        self._check(b)
        first, n = self.known[b], k.shape[0]
        if n == 0:
            raise ValueError("a prompt without tokens")
        slot = torch.arange(first, first + n, dtype=torch.int32, device=k.device)
        append = B.AppendProblem(self._planes(k, v, index_k), slot, torch.full_like(slot, b))
        append.desc()                                     # (refuses wrong tensors before pages are taken)
        self._append(append, {b: first + n})
        self.lens[b], self.live[b] = first + n, 1

    def step(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, index_q: Optional[torch.Tensor] = None,
             index_k: Optional[torch.Tensor] = None, index_w: Optional[torch.Tensor] = None,
             segments: int = 16) -> torch.Tensor:
        """One token of every request that has begun: q [B, q_heads, dim], k and v
        [B, kv_heads, dim], index_q [B, index_heads, index_dim], index_k [B, index_dim],
        as the projections leave them; index_w [B, index_heads] float32, contiguous.  Rows
        of requests that have ended are passed by, their output is 0.  A step that is
        refused leaves the cache as it was.  Returns [B, 1, q_heads, dim]; its buffer is
        reused."""
        requests = self.lens.shape[0]
        grow = {b: n + 1 for b, n in enumerate(self.known) if n}
        longest = max(grow.values(), default=0)
        # Whatever can be refused is, before anything is changed.
        append = B.AppendProblem(self._planes(k, v, index_k, q, index_q), self.slot)
        append.desc()
        ids, need = None, 0
        if self.top_k is not None:
            heads = self.index_q.shape[1]
            if not 0 <= segments <= B.IDX_MAX_SEGMENTS:
                raise ValueError(f"segments={segments} outside [0, {B.IDX_MAX_SEGMENTS}]")
            if index_w is None or index_w.numel() != requests * heads or index_w.shape[-1] != heads:
                raise ValueError(f"index_w: expected [{requests}, {heads}], got "
                                 f"{None if index_w is None else tuple(index_w.shape)}")
            if index_w.device != self.lens.device:
                raise ValueError(f"index_w: on {index_w.device}, the cache is on {self.lens.device}")
            ids, slots = self.ids, self.index_k.shape[1]
            p = B.Problem(self.index_q, index_w, self.index_k.view(requests * slots, -1), self.lens, max(longest, 1),
                          self.key_off)
            need = B.idx_topk_workspace_size(p, self.top_k)
        a = B.PagedAttnProblem(self.q, q.shape[-1] ** -0.5, self.k, self.v, self.table, self.lens, longest, ids)
        need = max(need, B.attn_paged_workspace_size(a))
        if self.ws is None or self.ws.numel() < need:
            self.ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        self.lens += self.live
        torch.sub(self.lens, 1, out=self.slot)            # -1 for those that have ended
        try:
            self._append(append, grow)
        except Exception:
            self.lens -= self.live
            raise
        if ids is not None:
            flat = ids.view(requests, -1)
            B.idx_topk(p, self.top_k, flat, None, self.ws)
            B.witness_merge(flat, self.lens, max(self.top_k - segments, 0), segments, segments)
        B.attn_paged(a, self.out, None, self.ws)
        return self.out


def decode_step_example(seed: int = 0, requests: int = 8, prefix: int = 1000, slots: int = 2100, K: int = 256,
                        n_keep: int = 2000, q_heads: int = 32, kv_heads: int = 4, dim: int = 128,
                        index_heads: int = 16) -> dict:
    """Fills the caches, runs a few decode steps with random tokens and trims."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    c = DecodeCache(requests, slots, q_heads, kv_heads, dim, 128, K, rn(prefix, kv_heads, dim),
                    rn(prefix, kv_heads, dim))
    n = slots - 4
    c.fill(rn(requests, n, kv_heads, dim), rn(requests, n, kv_heads, dim), rn(requests, n, 128))
    finite = True
    for _ in range(4):
        c.append(rn(requests, kv_heads, dim), rn(requests, kv_heads, dim), rn(requests, 128))
        out = c.step(rn(requests, 1, q_heads, dim), rn(requests, index_heads, 128),
                     torch.rand((requests, index_heads), generator=g, device="cuda"))
        finite &= bool(torch.isfinite(out).all())
    c.trim(n_keep, 4, n_keep // 8)
    return {"len_after": c.lens.view(-1).tolist(), "finite": finite, "mass": c.mass[..., :n_keep], "pos": c.pos}


def paged_step_example(seed: int = 0, requests: int = 8, max_len: int = 4096, page_size: int = 64, top_k: int = 256,
                       q_heads: int = 32, kv_heads: int = 4, dim: int = 128, index_heads: int = 16) -> dict:
    """Requests of several lengths begin, take a few steps with random tokens, and
    one of them ends."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    norms = {n: torch.ones(dim, device="cuda") for n in ("q", "k")}
    c = PagedCache(requests, max_len, requests * max_len // page_size // 2, page_size, q_heads, kv_heads, dim, index_heads,
                   128, top_k, norms=norms)
    for b in range(requests):
        n = max(1, (max_len // 2 - 8) * (b + 1) // requests)
        c.prompt(b, rn(n, kv_heads, dim), rn(n, kv_heads, dim), rn(n, 128))
    finite = True
    for i in range(4):
        if i == 2:
            c.release(0)
        out = c.step(rn(requests, q_heads, dim), rn(requests, kv_heads, dim), rn(requests, kv_heads, dim),
                     rn(requests, index_heads, 128), rn(requests, 128),
                     torch.rand((requests, index_heads), generator=g, device="cuda"))
        finite &= bool(torch.isfinite(out).all())
    return {"lens": c.lens.tolist(), "free": len(c.free), "finite": finite, "ended": bool((out[0] == 0).all())}


if __name__ == "__main__":
    got = decode_step_example()
    print("slots kept per request:", got["len_after"], "finite outputs:", got["finite"])
    got = paged_step_example()
    print("slots per request in pages:", got["lens"], "free pages:", got["free"], "finite outputs:", got["finite"])
