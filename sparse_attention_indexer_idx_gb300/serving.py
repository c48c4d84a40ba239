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


if __name__ == "__main__":
    got = decode_step_example()
    print("slots kept per request:", got["len_after"], "finite outputs:", got["finite"])
