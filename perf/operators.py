"""Measured cases of the attention and cache-eviction operators.

Two operators, as a decode step uses them after the indexer has chosen tokens:

attn   attention of a batch of requests over a prefix that all of them share
       (stored once) and each request's own cache behind it: every slot of
       that cache, or the slots that a selection lists; the sum of each slot's
       attention weights is added to its running mass;
evict  eviction from the requests' caches by that mass: the slots with the
       largest mass stay, next to the first and the last positions, and the
       rows of the cache move into the slots that became free.

`run` computes them in plain torch operations in 32 bits, or, with `own`, by
the library's entry points.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases --
def _attn(name=None, **kw):
    c = dict(op="attn", B=1, T=1, Hq=32, Hkv=8, D=128, P=0, S=1, W=0, ids_per_head=False, mass="head",
             ragged=True, part_prefix=False, layout="bshd", dtype="bf16")
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def _evict(name=None, **kw):
    c = dict(op="evict", B=1, Hm=8, Hkv=8, S=64, keep=32, first=4, last=16, D=128, ikeys=False, ragged=True,
             layout="bshd", dtype="bf16")
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one chat request behind a system prompt: the latency of a single call
        _attn("one request", P=1024, S=200),
        # a batch of chats behind one system prompt, ragged private parts
        _attn("batch 32", B=32, P=8192, S=1024),
        # several drafted tokens a request, odd lengths, heads of 64, fp16, head-major cache
        _attn("drafted tokens", B=16, T=5, Hq=32, Hkv=4, D=64, P=4095, S=777, dtype="f16", layout="bhsd"),
        # a document that many requests ask about: matrix-bound, the largest
        _attn("shared document", B=128, Hq=64, Hkv=8, P=65536, S=2048),
        # one key and value head for each query head; some requests share only part of the prefix
        _attn("one head each", B=24, Hq=16, Hkv=16, P=5000, S=333, part_prefix=True, mass="none"),
        # long private caches and no shared part: bound by reading them
        _attn("private caches", B=16, Hq=64, Hkv=8, S=32768, mass="all"),
        # the indexer's 2048 tokens of each request's 32,768
        _attn("selected 2048", B=64, Hq=32, Hkv=4, S=32768, W=2048, mass="all"),
        # selections of each drafted token and key head (block selection) behind a prefix, fp16
        _attn("selected, drafted", B=8, T=3, Hq=64, Hkv=8, D=64, P=1000, S=8000, W=1023, ids_per_head=True,
              dtype="f16"),
        # one cache just over its budget
        _evict("one cache", S=1040, keep=1024, Hm=8, ragged=False),
        # a decode batch trimmed back to its budget, each key head for itself
        _evict("trim a batch", B=64, S=4160, keep=4096, last=256, Hm=8, ragged=False),
        # after a prompt: an eighth of the slots stays, one choice for all heads, index keys moved along
        _evict("after the prompt", B=4, S=131072, keep=16384, last=1024, Hm=1, ikeys=True),
        # half of each cache goes, odd sizes, head-major, fp16
        _evict("half", B=24, S=10007, keep=5001, last=501, Hm=4, Hkv=4, D=64, layout="bhsd", dtype="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _cost(c):
    w = work(c)
    if c["op"] == "attn":
        # the plain form's 32-bit scores, and its gathered rows
        lanes = c["B"] * c["T"] * c["Hq"] * (c["P"] + (c["W"] or c["S"]))
        rows = c["B"] * c["T"] * c["W"] * c["Hkv"] * c["D"]
        return max(lanes / 6e8, rows / 4e8, _cache_elems(c) / 1.2e9, w["flops"] / 3e11)
    return max(_cache_elems(c) / 1.2e9, c["B"] * c["Hm"] * c["S"] / 3e7)


def _cache_elems(c):
    return c["B"] * c["S"] * c["Hkv"] * c["D"]


def draw(rng):
    while True:
        if rng.random() < 0.35:
            Hkv = rng.choice([1, 2, 4, 8])
            S = _log(rng, 16, 131072)
            keep = max(1, min(S, int(S * rng.choice([0.125, 0.25, 0.5, 0.75, 0.97]) + rng.randint(0, 5))))
            c = _evict(B=_log(rng, 1, 64), Hkv=Hkv, Hm=rng.choice([1, Hkv]), S=S, keep=keep,
                       first=min(keep // 2, rng.randint(0, 8)), last=int(keep * rng.uniform(0, 0.4)),
                       D=rng.choice([64, 128]), ragged=rng.random() < 0.7, layout=rng.choice(["bshd", "bhsd"]),
                       dtype=rng.choice(["bf16", "f16"]))
            c["ikeys"] = c["Hm"] == 1 and rng.random() < 0.6
        else:
            Hkv, G = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 4, 7, 8, 16])
            T = rng.choice([1, 1, 1, 2, 4, 8])
            P = 0 if rng.random() < 0.2 else _log(rng, 1, 65536)
            S = _log(rng, T, 32768)
            W = _log(rng, 1, min(S, 2048)) if rng.random() < 0.35 else 0
            c = _attn(B=_log(rng, 1, 128), T=T, Hq=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128]), P=P, S=S, W=W,
                      ids_per_head=W > 0 and rng.random() < 0.4, mass=rng.choice(["none", "head", "all"]),
                      ragged=rng.random() < 0.8, part_prefix=P > 0 and rng.random() < 0.3,
                      layout=rng.choice(["bshd", "bhsd"]), dtype=rng.choice(["bf16", "bf16", "f16"]))
        if _cost(c) <= 1.0:
            return c


def _lens(c):
    """The requests' private lengths: from half the slots to all of them, the same set for every seed."""
    B, S, least = c["B"], c["S"], c.get("T", 1)
    if not c["ragged"]:
        return [S] * B
    return [max(least, S - (i * 37 % B) * (S // 2) // B) for i in range(B)]


def _prefix_lens(c):
    if not c["part_prefix"]:
        return [c["P"]] * c["B"]
    return [c["P"] - (i * 13 % 4) * (c["P"] // 4) for i in range(c["B"])]


def work(c):
    if c["op"] == "attn":
        B, T, Hq, Hkv, D, W = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "W"))
        lens, pl = _lens(c), _prefix_lens(c)
        byte = 2 * B * T * Hq * D * 2 + B * T * Hq * 4 + 2 * max(pl + [0]) * Hkv * D * 2
        keys = T * sum(pl)  # (token, key) pairs of one head
        if W:
            listed_ids = T * sum(min(W, n) for n in lens)
            byte += 2 * listed_ids * Hkv * D * 2 + B * T * W * 4 * (Hkv if c["ids_per_head"] else 1)
            touched = sum(min(W * T * (Hkv if c["ids_per_head"] else 1), n) for n in lens)
            keys += listed_ids
        else:
            byte += 2 * sum(lens) * Hkv * D * 2
            touched = sum(lens)
            keys += T * sum(lens) - B * T * (T - 1) // 2
        if c["mass"] != "none":
            byte += 8 * touched * (Hkv if c["mass"] == "head" else 1)
        return {"bytes": byte, "flops": 4 * keys * Hq * D}
    B, Hm, Hkv, D, keep = (c[k] for k in ("B", "Hm", "Hkv", "D", "keep"))
    byte = moved = 0
    for n in _lens(c):
        byte += Hm * (8 * n + 12 * min(n, keep))
        if n > keep:
            # of the kept slots that are not protected, a share (n - keep) / n lies behind the budget
            moved += (Hkv if Hm == 1 else Hm) * int(keep * (n - keep) / n)
    row = 2 * D * 2  # a key and a value
    byte += 2 * moved * row
    if c["ikeys"]:
        byte += 2 * (moved // Hkv) * 128 * 2
    return {"bytes": byte, "flops": 0}


# ------------------------------------------------------------------ inputs --
def _rand(g, shape, dtype, dev):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32 if dev == "cpu" else dtype).to(dtype)


def _cache(c, g, dev):
    """[B, S, Hkv, D] keys or values in the case's memory order."""
    B, S, Hkv, D = c["B"], c["S"], c["Hkv"], c["D"]
    if c["layout"] == "bhsd":
        return _rand(g, (B, Hkv, S, D), DT[c["dtype"]], dev).transpose(1, 2)
    return _rand(g, (B, S, Hkv, D), DT[c["dtype"]], dev)


def _hot(k, u, share, g):
    """Adds each head's direction to a share of the keys: the tokens that attention goes to."""
    n = k.shape[-3]
    pick = torch.rand(n, generator=g, device=k.device) < share
    pick[: min(4, n)] = True
    at = pick.nonzero().squeeze(1)
    k[..., at, :, :] = (k[..., at, :, :].float() + 0.6 * u).to(k.dtype)
    return k


def prepare(c, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = DT[c["dtype"]]
    B, S, Hkv, D = c["B"], c["S"], c["Hkv"], c["D"]
    perm = torch.randperm(B, generator=g, device=dev)
    lens = torch.tensor(_lens(c), dtype=torch.int32, device=dev)[perm]
    st = {"case": c}
    if c["op"] == "attn":
        T, Hq, P, W = c["T"], c["Hq"], c["P"], c["W"]
        u = torch.randn((Hkv, D), generator=g, device=dev)
        u = u * (math.sqrt(D) / u.norm(dim=1, keepdim=True))
        q = torch.randn((B, T, Hkv, Hq // Hkv, D), generator=g, device=dev) + 0.6 * u[:, None]
        st["q"] = q.reshape(B, T, Hq, D).to(dt)
        st["scale"] = 1.0 / math.sqrt(D)
        st["k"], st["v"] = _hot(_cache(c, g, dev), u, 0.01, g), _cache(c, g, dev)
        st["lens"] = lens
        st["pk"] = st["pv"] = st["prefix_len"] = st["ids"] = st["mass"] = None
        if P:
            st["pk"] = _hot(_rand(g, (P, Hkv, D), dt, dev), u, 0.005, g)
            st["pv"] = _rand(g, (P, Hkv, D), dt, dev)
        if c["part_prefix"]:
            st["prefix_len"] = torch.tensor(_prefix_lens(c), dtype=torch.int32, device=dev)[perm]
        if W:
            # distinct visible slots in no order (a top-K lists them by score), -1 behind the last
            shape = (B, T, Hkv if c["ids_per_head"] else 1, S)
            r = torch.rand(shape, generator=g, device=dev)
            t = torch.arange(T, device=dev).view(1, T, 1, 1)
            seen = lens.view(B, 1, 1, 1) - T + t + 1
            r = torch.where(torch.arange(S, device=dev) < seen, r, -1.0)
            val, idx = r.topk(W, dim=-1)
            ids = torch.where(val >= 0, idx, -1).to(torch.int32)
            st["ids"] = ids if c["ids_per_head"] else ids.squeeze(2).contiguous()
        if c["mass"] != "none":
            shape = (B, Hkv if c["mass"] == "head" else 1, S)
            st["mass"] = torch.randn(shape, generator=g, device=dev).mul_(1.5).exp_()
        st["out"] = torch.empty((B, T, Hq, D), dtype=dt, device=dev)
        st["lse"] = torch.empty((B, T, Hq), dtype=torch.float32, device=dev)
        return st
    Hm, keep = c["Hm"], c["keep"]
    st["k"], st["v"] = _cache(c, g, dev), _cache(c, g, dev)
    if c["ikeys"]:
        st["ik"] = _rand(g, (B, S, 128), dt, dev)
    # heavy-tailed masses; a fifth of the slots was never attended to and ties at zero
    m = torch.randn((B, Hm, S), generator=g, device=dev).mul_(1.5).exp_()
    st["mass"] = torch.where(torch.rand((B, Hm, S), generator=g, device=dev) < 0.2, 0.0, m)
    st["lens"] = lens.view(B, 1).expand(B, Hm).contiguous()
    # earlier evictions left the positions in no order
    st["pos"] = torch.rand((B, Hm, S), generator=g, device=dev).argsort(dim=-1).to(torch.int32)
    st["cur"] = torch.full((B,), S, dtype=torch.int32, device=dev)
    for name, t in (("out_src", torch.int32), ("out_pos", torch.int32), ("out_mass", torch.float32)):
        st[name] = torch.empty((B, Hm, keep), dtype=t, device=dev)
    st["out_len"] = torch.empty((B, Hm), dtype=torch.int32, device=dev)
    return st


# -------------------------------------------------------------- plain form --
def _plain_attn(s):
    c = s["case"]
    B, T, Hq, Hkv, D, P, S, W = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "P", "S", "W"))
    dev = s["q"].device
    q = s["q"].float().view(B, T, Hkv, Hq // Hkv, D) * s["scale"]
    t = torch.arange(T, device=dev).view(1, T, 1)
    seen = s["lens"].view(B, 1, 1) - T + t + 1  # private slots that token t sees
    if W:
        ids = s["ids"].long() if c["ids_per_head"] else s["ids"].long().unsqueeze(2).expand(B, T, Hkv, W)
        see = (ids >= 0) & (ids < seen.unsqueeze(3))
        at = ids.clamp(0, S - 1)
        b = torch.arange(B, device=dev).view(B, 1, 1, 1)
        h = torch.arange(Hkv, device=dev).view(1, 1, Hkv, 1)
        x = torch.einsum("bthgd,bthwd->bthgw", q, s["k"][b, at, h].float())
        x = torch.where(see.unsqueeze(3), x, -math.inf)
        vx = s["v"][b, at, h].float()
    else:
        x = torch.einsum("bthgd,bshd->bthgs", q, s["k"].float())
        see = torch.arange(S, device=dev) < seen
        x = torch.where(see.view(B, T, 1, 1, S), x, -math.inf)
    top = x.amax(-1)
    if P:
        y = torch.einsum("bthgd,phd->bthgp", q, s["pk"].float())
        if s["prefix_len"] is not None:
            y = torch.where(torch.arange(P, device=dev) < s["prefix_len"].view(B, 1, 1, 1, 1), y, -math.inf)
        top = torch.maximum(top, y.amax(-1))
    base = torch.where(top == -math.inf, 0.0, top).unsqueeze(-1)
    x = torch.exp(x - base)
    total = x.sum(-1)
    o = torch.einsum("bthgw,bthwd->bthgd", x, vx) if W else torch.einsum("bthgs,bshd->bthgd", x, s["v"].float())
    if P:
        y = torch.exp(y - base)
        total = total + y.sum(-1)
        o = o + torch.einsum("bthgp,phd->bthgd", y, s["pv"].float())
    some = total > 0
    o = torch.where(some.unsqueeze(-1), o / torch.where(some, total, 1.0).unsqueeze(-1), 0.0)
    lse = torch.log(total) + base.squeeze(-1)
    s["out"].copy_(o.view(B, T, Hq, D))
    s["lse"].copy_(lse.view(B, T, Hq))
    if s["mass"] is not None:
        w = x / torch.where(some, total, 1.0).unsqueeze(-1)
        if W:
            w = w.sum(3)  # [B, T, Hkv, W]
            if c["mass"] == "all":
                add = torch.zeros((B, S), device=dev)
                add.scatter_add_(1, at.reshape(B, -1), w.reshape(B, -1))
                s["mass"] += add.unsqueeze(1)
            else:
                add = torch.zeros((B, Hkv, S), device=dev)
                add.scatter_add_(2, at.transpose(1, 2).reshape(B, Hkv, -1), w.transpose(1, 2).reshape(B, Hkv, -1))
                s["mass"] += add
        else:
            w = w.sum((1, 3))  # [B, Hkv, S]
            s["mass"] += w.sum(1, keepdim=True) if c["mass"] == "all" else w
    return {"out": s["out"], "lse": s["lse"], "mass": s["mass"]}


def _plain_evict(s):
    c = s["case"]
    B, S, Hm, Hkv, keep = (c[k] for k in ("B", "S", "Hm", "Hkv", "keep"))
    dev = s["mass"].device
    slot = torch.arange(S, device=dev)
    n = s["lens"].long().unsqueeze(-1)
    new = n.clamp(max=keep)
    cur = s["cur"].view(B, 1, 1)
    guard = (s["pos"] < c["first"]) | (s["pos"] >= cur - c["last"])
    rank = torch.where(guard, math.inf, s["mass"])
    rank = torch.where(slot < n, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.zeros((B, Hm, S), dtype=torch.bool, device=dev)
    kept.scatter_(2, order, slot[:keep] < new)
    # the slots behind the budget that stay, ascending, go to the freed slots before it, ascending
    tail = torch.sort(torch.where(kept & (slot >= new), slot, S), dim=-1).values[..., :keep]
    hole = ~kept[..., :keep] & (slot[:keep] < new)
    nth = (hole.long().cumsum(-1) - 1).clamp(min=0)
    src = torch.where(hole, tail.gather(-1, nth), slot[:keep])
    here = slot[:keep] < new
    at = src.clamp(max=S - 1)
    s["out_src"].copy_(torch.where(here, src, -1))
    s["out_len"].copy_(new.squeeze(-1))
    s["out_pos"].copy_(torch.where(here, s["pos"].gather(2, at), -1))
    s["out_mass"].copy_(torch.where(here, s["mass"].gather(2, at), 0.0))
    at = torch.where(here, at, slot[:keep]).expand(B, Hkv, keep).transpose(1, 2)
    b = torch.arange(B, device=dev).view(B, 1, 1)
    h = torch.arange(Hkv, device=dev).view(1, 1, Hkv)
    s["k"][:, :keep] = s["k"][b, at, h]
    s["v"][:, :keep] = s["v"][b, at, h]
    if c["ikeys"]:
        s["ik"][:, :keep] = s["ik"][b.squeeze(2), at[..., 0]]
    return _evict_out(s)


def _evict_out(s):
    return {k: s[k] for k in ("out_src", "out_len", "out_pos", "out_mass", "k", "v", "ik") if k in s}


# --------------------------------------------------------------------- run --
def run(s):
    c = s["case"]
    if not own:
        return _plain_attn(s) if c["op"] == "attn" else _plain_evict(s)
    from sparse_attention_indexer_idx_gb300 import binding
    if c["op"] == "attn":
        if "plan" not in s:
            s["plan"] = binding.AttnProblem(q=s["q"], scale=s["scale"], k=s["k"], v=s["v"], lens=s["lens"],
                                            pk=s["pk"], pv=s["pv"], prefix_len=s["prefix_len"], ids=s["ids"])
            n = binding.attn_shared_workspace_size(s["plan"], mass=s["mass"] is not None)
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=s["q"].device)
        binding.attn_shared(s["plan"], s["out"], s["lse"], s["mass"], s["ws"])
        return {"out": s["out"], "lse": s["lse"], "mass": s["mass"]}
    if "plan" not in s:
        s["plan"] = binding.EvictProblem(mass=s["mass"], lens=s["lens"], n_keep=c["keep"], n_first=c["first"],
                                         n_last=c["last"], pos=s["pos"], cur=s["cur"],
                                         planes=[s[k] for k in ("k", "v", "ik") if k in s])
    binding.cache_evict(s["plan"], s["out_src"], s["out_len"], s["out_pos"], s["out_mass"])
    return _evict_out(s)


# ------------------------------------------------- the definition, 64 bits --
def exact(c, seed):
    s = prepare(c, seed)
    return _exact_attn(c, s) if c["op"] == "attn" else _exact_evict(c, s)


def _exact_attn(c, s):
    B, T, Hq, Hkv, D, P, S, W = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "P", "S", "W"))
    G = Hq // Hkv
    dev = s["q"].device
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=dev)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device=dev)
    mass = None if s["mass"] is None else s["mass"].double()
    if P:
        pk, pv = s["pk"].double().permute(1, 0, 2).contiguous(), s["pv"].double().permute(1, 0, 2).contiguous()
    lens = s["lens"].tolist()
    pls = [P] * B if s["prefix_len"] is None else s["prefix_len"].tolist()
    for b in range(B):
        if not W:
            kb, vb = (s[x][b, : lens[b]].double().permute(1, 0, 2) for x in ("k", "v"))  # [Hkv, n, D]
        for t in range(T):
            n = max(0, lens[b] - T + t + 1)
            qt = s["q"][b, t].double().view(Hkv, G, D)
            if W:
                ids = s["ids"][b, t].long().view(-1, W)
                if ids.shape[0] == 1:  # one list for all heads: its listed slots only
                    one = ids[0][(ids[0] >= 0) & (ids[0] < n)]
                    see = torch.ones((Hkv, one.numel()), dtype=torch.bool, device=dev)
                    slots = one.expand(Hkv, -1)
                else:
                    see = (ids >= 0) & (ids < n)
                    slots = torch.where(see, ids, 0)
                h = torch.arange(Hkv, device=dev).view(Hkv, 1)
                kt, vt = s["k"][b][slots, h].double(), s["v"][b][slots, h].double()
            else:
                kt, vt = kb[:, :n], vb[:, :n]
            z = s["scale"] * (qt @ kt.transpose(1, 2))  # [Hkv, G, n]
            if W:
                z = z.masked_fill(~see.unsqueeze(1), -math.inf)
            m = z.shape[-1]
            if pls[b]:
                z = torch.cat([z, s["scale"] * (qt @ pk[:, : pls[b]].transpose(1, 2))], -1)
                vt = torch.cat([vt, pv[:, : pls[b]]], 1)
            if z.shape[-1] == 0:
                continue
            l = torch.logsumexp(z, -1)
            p = torch.exp(z - l.unsqueeze(-1)).nan_to_num(0.0)
            lse[b, t] = l.view(Hq)
            out[b, t] = (p @ vt).view(Hq, D)
            if mass is not None:
                w = p[..., :m].sum(1)  # [Hkv, m]
                for h in range(Hkv):
                    row = mass[b, h if c["mass"] == "head" else 0]
                    if W:
                        row.index_add_(0, slots[h], w[h])
                    else:
                        row[:m] += w[h]
    return {"out": out, "lse": lse, "mass": mass}


def _exact_evict(c, s):
    """Which values stay where, by each row's own ranking; moved values keep their bits."""
    B, Hm, Hkv, keep = (c[k] for k in ("B", "Hm", "Hkv", "keep"))
    if B * Hm > 512:
        return None
    out_mass = torch.zeros((B, Hm, keep), dtype=torch.float64, device=s["mass"].device)
    k, v = s["k"].clone(), s["v"].clone()
    ik = s["ik"].clone() if c["ikeys"] else None
    for b in range(B):
        for h in range(Hm):
            n = int(s["lens"][b, h])
            pos, m = s["pos"][b, h, :n], s["mass"][b, h, :n].double()
            guard = (pos < c["first"]) | (pos >= int(s["cur"][b]) - c["last"])
            free = (~guard).nonzero().squeeze(1)
            room = max(0, min(n, keep) - int(guard.sum()))
            best = free[torch.argsort(m[free], descending=True, stable=True)[:room]]
            stay = guard.clone()
            stay[best] = True
            idx = torch.arange(min(n, keep), device=m.device)
            holes = (~stay[: idx.numel()]).nonzero().squeeze(1)
            late = stay.nonzero().squeeze(1)
            late = late[late >= idx.numel()][: holes.numel()]
            idx[holes] = late
            out_mass[b, h, : idx.numel()] = m[idx]
            for g in range(Hkv) if Hm == 1 else (h,):
                k[b, holes, g] = s["k"][b, late, g]
                v[b, holes, g] = s["v"][b, late, g]
            if ik is not None:
                ik[b, holes] = s["ik"][b, late]
    got = {"out_src": None, "out_len": None, "out_pos": None, "out_mass": out_mass, "k": k, "v": v}
    if ik is not None:
        got["ik"] = ik
    return got


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(6)]:
        w = work(case)
        print(case, "%.3g GB %.3g GFLOP" % (w["bytes"] / 1e9, w["flops"] / 1e9))
