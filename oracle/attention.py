"""Oracle of the decode-step attention (shared prefix, private caches, id
lists, running masses) and of the eviction by mass: numpy, 64 bits, one row at a
time, straight from the definitions."""
import numpy as np


def attn_shared(q, scale, k=None, v=None, lens=None, pk=None, pv=None, prefix_len=None, ids=None, mass=None):
    """q [B, T, Hq, D]; k, v [B, S, n_kv, D]; lens [B] or [B, n_kv]; pk, pv
    [P, n_kv, D]; prefix_len [B]; ids [B, T, W] or [B, T, n_kv, W]; mass
    [B, n_kv or 1, S].  Returns a dict: out, lse, mass (a new array) and, for
    error bounds, absv = sum p |v| and absx = scale sum |q||k| (largest over the
    row's keys)."""
    f = lambda x: None if x is None else np.asarray(x, dtype=np.float64)  # noqa: E731
    q, k, v, pk, pv = f(q), f(k), f(v), f(pk), f(pv)
    B, T, Hq, D = q.shape
    n_kv = (k if k is not None else pk).shape[-2]
    G = Hq // n_kv
    out = np.zeros((B, T, Hq, D))
    absv = np.zeros((B, T, Hq, D))
    lse = np.full((B, T, Hq), -np.inf)
    absx = np.zeros((B, T, Hq))
    new_mass = None if mass is None else np.array(mass, dtype=np.float64)
    for b in range(B):
        for t in range(T):
            for hq in range(Hq):
                h = hq // G
                keys, vals, slots = [], [], np.zeros(0, dtype=np.int64)
                if pk is not None:
                    n = pk.shape[0] if prefix_len is None else int(prefix_len[b])
                    keys.append(pk[:n, h])
                    vals.append(pv[:n, h])
                if k is not None:
                    ln = int(lens[b]) if np.ndim(lens) == 1 else int(lens[b][h if np.shape(lens)[1] > 1 else 0])
                    n = max(0, ln - T + t + 1)
                    if ids is None:
                        slots = np.arange(n)
                    else:
                        row = np.asarray(ids[b, t] if np.ndim(ids) == 3 else ids[b, t, h], dtype=np.int64)
                        slots = row[(row >= 0) & (row < n)]
                    keys.append(k[b, slots, h])
                    vals.append(v[b, slots, h])
                kk, vv = np.concatenate(keys), np.concatenate(vals)
                if len(kk) == 0:
                    continue
                x = scale * (kk @ q[b, t, hq])
                absx[b, t, hq] = abs(scale) * (np.abs(kk) @ np.abs(q[b, t, hq])).max()
                top = x.max()
                e = np.exp(x - top)
                lse[b, t, hq] = top + np.log(e.sum())
                p = e / e.sum()
                out[b, t, hq] = p @ vv
                absv[b, t, hq] = p @ np.abs(vv)
                if new_mass is not None and len(slots):
                    m = h if new_mass.shape[1] > 1 else 0
                    new_mass[b, m, slots] += p[len(p) - len(slots):]
    return {"out": out, "lse": lse, "mass": new_mass, "absv": absv, "absx": absx}


def cache_evict(mass, lens, n_keep, n_first=0, n_last=0, pos=None, cur=None):
    """mass, pos [B, M, S]; lens [B, M]; cur [B].  Returns (src [B, M, n_keep],
    new_len, new_pos, new_mass), padded with -1, -1 and 0."""
    B, M, S = mass.shape
    src = np.full((B, M, n_keep), -1, dtype=np.int32)
    new_len = np.zeros((B, M), dtype=np.int32)
    new_pos = np.full((B, M, n_keep), -1, dtype=np.int32)
    new_mass = np.zeros((B, M, n_keep), dtype=mass.dtype)
    for b in range(B):
        for m in range(M):
            n = int(lens[b, m])
            at = np.arange(n) if pos is None else pos[b, m, :n].astype(np.int64)
            end = n if cur is None else int(cur[b])
            rank = mass[b, m, :n].astype(np.float64)
            rank[np.isnan(rank)] = -np.inf
            rank[(at < n_first) | (at >= end - n_last)] = np.inf
            nk = min(n, n_keep)
            stay = np.zeros(n, dtype=bool)
            stay[np.lexsort((np.arange(n), -rank))[:nk]] = True
            late, holes = nk + np.flatnonzero(stay[nk:]), np.flatnonzero(~stay[:nk])
            row = np.arange(nk)
            row[holes] = late   # both ascending, and equally many
            src[b, m, :nk] = row
            new_len[b, m] = nk
            new_pos[b, m, :nk] = at[row]
            new_mass[b, m, :nk] = mass[b, m, row]
    return src, new_len, new_pos, new_mass
