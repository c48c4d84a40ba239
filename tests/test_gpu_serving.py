"""A decode step as it is used, step by step against the oracles: the indexer's
choice, its witnesses, attention behind a shared prefix, the masses, eviction of
every plane, and the steps after it, when slots and positions have parted."""
import numpy as np
import pytest
import torch

from helpers import EPS, check_topk_row
from oracle import attention as oa
from oracle import dsa as od
from oracle import witness as ow
from test_gpu_attn import B, DT  # noqa: F401  (B is a fixture)

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # rounding of a weight and of an output, see test_gpu_attn


def num(x):
    return x.float().cpu().numpy() if x.is_floating_point() else x.cpu().numpy()


def check_step(B, c, q, iq, iw, segments, dtype):  # noqa: F811
    """One step, against the oracles on the caches as they are."""
    requests, slots = c.index_k.shape[:2]
    lens = c.lens.view(-1)
    mass0 = num(c.mass)
    p = B.Problem(iq, iw, c.index_k.view(requests * slots, -1), lens, slots, c.key_off)
    learned = torch.empty_like(c.ids)
    ws = torch.empty(B.idx_topk_workspace_size(p, c.top_k), dtype=torch.uint8, device="cuda")
    B.idx_topk(p, c.top_k, learned, None, ws)
    out = c.step(q, iq, iw, segments)
    torch.cuda.synchronize()
    K, ln = c.top_k, num(lens).copy()
    for b in range(requests):
        s, a = od.indexer_score(num(iq[b]), num(iw[b]), num(c.index_k[b, :ln[b]]))
        check_topk_row(num(learned[b]), None, s, a, K, EPS["bf16"])
    ids = ow.apply_topology_witnesses(num(learned), K, ln, max(K - segments, 0), segments, segments)
    assert np.array_equal(num(c.ids), ids)
    prefix = () if c.prefix_k is None else (num(c.prefix_k), num(c.prefix_v))
    D = q.shape[-1]
    ref = oa.attn_shared(num(q), D ** -0.5, num(c.k), num(c.v), ln, *(prefix or (None, None)), ids=ids[:, None], mass=mass0)
    dx = D * 2.0 ** -23 * ref["absx"] + 2.0 ** -21
    tol = ref["absv"] * (2.2 * U[dtype] + 4 * dx[..., None]) + 1e-6
    if dtype == "f16":
        keys = K + (len(prefix[0]) if prefix else 0)
        tol = tol + keys * 2.0 ** -25 * np.abs(num(c.v)).max()
    assert (np.abs(num(out) - ref["out"]) <= tol).all()
    add = ref["mass"] - mass0
    mt = add * (4 * dx.max() + q.shape[2] * 2.0 ** -24) + 2.0 ** -22 * ref["mass"] + 1e-9
    assert (np.abs(num(c.mass) - ref["mass"]) <= mt).all()


def check_trim(c, n_keep, n_first, n_last):
    before = {n: num(getattr(c, n)).copy() for n in ("k", "v", "index_k", "mass", "pos", "lens", "cur")}
    held = torch.cuda.memory_allocated()
    moved = c.trim(n_keep, n_first, n_last)
    assert torch.cuda.memory_allocated() == held         # a trim takes no memory
    torch.cuda.synchronize()
    src, ln, pos, mass = oa.cache_evict(before["mass"], before["lens"], n_keep, n_first, n_last, before["pos"],
                                        before["cur"])
    assert np.array_equal(num(moved), src)
    assert np.array_equal(num(c.lens), ln) and np.array_equal(num(c.cur), before["cur"])
    assert np.array_equal(num(c.pos)[..., :n_keep], pos) and np.array_equal(num(c.mass)[..., :n_keep], mass)
    for n in ("k", "v", "index_k"):
        want, got = before[n].copy(), num(getattr(c, n))
        for b in range(len(want)):
            m = ln[b, 0]
            want[b, :m] = want[b, src[b, 0, :m]]
        assert np.array_equal(got, want)
    return src, before["lens"]


@pytest.mark.parametrize("dtype,prefix", [("bf16", 70), ("f16", 70), ("bf16", 0)])
def test_steps_and_trims(B, dtype, prefix):  # noqa: F811
    from sparse_attention_indexer_idx_gb300 import serving
    requests, slots, q_heads, kv_heads, dim, K, segments = 3, 300, 8, 2, 64, 96, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    rn = lambda *s, dt=DT[dtype]: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    bf = torch.bfloat16
    shared = (rn(prefix, kv_heads, dim), rn(prefix, kv_heads, dim)) if prefix else ()
    c = serving.DecodeCache(requests, slots, q_heads, kv_heads, dim, 128, K, *shared, dtype=DT[dtype])
    c.fill(rn(requests, 290, kv_heads, dim), rn(requests, 290, kv_heads, dim), rn(requests, 290, 128, dt=bf),
           lens=[290, 40, 203])

    def steps(n):
        for _ in range(n):
            c.append(rn(requests, kv_heads, dim), rn(requests, kv_heads, dim), rn(requests, 128, dt=bf))
            check_step(B, c, rn(requests, 1, q_heads, dim), rn(requests, 16, 128, dt=bf),
                       torch.rand((requests, 16), generator=g, device="cuda"), segments, dtype)

    steps(3)
    src, ln = check_trim(c, 200, 4, 25)
    assert (src[0, 0] != np.arange(200)).any()           # rows did move
    steps(3)                                             # slots are out of the order of their positions
    check_trim(c, 150, 4, 25)
    steps(1)
    assert c.cur.tolist() == [297, 47, 210]
    assert B.device_error() == 0
