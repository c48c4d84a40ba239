"""attn_shared over selections: a list without entries (W = 0) selects no slot,
which is not the same as no list (every slot); the positions of selected blocks
are lists too."""
import numpy as np
import pytest
import torch

from oracle import block_select as ob
from test_gpu_attn import B, check, make, run  # noqa: F401  (B is a fixture)

pytestmark = pytest.mark.gpu


def _empty(t, per_head):
    b, T = t["q"].shape[:2]
    t["ids"] = torch.zeros((b, T, t["k"].shape[2], 0) if per_head else (b, T, 0), dtype=torch.int32)
    return t


EMPTY = [
    dict(B=2, T=1, Hq=8, n_kv=2, S=100, lens=[100, 7], mass=2),
    dict(B=2, T=3, Hq=8, n_kv=4, S=65, mass=1, D=64, dtype="f16"),
    dict(B=3, T=1, Hq=8, n_kv=2, S=40, P=33, mass=1, prefix_len=[0, 1, 33]),
    dict(B=40, T=1, Hq=16, n_kv=2, S=9, P=9000, mass=2),            # the prefix on the tensor cores
]


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("case", range(len(EMPTY)))
def test_an_empty_selection_selects_nothing(B, case, per_head):  # noqa: F811
    t = _empty(make(400 + case, **EMPTY[case]), per_head)
    assert B.device_error() == 0
    out, lse, mass, p, ws = run(B, t)
    torch.cuda.synchronize()
    assert B.device_error() == 0
    assert torch.equal(mass.cpu(), t["mass"])
    if "pk" not in t:
        assert (out == 0).all() and torch.isneginf(lse).all()
    few = [0, len(out) // 2, len(out) - 1]
    sub = dict(t, **{n: t[n][few] for n in ("q", "k", "v", "lens", "mass", "ids", "prefix_len") if n in t})
    check(sub, out[few], lse[few], mass[few])


def test_a_list_of_paddings_and_a_list_that_is_a_slice(B):  # noqa: F811
    t = make(410, B=2, T=1, Hq=8, n_kv=2, S=50, lens=[50, 20], mass=1)
    for ids in (torch.full((2, 1, 5), -1, dtype=torch.int32), torch.zeros((2, 1, 5), dtype=torch.int32)[..., :0]):
        t["ids"] = ids
        out, lse, mass, _, _ = run(B, t)
        assert (out == 0).all() and np.isneginf(lse.cpu().numpy()).all()
        assert torch.equal(mass.cpu(), t["mass"])


@pytest.mark.parametrize("per_head", [False, True])
def test_an_empty_selection_of_an_empty_cache(B, per_head):  # noqa: F811
    t = make(411, B=2, T=1, Hq=8, n_kv=2, P=50)
    d = {n: t[n].cuda() for n in ("q", "pk", "pv")}
    none = torch.empty((2, 0, 2, 128), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty((2, 1, 2, 0) if per_head else (2, 1, 0), dtype=torch.int32, device="cuda")
    p = B.AttnProblem(d["q"], t["scale"], none, none, torch.zeros(2, dtype=torch.int32, device="cuda"), d["pk"], d["pv"],
                      ids=ids)
    out, lse = torch.empty_like(d["q"]), torch.empty((2, 1, 8), device="cuda")
    ws = torch.empty(B.attn_shared_workspace_size(p, False), dtype=torch.uint8, device="cuda")
    B.attn_shared(p, out, lse, None, ws)
    check(t, out, lse, None)


@pytest.mark.parametrize("T,L,P,dtype", [(1, 1000, 0, "bf16"), (3, 1500, 200, "f16"), (4, 517, 0, "bf16")])
def test_positions_of_selected_blocks(B, T, L, P, dtype):  # noqa: F811
    """From block scores to attention: each token's and KV head's blocks, the
    positions that they cover, and attention over these."""
    n_kv, bs, top = 4, 64, 3
    t = make(420 + T, B=1, T=T, Hq=16, n_kv=n_kv, S=L, P=P, D=128, lens=[L], mass=n_kv, dtype=dtype)
    g = torch.Generator().manual_seed(421)
    index_q, index_k = torch.randn(T, n_kv, 128, generator=g), torch.randn(L, 128, generator=g)
    pos = torch.arange(L - T, L, dtype=torch.int32)
    cfg = B.block_sparse_config(bs, top, 1, 1)
    dev = {"device": "cuda", "dtype": torch.int32}
    blocks, counts = torch.empty((T, n_kv, top), **dev), torch.empty((T, n_kv), **dev)
    ws = torch.empty(B.block_select_workspace_size(T, n_kv, L, cfg), dtype=torch.uint8, device="cuda")
    B.block_select(index_q.cuda(), index_k.cuda(), pos.cuda(), cfg, blocks, counts, ws)
    ids = torch.empty((T, n_kv, top * bs), **dev)
    B.block_positions(blocks, counts, pos.cuda(), L, bs, ids, None)
    t["ids"] = ids.cpu().view(1, T, n_kv, top * bs)
    chosen, cover = blocks.cpu().numpy(), t["ids"].numpy()[0]
    for i in range(T):
        for h in range(n_kv):
            want = ob.positions_of_blocks([b for b in chosen[i, h] if b >= 0], int(pos[i]), L, bs)
            assert [x for x in cover[i, h] if x >= 0] == want
    assert (t["ids"] == -1).any()          # the last block ends inside the cache
    out, lse, mass, _, _ = run(B, t)
    torch.cuda.synchronize()
    check(t, out, lse, mass)
    assert B.device_error() == 0


@pytest.mark.parametrize("kw", [
    dict(T=1, mass=1), dict(T=3, mass=2, D=64), dict(T=2, mass=1, ids_per_head=True, dtype="f16"),
    dict(T=1, Hq=64, mass=1, P=30),
])
def test_lists_under_lengths_of_each_kv_head(B, kw):  # noqa: F811
    a = dict(dict(B=3, Hq=8, n_kv=2, S=120, W=90, lens=[[120, 3], [0, 77], [1, 119]], per_head_lens=True), **kw)
    t = make(430, **a)
    out, lse, mass, _, _ = run(B, t)
    torch.cuda.synchronize()
    assert B.device_error() == 0
    check(t, out, lse, mass)
