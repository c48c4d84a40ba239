"""attn_shared over selections that hold nothing: a list without entries (W = 0)
selects no slot, which is not the same as no list (every slot)."""
import numpy as np
import pytest
import torch

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
