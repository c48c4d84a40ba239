"""cache_evict where a block has a long slice: many rows of one block each with
more than 8,192 slots, slices whose words of 32 slots take a thread more than
one round (above 32,768), and the longest rows that it takes.  All exact."""
import numpy as np
import pytest
import torch

from test_gpu_evict import B, case, reference, same  # noqa: F401  (B is a fixture)

pytestmark = pytest.mark.gpu

CASES = [
    # a block for each row (there are more rows than SMs)
    dict(Bn=20, M=8, S=9001, keep=4500, first=4, last=300),
    dict(Bn=20, M=8, S=12000, keep=11990, lens=12000, kind="ties"),
    dict(Bn=20, M=8, S=8193, keep=17, lens=8193, kind="near"),
    dict(Bn=160, M=1, S=9999, keep=5000, kind="odd", pos=False, last=100),
    dict(Bn=20, M=8, S=33000, keep=16000, lens=33000, last=500),        # two rounds of words
    dict(Bn=20, M=8, S=49152, keep=40000, kind="ties", lens=49152),     # the longest slice of one block
    # a row over eight blocks: keep below and above one block's slice
    dict(Bn=1, M=1, S=300001, keep=20000, lens=300001, first=4, last=1000),
    dict(Bn=1, M=1, S=300001, keep=150000, lens=300001, kind="ties"),
    dict(Bn=1, M=1, S=393216, keep=49000, lens=393216, kind="ties"),
    dict(Bn=1, M=1, S=393216, keep=393215, lens=393216, last=100000),
    dict(Bn=2, M=1, S=393216, keep=200000, lens=[[393216], [199999]], kind="near"),
    dict(Bn=1, M=1, S=393216, keep=300000, lens=393216, kind="zeros"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_long_slices(B, i):  # noqa: F811
    c = case(140 + i, **CASES[i])
    Bn, M, S = c["mass"].shape
    want = reference(c)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    K = c["n_keep"]
    plane = torch.arange(Bn * S * M, dtype=torch.int32).view(Bn, S, M, 1)     # each row says where it was
    moved = plane.cuda()
    src = torch.full((Bn, M, K), 77, dtype=torch.int32, device="cuda")
    ln = torch.full((Bn, M), 77, dtype=torch.int32, device="cuda")
    po, ms = torch.full_like(src, 77), torch.full((Bn, M, K), 77.0, device="cuda")
    assert B.device_error() == 0
    p = B.EvictProblem(planes=(moved,), **d)
    B.cache_evict(p, src, ln, po, ms)
    torch.cuda.synchronize()
    assert B.device_error() == 0
    assert same(src, want[0]) and same(ln, want[1]) and same(po, want[2]) and same(ms, want[3])
    e = plane.numpy().copy()
    for b in range(Bn):
        for m in range(M):
            n = want[1][b, m]
            e[b, :n, m] = plane.numpy()[b, want[0][b, m, :n], m]
    assert np.array_equal(moved.cpu().numpy(), e)
    # in place: positions and masses over themselves, the freed slots cleared
    B.cache_evict(B.EvictProblem(**d), src, None, d["pos"], d["mass"])
    assert same(src, want[0]) and same(d["mass"][..., :K], want[3])
    if d["pos"] is not None:
        assert same(d["pos"][..., :K], want[2])
    for b in range(Bn):
        n = int(c["lens"][b, 0])
        assert (d["mass"][b, 0, min(n, K):n] == 0).all()
