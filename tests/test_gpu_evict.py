"""cache_evict against the oracle: everything it returns is a choice or a copy,
so all of it is compared exactly."""
import numpy as np
import pytest
import torch

from oracle import attention as oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sparse_attention_indexer_idx_gb300 import binding
    binding.lib()
    return binding


def case(seed, Bn=2, M=2, S=100, keep=40, first=0, last=0, lens=None, pos=True, kind="heavy"):
    g = torch.Generator().manual_seed(seed)
    mass = torch.randn((Bn, M, S), generator=g).mul(1.5).exp()
    if kind == "ties":
        mass = torch.randint(0, 3, (Bn, M, S), generator=g).float()
    elif kind == "zeros":
        mass = torch.zeros(Bn, M, S)
        mass[..., ::2] = -0.0
    elif kind == "odd":
        mass[torch.rand(mass.shape, generator=g) < 0.2] = float("nan")
        mass[torch.rand(mass.shape, generator=g) < 0.1] = float("inf")
        mass[torch.rand(mass.shape, generator=g) < 0.1] = -float("inf")
        mass[torch.rand(mass.shape, generator=g) < 0.2] *= -1
    elif kind == "near":  # keys that agree in their upper digits
        mass = 1.0 + torch.randint(0, 900, (Bn, M, S), generator=g).float() * 2.0 ** -23
    if lens is None:
        lens = torch.randint(0, S + 1, (Bn, M), generator=g)
    lens = torch.as_tensor(lens, dtype=torch.int32).expand(Bn, M).contiguous()
    p = torch.stack([torch.randperm(2 * S, generator=g)[:S] for _ in range(Bn * M)]).view(Bn, M, S).to(torch.int32)
    return dict(mass=mass, lens=lens, n_keep=keep, n_first=first, n_last=last, pos=p if pos else None,
                cur=torch.full((Bn,), 2 * S, dtype=torch.int32) if pos else None)


def reference(c):
    num = lambda x: None if x is None else x.numpy()  # noqa: E731
    return oracle.cache_evict(num(c["mass"]), num(c["lens"]), c["n_keep"], c["n_first"], c["n_last"], num(c["pos"]),
                              num(c["cur"]))


def same(got, want):
    return np.array_equal(got.cpu().numpy(), want, equal_nan=want.dtype.kind == "f")


CASES = [
    dict(S=1, keep=1, lens=1), dict(S=5, keep=9), dict(S=2, keep=1, lens=2), dict(S=33, keep=32, lens=33),
    dict(S=100, keep=40, first=3, last=10), dict(S=100, keep=40, pos=False, first=3, last=10),
    dict(S=100, keep=40, kind="ties", lens=100), dict(S=1000, keep=333, kind="zeros", lens=1000),
    dict(S=1000, keep=333, kind="odd", lens=999), dict(S=5000, keep=2048, kind="near", lens=5000),
    dict(S=5000, keep=4999, lens=5000, last=1000), dict(S=4097, keep=1, lens=4097, kind="ties"),
    dict(Bn=1, M=1, S=20001, keep=7001, first=4, last=501, lens=20001),
    dict(Bn=1, M=1, S=70000, keep=69000, lens=70000, kind="ties"),
    dict(Bn=3, M=1, S=120000, keep=30000, lens=[[120000], [29999], [64001]], last=1000),
    dict(Bn=64, M=8, S=600, keep=512, last=64), dict(Bn=2, M=2, S=64, keep=30, lens=[[0, 1], [30, 31]]),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_oracle(B, i):
    c = case(40 + i, **CASES[i])
    Bn, M, S = c["mass"].shape
    want = reference(c)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    g = torch.Generator().manual_seed(i)
    heads = M if M > 1 else 3
    k = torch.randint(0, 2 ** 31, (Bn, S, heads, 5), generator=g, dtype=torch.int32)          # 20-byte rows
    v = torch.randint(0, 2 ** 31, (Bn, heads, S, 8), generator=g, dtype=torch.int32).transpose(1, 2)
    planes = [k.cuda(), v.cuda()]
    flat = None
    if M == 1:
        flat = torch.randint(0, 255, (Bn, S, 7), generator=g, dtype=torch.uint8)              # odd bytes, one head
        planes.append(flat.cuda())
    assert B.device_error() == 0
    K = c["n_keep"]
    src = torch.full((Bn, M, K), 77, dtype=torch.int32, device="cuda")
    ln = torch.full((Bn, M), 77, dtype=torch.int32, device="cuda")
    po, ms = torch.full_like(src, 77), torch.full((Bn, M, K), 77.0, device="cuda")
    p = B.EvictProblem(planes=planes, **d)
    for _ in range(2):  # the same call again leaves the same result
        B.cache_evict(p, src, ln, po, ms)
        torch.cuda.synchronize()
        assert same(src, want[0]) and same(ln, want[1]) and same(po, want[2]) and same(ms, want[3])
        for plane, orig in zip(planes, (k, v, flat)):
            o = orig.numpy()
            e = o.copy()
            for b in range(Bn):
                for h in range(o.shape[2] if o.ndim == 4 else 1):
                    m = 0 if M == 1 else h
                    n = want[1][b, m]
                    at = (b, slice(0, n), h) if o.ndim == 4 else (b, slice(0, n))
                    e[at] = o[b, want[0][b, m, :n], h] if o.ndim == 4 else o[b, want[0][b, m, :n]]
            assert np.array_equal(plane.cpu().numpy(), e)
    assert B.device_error() == 0


def test_in_place_outputs(B):
    c = case(90, Bn=3, M=2, S=300, keep=128, lens=[[300, 128], [0, 129], [64, 290]], last=20)
    want = reference(c)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    src = torch.empty((3, 2, 128), dtype=torch.int32, device="cuda")
    before = d["mass"].clone()
    B.cache_evict(B.EvictProblem(**d), src, d["lens"], d["pos"], d["mass"])
    assert same(src, want[0]) and same(d["lens"], want[1])
    assert same(d["pos"][..., :128], want[2]) and same(d["mass"][..., :128], want[3])
    for b in range(3):
        for m in range(2):
            n = int(c["lens"][b, m])
            assert (d["mass"][b, m, min(n, 128):n] == 0).all() and (d["pos"][b, m, min(n, 128):n] == -1).all()
            assert torch.equal(d["mass"][b, m, max(n, 128):], before[b, m, max(n, 128):])


def test_bad_lengths_are_empty_rows(B):
    c = case(91, Bn=1, M=3, S=50, keep=20, lens=[[51, -2, 50]])
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    src = torch.empty((1, 3, 20), dtype=torch.int32, device="cuda")
    ln = torch.empty((1, 3), dtype=torch.int32, device="cuda")
    assert B.device_error() == 0
    B.cache_evict(B.EvictProblem(**d), src, ln)
    assert B.device_error() == B.DEVERR_BAD_ROW
    c["lens"] = torch.tensor([[0, 0, 50]], dtype=torch.int32)
    want = reference(c)
    assert same(src, want[0]) and same(ln, want[1])


def test_refusals(B):
    m = torch.zeros((1, 2, 8), device="cuda")
    ln = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    src = torch.zeros((1, 2, 4), dtype=torch.int32, device="cuda")
    plane = torch.zeros((1, 8, 2, 4), device="cuda")
    for kw in (dict(n_keep=0), dict(n_keep=4, n_first=3, n_last=2), dict(n_keep=4, n_first=-1)):
        with pytest.raises((B.IdxError, ValueError)):
            B.cache_evict(B.EvictProblem(m, ln, **kw), src[..., : kw["n_keep"]].contiguous())
    for bad in (plane[:, :, :1], plane[:, :7], plane.transpose(2, 3)):
        with pytest.raises(ValueError):
            B.cache_evict(B.EvictProblem(m, ln, 4, planes=(bad,)), src)
    with pytest.raises(ValueError):
        B.cache_evict(B.EvictProblem(m, ln, 4), src[..., :3].contiguous())
    with pytest.raises(B.IdxError):  # in place, but with another row stride
        B.cache_evict(B.EvictProblem(m, ln, 4), src, out_mass=m.view(-1)[:8].view(1, 2, 4))
