"""Scores that are no numbers show: a row that sees a key whose score is NaN (or
+inf) gets NaN in out, in lse and in the masses of the slots that it sees, as by
the formula; rows that do not see it keep their bits.  A score of -inf is a
weight of zero."""
import pytest
import torch

from test_gpu_attn import B, make, run  # noqa: F401  (B is a fixture)

pytestmark = pytest.mark.gpu


def _seen(t, b, tok, h):
    """Private slots that row (b, tok) of KV head h sees."""
    S = t["k"].shape[1]
    n = t["lens"][b] if t["lens"].dim() == 1 else t["lens"][b, h if t["lens"].shape[1] > 1 else 0]
    n = max(0, int(n) - t["q"].shape[1] + tok + 1)
    see = torch.arange(S) < n
    if "ids" in t:
        ids = t["ids"][b, tok] if t["ids"].dim() == 3 else t["ids"][b, tok, h]
        listed = torch.zeros(S, dtype=torch.bool)
        listed[ids[(ids >= 0) & (ids < n)].long()] = True
        see &= listed
    return see


def _compare(B, t, bad, hit):  # noqa: F811
    """t clean, bad with a value planted; hit(b, t, hq): whether that row meets it."""
    want = [None if x is None else x.clone() for x in run(B, t)[:3]]
    out, lse, mass, _, _ = run(B, bad)
    torch.cuda.synchronize()
    assert B.device_error() == 0
    Bn, T, Hq, _ = t["q"].shape
    rows = torch.tensor([[[bool(hit(b, i, h)) for h in range(Hq)] for i in range(T)] for b in range(Bn)]).cuda()
    assert rows.any()
    assert torch.isnan(out[rows].float()).all() and torch.isnan(lse[rows]).all()
    assert torch.equal(out[~rows], want[0][~rows]) and torch.equal(lse[~rows], want[1][~rows])
    if mass is None:
        return
    G = Hq // (t["k"].shape[2])
    none = torch.zeros_like(t["mass"], dtype=torch.bool)
    for b, i, h in rows.nonzero().tolist():
        none[b, h // G if t["mass"].shape[1] > 1 else 0] |= _seen(t, b, i, h // G)
    none = none.cuda()
    assert torch.isnan(mass[none]).all()
    assert torch.equal(mass[~none], want[2][~none])


def _planted(t, name, at, x=float("nan")):
    bad = dict(t)
    bad[name] = t[name].clone()
    bad[name][at] = x
    return bad


@pytest.mark.parametrize("kw", [
    dict(T=3, Hq=8, n_kv=2, S=100, lens=[100, 50], mass=2),
    dict(T=3, Hq=8, n_kv=2, S=100, lens=[100, 50], mass=1, D=64, dtype="f16", P=20),
    dict(T=3, Hq=64, n_kv=2, S=100, lens=[100, 50], mass=1),                       # several row tiles
    dict(T=3, Hq=8, n_kv=2, S=100, lens=[100, 50], mass=2, W=100, ids_per_head=True),
    dict(T=3, Hq=8, n_kv=2, S=100, lens=[100, 50], mass=1, W=90, D=64),
    dict(T=1, Hq=64, n_kv=2, S=4000, lens=[100, 4000], mass=1, W=300, D=64),
])
def test_a_private_key(B, kw):  # noqa: F811
    t = make(500, B=2, **kw)
    T, Hq = t["q"].shape[1:3]
    slot = 99 if T > 1 else 40
    if "ids" in t:
        t["ids"][0][..., 3] = slot       # listed for every token of request 0
        rest = t["ids"][0].clone()
        rest[..., 3] = -1
        t["ids"][0] = torch.where(rest == slot, -1, t["ids"][0])
    G = Hq // 2
    _compare(B, t, _planted(t, "k", (0, slot, 1)), lambda b, i, h: b == 0 and h // G == 1 and _seen(t, 0, i, 1)[slot])


def test_a_query(B):  # noqa: F811
    t = make(501, B=2, T=2, Hq=8, n_kv=2, S=70, P=40, lens=[70, 69], mass=2)
    _compare(B, t, _planted(t, "q", (1, 0, 2, 5)), lambda b, i, h: (b, i, h) == (1, 0, 2))


@pytest.mark.parametrize("kw", [
    dict(T=3, mass=2), dict(T=3, mass=1), dict(T=3, mass=1, ids_per_head=True, D=64),
    dict(T=1, mass=1, per_head_lens=True, lens=[[100, 50], [31, 90]]),
])
def test_a_query_whose_list_names_slots_that_it_does_not_see(B, kw):  # noqa: F811
    # other rows see them: their masses get those rows' weights and nothing else
    t = make(506, **dict(dict(B=2, Hq=8, n_kv=2, S=100, W=100, lens=[100, 60]), **kw))
    _compare(B, t, _planted(t, "q", (0, 0, 5, 3)), lambda b, i, h: (b, i, h) == (0, 0, 5))


@pytest.mark.parametrize("kw", [
    dict(B=2, T=1, Hq=8, n_kv=2, S=30, P=200, prefix_len=[90, 200], lens=[30, 30], mass=1),
    dict(B=20, T=1, Hq=8, n_kv=2, S=5, P=300, prefix_len=[15 * i for i in range(1, 21)], mass=2),   # a line of its own
    dict(B=40, T=1, Hq=16, n_kv=2, S=9, P=9000, prefix_len=[225 * i for i in range(1, 41)], mass=2),  # tensor cores
    dict(B=20, T=1, Hq=8, n_kv=2, P=40000, D=64, dtype="f16", prefix_len=[2000 * i for i in range(1, 21)]),
    dict(B=1, T=1, Hq=4, n_kv=2, P=30011, S=50, mass=1, prefix_len=[30011]),                          # many pieces
])
def test_a_key_of_the_prefix(B, kw):  # noqa: F811
    t = make(502, **kw)
    at = t["pk"].shape[0] // 2 + 1
    G = t["q"].shape[2] // 2
    _compare(B, t, _planted(t, "pk", (at, 1)), lambda b, i, h: h // G == 1 and t["prefix_len"][b] > at)


def test_nothing_but_nan(B):  # noqa: F811
    t = make(503, B=2, T=1, Hq=8, n_kv=2, S=300, lens=[300, 1], mass=2)
    _compare(B, t, _planted(t, "k", (slice(None), slice(None), 0)), lambda b, i, h: h < 4)
    t = make(504, B=40, T=1, Hq=8, n_kv=2, P=9000)
    _compare(B, t, _planted(t, "pk", (slice(None), 1)), lambda b, i, h: h >= 4)


@pytest.mark.parametrize("T,S", [(1, 200), (3, 40000)])
def test_infinite_fp16_keys(B, T, S):  # noqa: F811
    # queries of +-1 in the dim whose key element leaves fp16's range: a score of
    # +inf is no number behind the softmax, one of -inf is a weight of zero
    t = make(505, B=1, T=T, Hq=8, n_kv=2, S=S, lens=[S], mass=2, D=64, dtype="f16")
    t["q"][..., 0] = torch.tensor([1.0, -1.0]).half().repeat(4)
    t["k"][0, 17, 1] = 0.0
    bad = _planted(t, "k", (0, 17, 1, 0), float("inf"))
    low = _planted(t, "k", (0, 17, 1, 0), 60000.0)       # a weight of zero under the queries of -1
    want, lse_want = run(B, low)[:2]
    out, lse, mass, _, _ = run(B, bad)
    assert torch.isnan(out[:, :, 4::2].float()).all() and torch.isnan(lse[:, :, 4::2]).all()
    for h in (0, 1, 2, 3, 5, 7):
        assert torch.equal(out[:, :, h], want[:, :, h]) and torch.equal(lse[:, :, h], lse_want[:, :, h])
    assert torch.isnan(mass[0, 1]).all() and torch.isfinite(mass[0, 0]).all()
