"""attn_paged's weights in 16 bits: with fp16 the small ones, which together can be
most of a row, keep their bits.  One dim of the queries and keys counts, so that
scores are exact; rows of every kernel, with boxes, single rows and lists.

Bounds: a weight and the output are rounded to the type (u), and 2^-17 stands for the
score's scale, the exponential and the sums.  fp16 weights are multiples of 2^-36 of
their row's largest at worst (2^-25 under references that leave them up to 2^11), the
output of 2^-24."""
import math

import pytest
import torch

from test_gpu_attn_paged import B, make, run  # noqa: F401  (B is a fixture)

pytestmark = pytest.mark.gpu

# what each case runs: clusters, streams of boxes, the tensor cores, rows one by one, lists
KINDS = {
    "clusters": dict(B=2, T=1, Hq=8, n_kv=2, S=6000, page=16),
    "clusters of 32 rows of 64": dict(B=2, T=4, Hq=32, n_kv=4, D=64, S=3001, page=64),
    "streams": dict(B=2, T=1, Hq=32, n_kv=4, S=40000, page=16),
    "streams of 64": dict(B=3, T=1, Hq=16, n_kv=8, D=64, S=30011, page=32),
    "tensor cores": dict(B=2, T=8, Hq=16, n_kv=2, S=30000, page=64),
    "tensor cores, 64": dict(B=2, T=40, Hq=4, n_kv=1, D=64, S=29999, page=128),
    "rows": dict(B=2, T=1, Hq=8, n_kv=2, S=5000, page=3),
    "long rows": dict(B=3, T=1, Hq=32, n_kv=8, S=20000, page=5),
    "lists": dict(B=2, T=1, Hq=8, n_kv=2, S=5000, W=4096),
    "long lists": dict(B=24, T=2, Hq=32, n_kv=4, S=4096, W=4000),
}


def exact_rows(kind, dtype, score, values, scale=math.log(2)):
    """A call whose slot s has the score `score(s)` (in units of the scale) and values of
    `values(s)` in every row; and what each row has to be."""
    kw = KINDS[kind]
    n, W = kw["S"], kw.get("W", 0)
    t = make(7, dtype=dtype, lens=[n] * kw["B"], **kw)
    t["scale"] = scale
    t["q"] = torch.zeros_like(t["q"])
    t["q"][..., 0] = 1
    s = torch.arange(n, device="cuda")
    x, v = score(s), values(s)
    for b in range(kw["B"]):
        pg, at = t["table"][b].long()[s // t["page"]], s % t["page"]
        t["k"][pg, at] = 0
        t["k"][pg, at, :, 0] = x.to(t["k"].dtype).unsqueeze(1)
        t["v"][pg, at] = v.to(t["v"].dtype).view(-1, 1, 1)
    see = torch.ones(kw["B"], kw["T"], n, dtype=torch.bool, device="cuda")
    if W:
        t["ids"] = torch.arange(W, dtype=torch.int32, device="cuda").expand(kw["B"], kw["T"], W).contiguous()
        see[..., W:] = False
    see &= s < torch.arange(n - kw["T"] + 1, n + 1, device="cuda").view(1, -1, 1)
    y = torch.where(see, x.double() * scale, -math.inf)
    lse = torch.logsumexp(y, -1)
    w = torch.softmax(y, -1)             # (of differences: a steep row's lse has no bits left for its count)
    return t, (w @ v.double()).unsqueeze(-1), (w @ v.abs().double()).unsqueeze(-1), lse.unsqueeze(-1), int(see.sum(-1).max())


@pytest.mark.parametrize("dtype,low", [("f16", 27), ("f16", 24), ("f16", 21), ("f16", 15), ("bf16", 27)])
@pytest.mark.parametrize("kind", KINDS)
def test_many_small_weights(B, kind, dtype, low):  # noqa: F811
    """Every 500th slot has the largest score and nothing to give; the others have all."""
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    t, want, absv, lse, n = exact_rows(kind, dtype, lambda s: torch.where(s % 500 == 3, 0.0, -low - (s % 4) / 4),
                                       lambda s: torch.where(s % 500 == 3, 0.0, 1.0 + (s % 8) / 8))
    scale = 2.0 ** min(10, low - 12)                     # outputs of fp16's normal range
    t["v"].mul_(scale)
    want, absv = want * scale, absv * scale
    out, l, _, _ = run(B, t)
    tol = absv * (2.2 * u + 2.0 ** -17) + (2.0 ** -24 + n * 2.0 ** -36 * 2 * scale if dtype == "f16" else 0)
    want, tol = (x.unsqueeze(-1).expand(out.shape) for x in (want, tol))
    err = (out.double() - want).abs()
    assert (err <= tol).all(), (err / tol).max().item()
    assert ((l.double() - lse).abs() <= 2.0 ** -20 * (1 + lse.abs())).all()
    assert B.device_error() == 0


@pytest.mark.parametrize("dtype,steep", [("bf16", 2), ("bf16", 19), ("bf16", 24), ("bf16", 31), ("bf16", 40), ("bf16", 90),
                                         ("f16", 19), ("f16", 20), ("f16", 24), ("f16", 28), ("f16", 40)])
@pytest.mark.parametrize("kind", KINDS)
def test_steep_scores_keep_to_the_largest(B, kind, dtype, steep):  # noqa: F811
    """Scores of 2^steep and more, as far apart, of either sign and rising along the
    cache: a row is the average of the slots that share its largest one."""
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    scores = {
        "above zero": lambda s: 3 - (s * 7 % 9) / 4,
        "below zero": lambda s: -2 - (s * 5 % 7) / 8,
        "rising": lambda s: 1 + s.float().mul(60 / len(s)).floor() / 4 - 8,
    }
    for name, score in scores.items():
        t, want, absv, lse, n = exact_rows(kind, dtype, lambda s: score(s).float(), lambda s: 1.0 + (s % 8) / 8,
                                           scale=2.0 ** steep)
        out, l, _, _ = run(B, t)
        # (scores are off by 2^-23 of themselves at most, equal ones alike)
        near = 2.0 ** steep * 16 * 2.0 ** -23 if steep < 10 else 0
        want, tol = (x.unsqueeze(-1).expand(out.shape) for x in (want, absv * (2.2 * u + 2.0 ** -17 + near)))
        err = (out.double() - want).abs()
        assert (err <= tol).all(), (name, (err / tol).max().item())
        assert ((l.double() - lse).abs() <= 2.0 ** -20 * (1 + lse.abs())).all(), name
    assert B.device_error() == 0
