"""attn_paged under many tokens of a request at once, a prompt's queries among them:
up to 2^20 rows of a request.  Against 64-bit torch, a request at a time."""
import pytest
import torch

from test_gpu_attn_paged import B, make, run  # noqa: F401  (B is a fixture)
from test_gpu_attn_paged_tc import check

pytestmark = pytest.mark.gpu

CASES = [
    dict(B=2, T=129, Hq=8, n_kv=2, S=1000, lens=[1000, 129], page=16),
    dict(B=3, T=512, Hq=4, n_kv=4, S=700, lens=[512, 700, 3], page=64),                     # tokens before the cache's start
    dict(B=1, T=2000, Hq=16, n_kv=2, S=2000, lens=[2000], page=48, dtype="f16"),
    dict(B=2, T=1001, Hq=6, n_kv=2, D=64, S=3001, lens=[3001, 1001], page=128),
    dict(B=1, T=4096, Hq=8, n_kv=1, S=5000, lens=[5000], page=16),
    dict(B=1, T=700, Hq=8, n_kv=2, S=900, lens=[900], page=7),                             # row by row
    dict(B=2, T=300, Hq=12, n_kv=2, D=64, S=400, lens=[400, 0], page=1, dtype="f16"),
    dict(B=1, T=32768, Hq=32, n_kv=1, D=64, S=300, lens=[300], page=16),                    # 2^20 rows, most see nothing
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_64_bits(B, case):  # noqa: F811
    t = make(500 + case, **CASES[case])
    assert B.device_error() == 0
    out, lse, p, ws = run(B, t)
    torch.cuda.synchronize()
    assert B.device_error() == 0
    # a stretch of tokens at a time: the scores of all would not fit
    T, step = t["q"].shape[1], 1024
    for t0 in range(0, T, step):
        n = min(step, T - t0)
        part = dict(t, q=t["q"][:, t0: t0 + n], lens=[max(0, x - (T - t0 - n)) for x in t["lens"]])
        check(part, out[:, t0: t0 + n], lse[:, t0: t0 + n])
    again = torch.empty_like(out)
    B.attn_paged(p, again, None, ws)
    assert torch.equal(out, again)
