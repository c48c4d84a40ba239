"""Waits of attn_paged's kernels that do give up.  With a limit of 0 a wait gives up
where the phase is not there at the hardware's first look, which itself lasts a
while: with keys and values in L2 every tile may land in it, so L2 is emptied before
each call and calls are made until one reports a timeout (nine of ten did).  Clusters
under 32 rows are left out: next to none of theirs did."""
import pytest
import torch

from test_gpu_attn_paged import B, make, run  # noqa: F401  (B is a fixture)
from test_gpu_attn_paged_tc import check

pytestmark = pytest.mark.gpu

CALLS = 100
KINDS = {
    "tensor cores": dict(B=3, T=4, Hq=32, n_kv=4, S=24000, lens=[24000, 9000, 5], page=64),
    "tensor cores, 64": dict(B=2, T=12, Hq=32, n_kv=4, D=64, S=40000, lens=[40000, 31111], page=128, dtype="f16"),
    "streams": dict(B=2, T=1, Hq=32, n_kv=4, S=40000, page=16, lens=[40000] * 2),
    "streams of 64": dict(B=2, T=1, Hq=32, n_kv=4, D=64, S=80000, page=16, lens=[80000] * 2),
    "streams under 32 rows of 64": dict(B=3, T=4, Hq=32, n_kv=4, D=64, S=60000, page=64, lens=[60000] * 3),
    "clusters": dict(B=8, T=1, Hq=32, n_kv=8, S=3000, page=16, lens=[3000] * 8),
}


@pytest.mark.parametrize("kind", KINDS)
def test_a_wait_gives_up_and_later_calls_are_right(B, kind):  # noqa: F811
    t = make(61, **KINDS[kind])
    first, lse, _, ws = run(B, t)
    torch.cuda.synchronize()
    assert (ws.numel() == 0) == kind.startswith("clusters") and B.device_error() == 0
    check(t, first, lse)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    gave_up = 0
    B.set_wait_limit_ns(0)
    try:
        for _ in range(CALLS):
            flush.zero_()
            out, _, _, _ = run(B, t)
            torch.cuda.synchronize()
            err = B.device_error()
            assert err in (0, B.DEVERR_WAIT_TIMEOUT)
            if err:
                gave_up += 1
                if gave_up == 3:
                    break
            else:
                assert torch.equal(out, first)
    finally:
        B.set_wait_limit_ns(B.DEFAULT_WAIT_LIMIT_NS)
    out, lse2, _, _ = run(B, t)
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(lse2, lse) and B.device_error() == 0
    if not gave_up:
        pytest.skip(f"no wait of {CALLS} calls gave up")
