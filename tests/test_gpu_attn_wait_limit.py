"""The prefix kernel's waits with a limit of zero: blocks of one and of two row
tiles, with one run and with several, give up where a wait is not over at its
first (hardware-timed) look.  The call ends, a block that gave up has said so,
and the next call is whole again."""
import pytest
import torch

from test_gpu_attn import B, _prefix_only  # noqa: F401  (B is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,Hq,n_kv,P,D", [
    (20, 8, 2, 12000, 128),        # one row tile
    (64, 32, 4, 9000, 64),         # both
    (300, 16, 16, 3000, 64),       # 300 rows: a pair of row tiles, then one alone, cut evenly: blocks with several runs
])
def test_blocks_that_give_up(B, rows, Hq, n_kv, P, D):  # noqa: F811
    t, out, lse, p, ws = _prefix_only(B, 52, rows, Hq, n_kv, P, D)
    try:
        B.set_wait_limit_ns(0)
        other = torch.empty_like(out)
        B.attn_shared(p, other, None, None, ws)
        err = B.device_error()
    finally:
        B.set_wait_limit_ns(B.DEFAULT_WAIT_LIMIT_NS)
    assert err == B.DEVERR_WAIT_TIMEOUT or (err == 0 and torch.equal(other, out))
    again = torch.empty_like(out)
    B.attn_shared(p, again, lse, None, ws)
    assert B.device_error() == 0 and torch.equal(again, out)
