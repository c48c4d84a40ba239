"""Tensors of one call of rope_heads, paged_append and attn_paged lie on one device: a
kernel would fault on the others'.  On the host: CPU tensors that say they are on a GPU."""
import pytest
import torch

from sparse_attention_indexer_idx_gb300 import binding as B
from test_paged_step_checks import OnGpu, gpu


def plane(n=3):
    return B.HeadPlane(gpu(n, 2, 64), gpu(n, 2, 64))


class OnOther(OnGpu):
    device = torch.device("cuda", 1)


def test_tensors_of_two_devices_are_refused():
    def other(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype).as_subclass(OnOther)

    pos = gpu(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        B.RopeProblem([B.HeadPlane(gpu(3, 2, 64), other(3, 2, 64))], pos).desc()
    with pytest.raises(ValueError, match="device"):
        B.RopeProblem([plane()], other(3, dtype=torch.int32)).desc()
    with pytest.raises(ValueError, match="device"):
        B.AppendProblem([plane()], pos, other(3, dtype=torch.int32)).desc()

    def attn(**kw):
        t = dict(q=gpu(2, 1, 4, 64), k=gpu(5, 16, 2, 64), v=gpu(5, 16, 2, 64), table=gpu(2, 2, dtype=torch.int32),
                 lens=gpu(2, dtype=torch.int32))
        t.update(kw)
        return B.PagedAttnProblem(scale=1.0, **t)
    attn().desc()
    for kw in (dict(k=other(5, 16, 2, 64)), dict(table=other(2, 2, dtype=torch.int32)), dict(q=other(2, 1, 4, 64)),
               dict(ids=other(2, 1, 3, dtype=torch.int32))):
        with pytest.raises(ValueError, match="device"):
            attn(**kw).desc()
    p = attn()
    for out in (other(2, 1, 4, 64), gpu(2, 1, 4, 64)):
        for lse, ws in ((other(2, 1, 4, dtype=torch.float32), None), (None, other(64, dtype=torch.uint8))):
            with pytest.raises(ValueError, match="device"):
                B.attn_paged(p, out, lse, ws)
