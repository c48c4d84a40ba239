"""What an indexer problem's tensors have to be: their addresses are all that the
library gets, so a short or mistyped one would be read behind its end.  The checks
come before a tensor's device is looked at, and so run on CPU tensors."""
import pytest
import torch

from sparse_attention_indexer_idx_gb300 import binding as B

M, H, D, N = 2, 16, 128, 40


def problem(**kw):
    t = dict(q=torch.zeros(M, H, D, dtype=torch.bfloat16), w=torch.zeros(M, H),
             keys=torch.zeros(N, D, dtype=torch.bfloat16), key_len=torch.zeros(M, dtype=torch.int32), max_key_len=20,
             key_off=torch.zeros(M, dtype=torch.int64))
    return B.Problem(**dict(t, **kw))


@pytest.mark.parametrize("name,bad", [
    ("w", torch.zeros(M, H, dtype=torch.bfloat16)),          # half the bytes that are read
    ("w", torch.zeros(M, H, dtype=torch.float64)),
    ("w", torch.zeros(1, 3)),
    ("w", torch.zeros(M, H - 1)),
    ("w", None),
    ("key_len", torch.zeros(M, dtype=torch.int64)),
    ("key_len", torch.zeros(M - 1, dtype=torch.int32)),
    ("key_off", torch.zeros(M, dtype=torch.int32)),
    ("key_off", torch.zeros(1, dtype=torch.int64)),
    ("key_scale", torch.zeros(N - 1)),
    ("key_scale", torch.zeros(N, dtype=torch.bfloat16)),
    ("keys", torch.zeros(N, D - 1, dtype=torch.bfloat16)),
    ("keys", torch.zeros(N * D, dtype=torch.bfloat16)),
    ("keys", torch.zeros(N, D, dtype=torch.float16)),
    ("q", torch.zeros(M * H, D, dtype=torch.bfloat16)),
    ("q", torch.zeros(M, H, D, dtype=torch.float16)),
])
def test_short_and_mistyped_tensors_are_refused_by_name(name, bad):
    with pytest.raises(ValueError, match=f"^{name}: "):
        problem(**{name: bad}).c()


@pytest.mark.parametrize("kw", [{}, {"w": torch.zeros(M * H)}, {"w": torch.zeros(M + 1, H)}, {"key_off": None},
                                {"key_scale": torch.zeros(N), "keys": torch.zeros(N, D, dtype=torch.uint8)}])
def test_right_ones_come_as_far_as_the_device(kw):
    with pytest.raises(ValueError, match="CUDA"):
        problem(**kw).c()
