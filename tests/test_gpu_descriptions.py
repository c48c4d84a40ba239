"""A problem keeps its description from call to call; it is built again when a
tensor was replaced, or changed its shape, strides or memory in place."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sparse_attention_indexer_idx_gb300 import binding
    binding.lib()
    return binding


def _attn(seed=0, S=8, n_kv=8):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    return dict(q=rn(2, 1, 8, 64), scale=0.1, k=rn(2, S, n_kv, 64), v=rn(2, S, n_kv, 64),
                lens=torch.tensor([S, S - 2], dtype=torch.int32, device="cuda"))


def _call(B, p, W=None):
    out = torch.zeros((2, 1, 8, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.attn_shared_workspace_size(p, False) + (1 << 20), dtype=torch.uint8, device="cuda")
    B.attn_shared(p, out, None, None, ws)
    return out


def test_strides_changed_in_place(B):
    a = _attn()
    p = B.AttnProblem(**a)
    first = _call(B, p)
    a["k"].transpose_(1, 2)            # the same shape and memory, other strides
    a["v"].transpose_(1, 2)
    want = _call(B, B.AttnProblem(**a))
    assert not torch.equal(first, want)
    assert torch.equal(_call(B, p), want)


def test_strides_changed_behind_the_same_memory(B):
    a = _attn(1)
    p = B.AttnProblem(**a)
    first = _call(B, p)
    a["k"].data = a["k"].data.transpose(1, 2)
    want = _call(B, B.AttnProblem(**a))
    assert not torch.equal(first, want)
    assert torch.equal(_call(B, p), want)


def test_a_shape_changed_in_place(B):
    a = _attn(2, S=40)
    ids = torch.arange(40, dtype=torch.int32, device="cuda").repeat(2, 1).view(2, 1, 40).contiguous()
    p = B.AttnProblem(ids=ids, **a)
    first = _call(B, p)
    ids.resize_(2, 1, 20)              # [0..19] and [20..39]
    want = _call(B, B.AttnProblem(ids=ids, **a))
    assert not torch.equal(first, want)
    assert torch.equal(_call(B, p), want)


def test_a_field_and_memory_replaced(B):
    a = _attn(3)
    p = B.AttnProblem(**a)
    _call(B, p)
    a["v"] = a["v"] * 2
    p.v = a["v"]
    assert torch.equal(_call(B, p), _call(B, B.AttnProblem(**a)))
    a["k"].data = torch.zeros_like(a["k"])
    assert torch.equal(_call(B, p), _call(B, B.AttnProblem(**a)))


def test_a_plane_replaced_in_the_callers_list(B):
    """The problem's planes are those that it was given; a list that the caller
    changes afterwards does not change them unnoticed."""
    mass = torch.arange(8, dtype=torch.float32, device="cuda").view(1, 1, 8)
    lens = torch.full((1, 1), 8, dtype=torch.int32, device="cuda")
    src = torch.empty((1, 1, 4), dtype=torch.int32, device="cuda")
    rows = torch.arange(8, dtype=torch.float32, device="cuda").view(1, 8, 1)
    kept = torch.tensor([4.0, 5, 6, 7], device="cuda")
    one, two, three = rows.clone(), rows.clone() + 10, rows.clone() + 20
    planes = [one, two]
    p = B.EvictProblem(mass, lens, 4, planes=planes)
    B.cache_evict(p, src)
    assert torch.equal(one[0, :4, 0], kept) and torch.equal(two[0, :4, 0], kept + 10)
    assert isinstance(p.planes, tuple)
    planes[1] = three
    assert p.planes[1] is two
    with pytest.raises(TypeError):
        p.planes[1] = three
    p.planes = planes                  # assigned again: the new plane is compacted
    two.copy_(rows + 10)
    B.cache_evict(p, src)
    assert torch.equal(three[0, :4, 0], kept + 20)
    assert torch.equal(two, rows + 10)
