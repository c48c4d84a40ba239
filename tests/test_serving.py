"""The host's side of serving.DecodeCache: prompts, appending, full caches.  These
need no kernel, so they run on CPU tensors."""
import pytest
import torch

from sparse_attention_indexer_idx_gb300 import serving


def cache(requests=3, slots=6):
    return serving.DecodeCache(requests, slots, 4, 2, 8, 8, 4, device="cpu")


def token(i, requests=3):
    x = torch.full((requests, 2, 8), float(i)).bfloat16()
    return x, -x, x[:, 0]


def prompt(n, requests=3):
    x = torch.ones(requests, n, 2, 8).bfloat16()
    return x, x, x[:, :, 0]


def test_full_caches_refuse_a_token_and_stay_as_they_are():
    c = cache()
    c.fill(*prompt(4), lens=[4, 1, 0])
    for i in (2, 3):
        c.append(*token(i))
    before = {n: getattr(c, n).clone() for n in ("k", "v", "index_k", "lens", "pos", "cur")}
    with pytest.raises(ValueError):
        c.append(*token(4))
    assert all(torch.equal(before[n], getattr(c, n)) for n in before)
    assert c.lens.view(-1).tolist() == [6, 3, 2] and c.cur.tolist() == [6, 3, 2]


def test_a_cache_that_was_never_filled_takes_its_slots():
    c = cache(slots=2)
    c.append(*token(1))
    c.append(*token(2))
    with pytest.raises(ValueError):
        c.append(*token(3))
    assert c.pos[:, 0].tolist() == [[0, 1]] * 3


def test_tokens_go_behind_each_prompt():
    c = cache()
    c.fill(*prompt(4), lens=[4, 1, 0])
    c.append(*token(7))
    assert c.lens.view(-1).tolist() == [5, 2, 1]
    for b, at in enumerate((4, 1, 0)):
        assert (c.k[b, at] == 7).all() and (c.v[b, at] == -7).all() and (c.index_k[b, at] == 7).all()
        assert c.pos[b, 0].tolist() == [i if i <= at else -1 for i in range(6)]


def test_lengths_changed_past_the_count_index_nothing_out_of_range():
    c = cache()
    c.lens += 6
    c.append(*token(5))
    assert c.lens.view(-1).tolist() == [7] * 3    # the kernels report such a length


@pytest.mark.parametrize("n,lens", [(7, None), (4, [4, 4]), (4, [5, 0, 0]), (4, [-1, 0, 0])])
def test_prompts_that_do_not_fit_are_refused(n, lens):
    with pytest.raises(ValueError):
        cache().fill(*prompt(n), lens=lens)


@pytest.mark.parametrize("n_keep", [0, -1, 7])
def test_trims_to_no_slot_or_to_more_than_there_are_are_refused(n_keep):
    with pytest.raises(ValueError):
        cache().trim(n_keep, 0, 0)
