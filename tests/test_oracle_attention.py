"""Pins of the attention and eviction oracle on hand examples, and its
gradient-free invariants (no GPU)."""
import numpy as np

from oracle.attention import attn_shared, cache_evict


def test_two_keys_by_hand():
    # scores 0 and log 3: weights 1/4 and 3/4
    q = np.zeros((1, 1, 1, 2))
    q[..., 0] = np.log(3.0)
    k = np.array([[[[0.0, 5.0]], [[1.0, -2.0]]]])
    v = np.array([[[[4.0, 0.0]], [[0.0, 8.0]]]])
    r = attn_shared(q, 1.0, k, v, np.array([2]), mass=np.zeros((1, 1, 2)))
    assert np.allclose(r["out"][0, 0, 0], [1.0, 6.0])
    assert np.allclose(r["lse"], np.log(4.0))
    assert np.allclose(r["mass"], [[[0.25, 0.75]]])


def test_prefix_and_private_are_one_softmax():
    rng = np.random.default_rng(1)
    B, T, Hq, n_kv, D, P, S = 2, 3, 4, 2, 8, 5, 6
    q = rng.normal(size=(B, T, Hq, D))
    pk, pv = rng.normal(size=(2, P, n_kv, D))
    k, v = rng.normal(size=(2, B, S, n_kv, D))
    lens = np.array([S, 3])
    r = attn_shared(q, 0.3, k, v, lens, pk, pv)
    # the same with the prefix copied into every request's cache
    kk = np.concatenate([np.broadcast_to(pk, (B, P, n_kv, D)), k], 1)
    vv = np.concatenate([np.broadcast_to(pv, (B, P, n_kv, D)), v], 1)
    w = attn_shared(q, 0.3, kk, vv, lens + P)
    assert np.allclose(r["out"], w["out"]) and np.allclose(r["lse"], w["lse"])


def test_rows_without_keys_and_masked_ids():
    q = np.ones((1, 3, 1, 4))
    k = np.ones((1, 4, 1, 4))
    r = attn_shared(q, 1.0, k, k, np.array([2]), mass=np.zeros((1, 1, 4)))
    assert np.isneginf(r["lse"][0, 0, 0]) and (r["out"][0, 0] == 0).all()   # token 0 sees slots < 0
    assert np.allclose(r["mass"][0, 0], [1.5, 0.5, 0, 0])
    ids = np.array([[[-1, 3, 1], [0, -1, 9], [1, 0, -1]]])
    r = attn_shared(q, 1.0, k, k, np.array([2]), ids=ids, mass=np.zeros((1, 1, 4)))
    assert np.isneginf(r["lse"][0, 0, 0])
    assert np.allclose(r["mass"][0, 0], [1.5, 0.5, 0, 0])


def test_evict_by_hand():
    mass = np.array([[[5.0, 1.0, 4.0, 1.0, 9.0, 1.0]]], dtype=np.float32)
    src, n, pos, m = cache_evict(mass, np.array([[6]]), 4)
    # 9, 5, 4 and the first of the ones stay; slot 4 moves to the hole at 3
    assert src.tolist() == [[[0, 1, 2, 4]]] and n.tolist() == [[4]]
    assert m.tolist() == [[[5.0, 1.0, 4.0, 9.0]]]
    src, _, _, _ = cache_evict(mass, np.array([[6]]), 3, n_first=1, n_last=1)
    assert src.tolist() == [[[0, 4, 5]]]          # 0 and 5 are protected, 9 is the best of the rest
    src, n, _, _ = cache_evict(mass, np.array([[2]]), 4)
    assert src.tolist() == [[[0, 1, -1, -1]]] and n.tolist() == [[2]]


def test_evict_keeps_the_best_and_moves_only_into_holes():
    rng = np.random.default_rng(2)
    for _ in range(50):
        S = int(rng.integers(1, 40))
        n, keep = int(rng.integers(0, S + 1)), int(rng.integers(1, S + 1))
        mass = rng.integers(0, 5, size=(1, 1, S)).astype(np.float32)
        src, ln, _, m = cache_evict(mass, np.array([[n]]), keep)
        nk = min(n, keep)
        row = src[0, 0, :nk]
        assert ln[0, 0] == nk and len(set(row.tolist())) == nk
        assert all(s == j or s >= nk for j, s in enumerate(row))
        assert sorted(m[0, 0, :nk])[::-1] == sorted(mass[0, 0, :n])[::-1][:nk]
