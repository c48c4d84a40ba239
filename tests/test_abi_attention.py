"""attn_shared and cache_evict refuse bad arguments on the host, before any
launch: these calls pass no device memory and run without a GPU."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 4, 5, 6
ONE = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def B():
    from sparse_attention_indexer_idx_gb300 import build
    build.build()
    from sparse_attention_indexer_idx_gb300 import binding
    binding.lib()
    return binding


def attn(bd, **kw):
    D, n_kv, S, P = 128, 2, 64, 32
    a = dict(q=ONE, dtype=bd.IDX_BF16, scale=0.1, B=3, T=1, Hq=8, n_kv=n_kv, D=D, q_stride_b=8 * D, q_stride_t=8 * D,
             q_stride_h=D, k=ONE, v=ONE, S=S, k_stride_b=S * n_kv * D, k_stride_s=n_kv * D, k_stride_h=D,
             v_stride_b=S * n_kv * D, v_stride_s=n_kv * D, v_stride_h=D, len=ONE, pk=ONE, pv=ONE, P=P,
             pk_stride_s=n_kv * D, pk_stride_h=D, pv_stride_s=n_kv * D, pv_stride_h=D)
    a.update(kw)
    return bd.attn_problem(**a)


def call(B, p, out=ONE, mass=None, heads=1, ws=ONE, ws_bytes=1 << 40):
    return B.lib().attn_shared(ctypes.byref(p), out, None, mass, heads, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(len=None), INVALID),
    (dict(pk=None), INVALID), (dict(pv=None), INVALID), (dict(B=-1), INVALID), (dict(T=0), INVALID),
    (dict(Hq=0), INVALID), (dict(n_kv=0), INVALID), (dict(Hq=7), INVALID), (dict(S=-1), INVALID),
    (dict(P=-1), INVALID), (dict(W=-1), INVALID), (dict(W=4), INVALID), (dict(ids_per_head=1), INVALID),
    (dict(ids=ONE, W=4, S=0, k=None, v=None, len=None), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=ONE + 8), INVALID), (dict(k=ONE + 2), INVALID), (dict(k_stride_s=260), INVALID),
    (dict(v_stride_b=4), INVALID), (dict(pv=ONE + 4), INVALID), (dict(pk_stride_h=132), INVALID),
    (dict(dtype=0), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
    (dict(S=(1 << 30) + 1), UNSUPPORTED), (dict(P=(1 << 30) + 1), UNSUPPORTED),
    (dict(B=1 << 30, T=2), UNSUPPORTED), (dict(T=1 << 18, Hq=8), UNSUPPORTED),
    (dict(B=1 << 26, S=1 << 30), UNSUPPORTED), (dict(k_stride_b=1 << 50), UNSUPPORTED),
    (dict(q_stride_t=-(1 << 45)), UNSUPPORTED),
])
def test_attn_refusals(B, kw, status):
    p = attn(B, **kw)
    assert call(B, p) == status
    assert B.lib().attn_shared_workspace_size(ctypes.byref(p), 1) == 0


def test_attn_refuses_its_outputs(B):
    p = attn(B)
    need = B.lib().attn_shared_workspace_size(ctypes.byref(p), 1)
    less = B.lib().attn_shared_workspace_size(ctypes.byref(p), 0)
    assert need > less > 0
    assert call(B, p, out=None) == INVALID
    assert call(B, p, mass=ONE, heads=3) == INVALID
    assert call(B, p, mass=ONE, heads=2, ws_bytes=need - 1) == WORKSPACE
    assert call(B, p, ws_bytes=less - 1) == WORKSPACE
    assert call(B, p, ws=None) == INVALID
    assert B.lib().attn_shared(None, ONE, None, None, 1, ONE, 1, None) == INVALID
    assert B.lib().attn_shared_workspace_size(None, 1) == 0
    assert call(B, attn(B, B=0, q=None, k=None, v=None, len=None, pk=None, pv=None), out=None) == OK  # nothing to do


def evict(bd, planes=(), **kw):
    e = dict(mass=ONE, pos=ONE, len=ONE, cur=ONE, B=2, mass_heads=4, S=100, stride=100, n_keep=40, n_first=2, n_last=8)
    e.update(kw)
    arr = (bd.evict_plane * max(1, len(planes)))(*[bd.evict_plane(**dict(dict(
        base=ONE, row_bytes=256, heads=4, reserved=0, stride_b=1 << 20, stride_s=1024, stride_h=256), **p))
        for p in planes])
    r = bd.evict_problem(planes=arr, n_planes=len(planes), **e)
    r._keep = arr
    return r


@pytest.mark.parametrize("kw,planes,status", [
    (dict(B=-1), (), INVALID), (dict(mass_heads=0), (), INVALID), (dict(S=-1), (), INVALID),
    (dict(stride=99), (), INVALID), (dict(n_keep=0), (), INVALID), (dict(n_first=-1), (), INVALID),
    (dict(n_last=-1), (), INVALID), (dict(n_first=30, n_last=11), (), INVALID), (dict(mass=None), (), INVALID),
    (dict(len=None), (), INVALID), (dict(S=400000, stride=400000), (), UNSUPPORTED),
    (dict(n_keep=400000), (), UNSUPPORTED), (dict(B=1 << 20, mass_heads=2), (), UNSUPPORTED),
    (dict(), (dict(base=None),), INVALID), (dict(), (dict(heads=3),), INVALID), (dict(), (dict(heads=0),), INVALID),
    (dict(), (dict(row_bytes=-1),), INVALID), (dict(), (dict(row_bytes=1 << 21),), UNSUPPORTED),
    (dict(mass_heads=1), (dict(heads=70000),), UNSUPPORTED), (dict(), (dict(),) * 9, INVALID),
])
def test_evict_refusals(B, kw, planes, status):
    p = evict(B, planes, **kw)
    assert B.lib().cache_evict(ctypes.byref(p), ONE, None, None, None, 40, None) == status


def test_evict_refuses_its_outputs(B):
    L = B.lib()
    p = evict(B)
    assert L.cache_evict(ctypes.byref(p), None, None, None, None, 40, None) == INVALID
    assert L.cache_evict(ctypes.byref(p), ONE, None, ONE * 2, None, 39, None) == INVALID
    assert L.cache_evict(ctypes.byref(p), ONE, None, ONE, None, 40, None) == INVALID     # in place: stride 100
    assert L.cache_evict(ctypes.byref(p), ONE, None, None, ONE, 40, None) == INVALID
    assert L.cache_evict(None, ONE, None, None, None, 40, None) == INVALID
    assert L.cache_evict(ctypes.byref(evict(B, B=0)), None, None, None, None, 40, None) == OK
