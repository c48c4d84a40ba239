"""A step or a prompt of serving.PagedCache that is refused leaves the cache as it
was.  The refusals are the host's, so CPU tensors that say they are on a GPU stand
in for the real ones, and calls that would launch are recorded instead."""
import pytest
import torch

from sparse_attention_indexer_idx_gb300 import binding as B
from sparse_attention_indexer_idx_gb300 import serving

REQUESTS, QH, KH, DIM, IH, ID, TOP = 3, 4, 2, 64, 16, 128, 8


class OnGpu(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return self.device.index


def gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def calls(monkeypatch):
    from sparse_attention_indexer_idx_gb300 import build
    build.build()
    made = []
    for name in ("paged_append", "idx_topk", "witness_merge", "attn_paged"):
        def call(p, *a, _name=name, **kw):
            if hasattr(p, "desc"):
                p.desc()
            made.append(_name)
        monkeypatch.setattr(B, name, call)
    arange = torch.arange                                     # (a prompt makes its slots)
    monkeypatch.setattr(torch, "arange", lambda *a, **kw: arange(*a, **kw).as_subclass(OnGpu))
    return made


def cache(indexer=True, **kw):
    kw = dict(dict(index_heads=IH, index_dim=ID, top_k=TOP) if indexer else {}, **kw)
    c = serving.PagedCache(REQUESTS, 20, 8, 4, QH, KH, DIM, device="cpu", **kw)
    for n, t in list(vars(c).items()):
        if isinstance(t, torch.Tensor):
            setattr(c, n, t.as_subclass(OnGpu))
    return c


def rows(n, indexer=True):
    t = dict(q=gpu(n, QH, DIM), k=gpu(n, KH, DIM), v=gpu(n, KH, DIM))
    if indexer:
        t.update(index_q=gpu(n, IH, ID), index_k=gpu(n, ID), index_w=gpu(n, IH, dtype=torch.float32))
    return t


def state(c):
    return ([list(p) for p in c.pages], list(c.free), list(c.known), c.lens.tolist(), c.live.tolist(), c.table.tolist())


def begun(c, calls, indexer=True):
    """Two requests, one of them at a page's end: a step takes a page."""
    for b, n in ((0, 5), (2, 4)):
        t = rows(n, indexer)
        c.prompt(b, t["k"], t["v"], t.get("index_k"))
    calls.clear()
    return state(c)


def test_a_step_that_is_not_refused(calls):
    c = cache()
    begun(c, calls)
    c.step(**rows(REQUESTS))
    assert calls == ["paged_append", "idx_topk", "witness_merge", "attn_paged"]
    assert c.known == [6, 0, 5] and c.lens.tolist() == [6, 0, 5] and c.slot.tolist() == [5, -1, 4]


BAD = {
    "index_w of 16 bits": dict(index_w=gpu(REQUESTS, IH)),
    "index_w of other heads": dict(index_w=gpu(REQUESTS, IH + 1, dtype=torch.float32)),
    "index_w of fewer requests": dict(index_w=gpu(1, 3, dtype=torch.float32)),
    "index_w in one row": dict(index_w=gpu(REQUESTS * IH, dtype=torch.float32)),
    "index_w that has gaps": dict(index_w=gpu(REQUESTS, 2 * IH, dtype=torch.float32)[:, ::2]),
    "index_w on the host": dict(index_w=torch.zeros(REQUESTS, IH)),
    "no index_w": dict(index_w=None),
    "no index_q": dict(index_q=None),
    "no index_k": dict(index_k=None),
    "index_q of other heads": dict(index_q=gpu(REQUESTS, IH - 1, ID)),
    "index_k of another type": dict(index_k=gpu(REQUESTS, ID, dtype=torch.float32)),
    "q of another type": dict(q=gpu(REQUESTS, QH, DIM, dtype=torch.float16)),
    "q of other requests": dict(q=gpu(REQUESTS - 1, QH, DIM)),
    "k of other heads": dict(k=gpu(REQUESTS, KH + 1, DIM)),
    "v on the host": dict(v=torch.zeros(REQUESTS, KH, DIM, dtype=torch.bfloat16)),
    "segments below 0": dict(segments=-1),
    "segments above their limit": dict(segments=B.IDX_MAX_SEGMENTS + 1),
}


@pytest.mark.parametrize("bad", BAD)
def test_a_refused_step_changes_nothing(calls, bad):
    c = cache()
    before = begun(c, calls)
    with pytest.raises(ValueError):
        c.step(**dict(rows(REQUESTS), **BAD[bad]))
    assert state(c) == before and calls == []
    c.step(**rows(REQUESTS))                                  # as if it had not been called
    assert c.known == [6, 0, 5] and c.lens.tolist() == [6, 0, 5]


def test_a_refused_step_without_the_indexer_changes_nothing(calls):
    c = cache(indexer=False)
    before = begun(c, calls, indexer=False)
    for bad in (dict(q=gpu(REQUESTS, QH, DIM + 64)), dict(k=gpu(REQUESTS, KH, DIM // 2))):
        with pytest.raises(ValueError):
            c.step(**dict(rows(REQUESTS, False), **bad))
        assert state(c) == before and calls == []


def test_a_step_without_memory_for_its_workspace_changes_nothing(calls, monkeypatch):
    c = cache()
    before = begun(c, calls)

    def full(*a, **kw):
        raise torch.OutOfMemoryError("none left")
    rows_ = rows(REQUESTS)
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", full)
        with pytest.raises(torch.OutOfMemoryError):
            c.step(**rows_)
    assert state(c) == before and calls == []


def test_a_step_without_a_page_changes_nothing(calls):
    c = cache()
    begun(c, calls)
    t = rows(16)
    c.prompt(1, t["k"], t["v"], t["index_k"])                  # seven of eight pages, then two more are wanted
    t = rows(3)
    c.prompt(0, t["k"], t["v"], t["index_k"])                  # (request 0: a whole page as well)
    before = state(c)
    calls.clear()
    with pytest.raises(ValueError, match="pages"):
        c.step(**rows(REQUESTS))
    assert state(c) == before and calls == []


def test_an_append_that_the_library_refuses_gives_its_pages_back(calls, monkeypatch):
    c = cache()
    before = begun(c, calls)

    def refuse(*a, **kw):
        raise B.IdxError(4, "plane 0: src and dst need 16-byte aligned bases and strides")
    t = rows(9)
    with monkeypatch.context() as m:
        m.setattr(B, "paged_append", refuse)
        for call in (lambda: c.step(**rows(REQUESTS)), lambda: c.prompt(2, t["k"], t["v"], t["index_k"]),
                     lambda: c.prompt(1, t["k"], t["v"], t["index_k"])):
            with pytest.raises(B.IdxError):
                call()
            assert state(c) == before and calls == []
    c.step(**rows(REQUESTS))
    assert c.known == [6, 0, 5] and c.lens.tolist() == [6, 0, 5]


@pytest.mark.parametrize("bad", [dict(k=gpu(9, KH + 1, DIM)), dict(v=gpu(8, KH, DIM)), dict(index_k=None),
                                 dict(index_k=gpu(9, ID, dtype=torch.float32))])
def test_a_refused_prompt_takes_no_pages(calls, bad):
    c = cache()
    before = begun(c, calls)
    t = dict(rows(9), **bad)
    for b in (1, 2):
        with pytest.raises(ValueError):
            c.prompt(b, t["k"], t["v"], t["index_k"])
        assert state(c) == before and calls == []


@pytest.mark.parametrize("kw", [
    dict(index_dtype=torch.float16), dict(index_dtype=torch.float8_e4m3fn), dict(index_dim=96), dict(index_dim=512),
    dict(index_heads=129), dict(index_heads=128, index_dim=256), dict(index_rot=24), dict(index_dim=32, index_rot=64),
    dict(top_k=0), dict(top_k=B.IDX_MAX_K + 1), dict(dtype=torch.float32), dict(rot=72), dict(rot=-16), dict(rot=24),
    dict(eps=-1.0), dict(eps=float("nan")), dict(norms={"q": torch.ones(DIM + 1)}), dict(norms={"key": torch.ones(DIM)}),
    dict(norms={"index_q": torch.ones(DIM)})])
def test_a_cache_that_no_step_could_use_is_refused(kw):
    kw = dict(dict(index_heads=IH, index_dim=ID, top_k=TOP), **kw)
    with pytest.raises(ValueError):
        serving.PagedCache(REQUESTS, 20, 8, 4, QH, KH, DIM, device="cpu", **kw)


@pytest.mark.parametrize("q_heads,kv_heads,dim", [(5, 2, 64), (4, 0, 64), (0, 2, 64), (4, 2, 96), (4, 2, 256)])
def test_heads_that_attention_does_not_have_are_refused(q_heads, kv_heads, dim):
    with pytest.raises(ValueError):
        serving.PagedCache(REQUESTS, 20, 8, 4, q_heads, kv_heads, dim, device="cpu")


def test_caches_of_every_kind_that_steps_can_use():
    for kw in (dict(dtype=torch.float16, rot=0), dict(rot=32, index_heads=3, top_k=1, index_dim=32, index_rot=32),
               dict(index_heads=64, top_k=B.IDX_MAX_K, index_dim=256, index_rot=0, index_dtype=torch.float32),
               dict(norms={n: torch.ones(DIM) for n in ("q", "k")}, eps=0.0)):
        serving.PagedCache(REQUESTS, 20, 8, 4, QH, KH, DIM, device="cpu", **kw)
