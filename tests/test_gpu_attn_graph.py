"""A captured step, replayed after its tensors' contents changed, against an
eager call on the same contents."""
import pytest
import torch

from test_gpu_attn import B, make  # noqa: F401  (B is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [
    dict(B=20, T=1, Hq=16, n_kv=2, D=128, P=9000, S=300, mass=1),            # tensor cores, caches beside them
    dict(B=5, T=2, Hq=8, n_kv=2, D=64, P=100, S=700, mass=2, dtype="f16"),
    dict(B=6, T=1, Hq=32, n_kv=4, D=128, S=2000, W=200, mass=1),
    dict(B=3, T=3, Hq=16, n_kv=4, D=64, P=333, S=500, W=70, ids_per_head=True, mass=4),
])
def test_replays_on_new_contents(B, kw):  # noqa: F811
    names = ("q", "k", "v", "lens", "pk", "pv", "prefix_len", "ids", "mass")
    Bn, S, heads = kw["B"], kw["S"], kw["mass"]
    plen = [kw["P"] - 7 * i for i in range(Bn)] if "P" in kw else None

    def contents(seed):
        t = make(seed, prefix_len=None if plen is None else plen[::-1] if seed % 2 else plen, **kw)
        d = {n: t[n].cuda() for n in names if n in t}
        d["each"] = d["lens"].view(Bn, 1).expand(Bn, heads).contiguous()   # the same lengths for every mass head
        return t["scale"], d

    def problem(scale, d):
        p = B.AttnProblem(d["q"], scale, d["k"], d["v"], d["lens"], d.get("pk"), d.get("pv"), d.get("prefix_len"),
                          d.get("ids"))
        return p, B.EvictProblem(d["mass"], d["each"], S // 3, 2, 16, planes=(d["k"], d["v"]))

    def outputs(d):
        return (torch.zeros_like(d["q"]), torch.zeros(d["q"].shape[:-1], device="cuda"),
                torch.zeros((Bn, heads, S // 3), dtype=torch.int32, device="cuda"))

    def step(p, e, d, out, lse, src, ws):
        B.attn_shared(p, out, lse, d["mass"], ws)
        B.cache_evict(e, src)

    scale, d = contents(900)
    p, e = problem(scale, d)
    o = outputs(d)
    ws = torch.empty(B.attn_shared_workspace_size(p, True), dtype=torch.uint8, device="cuda")
    step(p, e, d, *o, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(p, e, d, *o, ws)
    torch.cuda.synchronize()
    for seed in (901, 902, 903):
        _, new = contents(seed)
        for n in new:
            d[n].copy_(new[n])
        g.replay()
        want = outputs(new)
        step(*problem(scale, new), new, *want, torch.empty_like(ws))
        torch.cuda.synchronize()
        for a, b in zip(o, want):
            assert torch.equal(a, b)
        for n in ("mass", "k", "v"):
            assert torch.equal(d[n], new[n])
    assert B.device_error() == 0
