"""attn_shared against the 64-bit oracle: head layouts, lengths of zero and one,
odd sizes, strides, id lists, partial prefixes, rows without keys, garbage in
slots that nobody sees, other streams, refusals.

Error bounds, from the arithmetic: a weight is rounded to the element type for
the product with v (relative u = 2^-8 for bf16, which has 8 significant bits,
2^-11 for fp16, which has 11, and for fp16 at most 2^-25 absolute below its
normal range), and so is the output; scores,
maxima and sums are fp32, whose accumulation over D terms moves x by at most
D 2^-23 scale sum|q||k| (absx), which moves a weight by that much, relatively."""
import numpy as np
import pytest
import torch

from oracle import attention as oracle

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def B():
    from sparse_attention_indexer_idx_gb300 import binding
    binding.lib()
    return binding


def make(seed, B=2, T=1, Hq=8, n_kv=2, D=128, P=0, S=0, W=0, ids_per_head=False, mass=0, lens=None, prefix_len=None,
         dtype="bf16", layout="bshd", garbage=False, per_head_lens=False):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    rn = lambda *s: torch.randn(*s, generator=g).to(dt)  # noqa: E731
    t = {"q": rn(B, T, Hq, D), "scale": 1.0 / D ** 0.5}
    if S:
        t["k"], t["v"] = rn(B, S, n_kv, D), rn(B, S, n_kv, D)
        if lens is None:
            lens = torch.randint(0, S + 1, (B, n_kv) if per_head_lens else (B,), generator=g)
        t["lens"] = torch.as_tensor(lens).to(torch.int32)
        if garbage:
            longest = t["lens"].view(B, -1).amax(1)
            for b in range(B):
                t["k"][b, int(longest[b]):] = float("nan")
                t["v"][b, int(longest[b]):] = float("nan")
    if P:
        t["pk"], t["pv"] = rn(P, n_kv, D), rn(P, n_kv, D)
        if prefix_len is not None:
            t["prefix_len"] = torch.as_tensor(prefix_len).to(torch.int32)
            if garbage:
                t["pk"][int(t["prefix_len"].max()):] = float("nan")
                t["pv"][int(t["prefix_len"].max()):] = float("nan")
    if W:
        shape = (B, T, n_kv, W) if ids_per_head else (B, T, W)
        flat = [torch.randperm(max(S, W), generator=g)[:W] for _ in range(int(np.prod(shape[:-1])))]
        ids = torch.stack(flat).view(shape).to(torch.int32)
        t["ids"] = torch.where(torch.rand(shape, generator=g) < 0.1, -1, ids.clamp(max=S + 5))
    if mass:
        t["mass"] = torch.rand(B, mass, S, generator=g)
    t["dtype"], t["layout"] = dtype, layout
    return t


def run(Bd, t, stream=None):
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in t.items()}
    if t["layout"] == "bhsd":
        for n in ("k", "v"):
            if n in dev:
                dev[n] = dev[n].transpose(1, 2).contiguous().transpose(1, 2)
        for n in ("pk", "pv"):
            if n in dev:
                dev[n] = dev[n].transpose(0, 1).contiguous().transpose(0, 1)
        dev["q"] = torch.cat([dev["q"], dev["q"]], -1)[..., : dev["q"].shape[-1]]   # rows of a wider projection
    p = Bd.AttnProblem(dev["q"], t["scale"], dev.get("k"), dev.get("v"), dev.get("lens"), dev.get("pk"),
                       dev.get("pv"), dev.get("prefix_len"), dev.get("ids"))
    out = torch.full(tuple(t["q"].shape), float("nan"), dtype=t["q"].dtype, device="cuda")
    lse = torch.full(tuple(t["q"].shape[:-1]), float("nan"), device="cuda")
    mass = dev.get("mass")
    ws = torch.full((Bd.attn_shared_workspace_size(p, mass is not None),), 0xFF, dtype=torch.uint8, device="cuda")
    Bd.attn_shared(p, out, lse, mass, ws, stream=stream)
    return out, lse, mass, p, ws


def check(t, out, lse, mass):
    num = lambda x: None if x is None else x.float().numpy() if x.is_floating_point() else x.numpy()  # noqa: E731
    ref = oracle.attn_shared(*(num(t["q"]), t["scale"]), *(num(t.get(n)) for n in
                             ("k", "v", "lens", "pk", "pv", "prefix_len", "ids", "mass")))
    D = t["q"].shape[-1]
    u = 2.0 ** -8 if t["dtype"] == "bf16" else 2.0 ** -11
    keys = (t["k"].shape[1] if "k" in t else 0) + (t["pk"].shape[0] if "pk" in t else 0)
    vmax = max(np.nanmax(np.abs(num(t[n]))) for n in ("v", "pv") if n in t)
    dx = D * 2.0 ** -23 * ref["absx"] + 2.0 ** -21
    got = out.float().cpu().numpy().astype(np.float64)
    tol = ref["absv"] * (2.2 * u + 4 * dx[..., None]) + 1e-6
    if t["dtype"] == "f16":
        tol = tol + keys * 2.0 ** -25 * vmax
    assert np.isfinite(got).all()
    assert (np.abs(got - ref["out"]) <= tol).all(), np.abs(got - ref["out"]).max()
    gl = lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(gl), empty)
    assert (got[empty] == 0).all()
    lt = dx + 2.0 ** -21 * (1 + np.abs(np.where(empty, 0, ref["lse"])))
    assert (np.abs(gl[~empty] - ref["lse"][~empty]) <= lt[~empty]).all()
    if mass is not None:
        gm = mass.cpu().numpy().astype(np.float64)
        add = ref["mass"] - num(t["mass"])
        rows = t["q"].shape[1] * t["q"].shape[2]
        mt = add * (4 * dx.max() + rows * 2.0 ** -24) + 2.0 ** -22 * ref["mass"] + 1e-9
        assert (np.abs(gm - ref["mass"]) <= mt).all(), np.abs(gm - ref["mass"]).max()


CASES = [
    dict(B=1, T=1, Hq=1, n_kv=1, S=1, lens=[1], mass=1),
    dict(B=1, T=1, Hq=8, n_kv=1, P=1),
    dict(B=2, T=1, Hq=32, n_kv=4, S=333, P=129, mass=4),
    dict(B=3, T=1, Hq=7, n_kv=1, S=515, lens=[0, 1, 515], mass=1, dtype="f16"),
    dict(B=3, T=5, Hq=16, n_kv=2, S=100, lens=[0, 3, 100], P=31, mass=2, D=64),
    dict(B=3, T=5, Hq=16, n_kv=2, S=100, lens=[0, 3, 100], mass=1, D=64, dtype="f16"),
    dict(B=2, T=8, Hq=32, n_kv=2, S=700, mass=2, garbage=True, layout="bhsd"),
    dict(B=2, T=3, Hq=28, n_kv=4, S=257, P=70, mass=1, per_head_lens=True, garbage=True, D=64, layout="bhsd"),
    dict(B=5, T=1, Hq=16, n_kv=16, P=777, S=65, prefix_len=[0, 1, 200, 500, 640], garbage=True),
    dict(B=2, T=2, Hq=8, n_kv=2, P=50, prefix_len=[0, 0], S=9, lens=[0, 1], mass=2),
    dict(B=4, T=1, Hq=64, n_kv=4, S=900, W=300, mass=1),
    dict(B=2, T=1, Hq=64, n_kv=1, S=900, W=1, mass=1, D=64),
    dict(B=2, T=3, Hq=16, n_kv=4, S=333, W=101, ids_per_head=True, mass=4, dtype="f16"),
    dict(B=2, T=4, Hq=16, n_kv=4, S=333, W=64, ids_per_head=True, mass=1, D=64, P=100, layout="bhsd"),
    dict(B=2, T=4, Hq=16, n_kv=4, S=333, W=77, mass=4, garbage=True, lens=[2, 300]),
    dict(B=1, T=1, Hq=40, n_kv=1, S=2000, lens=[1999], mass=1),
    # many rows on one prefix
    dict(B=70, T=1, Hq=16, n_kv=2, P=1000, S=20, mass=2),
    dict(B=33, T=4, Hq=16, n_kv=2, P=515, S=8, D=64, dtype="f16"),
    dict(B=130, T=1, Hq=8, n_kv=1, P=640, S=3, prefix_len=[(37 * i) % 641 for i in range(130)], mass=1),
    dict(B=64, T=2, Hq=32, n_kv=4, P=260, S=2, layout="bhsd", garbage=True, prefix_len=[200 - i for i in range(64)]),
    dict(B=40, T=1, Hq=64, n_kv=8, P=4097, S=33, mass=1, D=64),
    dict(B=2, T=60, Hq=16, n_kv=2, S=400, lens=[400, 61], mass=2),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_oracle(B, case):
    t = make(100 + case, **CASES[case])
    assert B.device_error() == 0
    out, lse, mass, p, ws = run(B, t)
    torch.cuda.synchronize()
    assert B.device_error() == 0
    check(t, out, lse, mass)
    # the same inputs again, masses restored, over the used workspace: the same bits
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    mass2 = None if mass is None else t["mass"].cuda()
    B.attn_shared(p, out2, lse2, mass2, ws)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert mass is None or torch.equal(mass, mass2)


def test_steep_scores(B):
    # scores in the hundreds, growing along the sequence: the running maximum keeps moving
    t = make(7, B=2, T=1, Hq=8, n_kv=2, P=600, S=600, lens=[600, 599], mass=2)
    ramp = torch.linspace(0, 30, 600).view(600, 1, 1)
    t["q"] = torch.ones_like(t["q"])
    t["pk"] = (ramp + 0 * t["pk"].float()).to(torch.bfloat16)
    t["k"] = (ramp + 1 + 0 * t["k"].float()).to(torch.bfloat16)
    out, lse, mass, _, _ = run(B, t)
    check(t, out, lse, mass)


def test_many_rows_steep(B):
    t = make(8, B=96, T=1, Hq=16, n_kv=2, P=900, S=4)
    ramp = torch.linspace(-20, 30, 900).view(900, 1, 1)
    t["q"] = (1 + 0 * t["q"].float()).to(torch.bfloat16)
    t["pk"] = (ramp + 0.1 * t["pk"].float()).to(torch.bfloat16)
    out, lse, mass, _, _ = run(B, t)
    check(t, out, lse, mass)


def test_optional_outputs_and_another_stream(B):
    t = make(9, B=3, T=1, Hq=8, n_kv=2, P=40, S=50, mass=2)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out, lse, mass, p, ws = run(B, t, stream=s)
    s.synchronize()
    check(t, out, lse, mass)
    out2 = torch.empty_like(out)
    B.attn_shared(p, out2, None, None, ws)
    assert torch.equal(out, out2)


def test_bad_lengths_are_empty_rows_and_reported(B):
    t = make(10, B=3, T=1, Hq=4, n_kv=1, S=20, lens=[20, 21, -1], mass=1)
    assert B.device_error() == 0
    out, lse, mass, _, _ = run(B, t)
    assert B.device_error() == B.DEVERR_BAD_ROW
    t["lens"] = torch.tensor([20, 0, 0], dtype=torch.int32)
    check(t, out, lse, mass)


def test_from_the_indexer_to_the_cache(B):
    """The decode step as it is used: the indexer's top-K with its witnesses,
    attention over those tokens behind a shared prefix, and the caches trimmed
    by the masses, the index keys along with them."""
    from sparse_attention_indexer_idx_gb300 import serving
    got = serving.decode_step_example(seed=3, requests=4, prefix=300, slots=700, K=128, n_keep=500)
    assert got["len_after"] == [500] * 4 and got["finite"]
    assert B.device_error() == 0


def test_refusals(B):
    t = make(11, B=2, T=1, Hq=8, n_kv=2, P=16, S=16, mass=2)
    out, lse, mass, p, ws = run(B, t)
    torch.cuda.synchronize()
    before = mass.clone()
    with pytest.raises(B.IdxError) as e:
        B.attn_shared(p, out, lse, mass, ws[:16])
    assert e.value.name == "WORKSPACE_TOO_SMALL"
    bad = dict(out=out[:1], lse=lse[:, :, :4], mass=mass[:, :1, :8])
    for name, x in bad.items():
        a = dict(out=out, lse=lse, mass=mass)
        a[name] = x
        with pytest.raises(ValueError):
            B.attn_shared(p, a["out"], a["lse"], a["mass"], ws)
    q = p.q
    for field, x in (("q", q.float()), ("q", q[..., :32]), ("k", p.k.half()), ("v", p.v[:, :8]), ("lens", p.lens.long()),
                     ("pk", p.pk[:, :1]), ("ids", torch.zeros(2, 2, 4, dtype=torch.int32, device="cuda")),
                     ("k", p.k.transpose(2, 3).contiguous().transpose(2, 3)), ("q", q[:, :, :7])):
        keep = getattr(p, field)
        setattr(p, field, x)
        with pytest.raises((ValueError, B.IdxError)):
            B.attn_shared(p, out if field != "q" else torch.empty_like(x), lse, mass, ws)
        setattr(p, field, keep)
    # rows that start off a 16-byte boundary
    wide = torch.zeros(2, 16, 2, 132, dtype=torch.bfloat16, device="cuda")
    p2 = B.AttnProblem(q, 1.0, wide[..., 4:], wide[..., 4:], p.lens)
    with pytest.raises(B.IdxError) as e:
        B.attn_shared(p2, out, lse, None, ws)
    assert e.value.name == "INVALID_ARG"
    torch.cuda.synchronize()
    assert torch.equal(before, mass)


def test_slots_beyond_32_bits(B):
    """A cache whose elements pass 2^32: the last request's rows lie behind it."""
    S, n_kv, D = 1 << 17, 8, 128
    Bn = 35                               # 35 * 2^17 * 8 * 128 elements = 2^32.1
    k = torch.zeros((Bn, S, n_kv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((Bn, S, n_kv, D), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(5)
    at = S - 40
    kk, vv = (torch.randn(40, n_kv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    k[-1, at:], v[-1, at:] = kk.cuda(), vv.cuda()
    ids = torch.full((Bn, 1, 40), -1, dtype=torch.int32, device="cuda")
    ids[-1, 0] = torch.arange(at, S)
    q = torch.randn(Bn, 1, 16, D, generator=g).to(torch.bfloat16)
    p = B.AttnProblem(q.cuda(), 0.1, k, v, torch.full((Bn,), S, dtype=torch.int32, device="cuda"), ids=ids)
    out = torch.empty((Bn, 1, 16, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((Bn, 1, 16), device="cuda")
    ws = torch.empty(B.attn_shared_workspace_size(p, False), dtype=torch.uint8, device="cuda")
    B.attn_shared(p, out, lse, None, ws)
    t = {"q": q[-1:], "scale": 0.1, "k": kk[None], "v": vv[None], "lens": torch.tensor([40], dtype=torch.int32),
         "dtype": "bf16"}
    check(t, out[-1:], lse[-1:], None)
    assert torch.isneginf(lse[:-1]).all() and (out[:-1] == 0).all()


def _prefix_only(B, seed, rows, Hq, n_kv, P, D, dtype="bf16", prefix_len=None, layout="bshd"):
    t = make(seed, B=rows, T=1, Hq=Hq, n_kv=n_kv, D=D, P=P, dtype=dtype, prefix_len=prefix_len, layout=layout,
             garbage=prefix_len is not None)
    out, lse, mass, p, ws = run(B, t)
    torch.cuda.synchronize()
    assert B.device_error() == 0
    return t, out, lse, p, ws


# pieces, lists and slots in unusual numbers
SHAPES = [
    dict(B=1, T=1, Hq=4, n_kv=1, P=30011, S=50, mass=1),                              # hundreds of pieces a row
    dict(B=2, T=1, Hq=28, n_kv=4, P=20000, D=64, prefix_len=[20000, 777], dtype="f16"),
    dict(B=1, T=3, Hq=8, n_kv=8, S=40000, mass=8, D=64),
    dict(B=2, T=4, Hq=64, n_kv=16, P=300, S=12, W=8, ids_per_head=True, mass=1, D=64),  # 64 short lists on 12 slots
    dict(B=2, T=20, Hq=64, n_kv=4, S=500, W=40, ids_per_head=True, mass=1, D=64),     # more rows than are held at once
    dict(B=2, T=1, Hq=600, n_kv=1, S=900, W=33, mass=1, D=64),                        # of one list
    dict(B=3, T=2, Hq=8, n_kv=2, S=3000, W=1500, mass=2, lens=[0, 1, 2900]),
    dict(B=2, T=1, Hq=256, n_kv=16, S=170, mass=1, D=64, lens=[170, 3]),              # many rows on few slots
    dict(B=1, T=9, Hq=128, n_kv=1, S=37, mass=1, D=64),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_pieces_lists_and_slots(B, case):
    t = make(200 + case, **SHAPES[case])
    out, lse, mass, p, ws = run(B, t)
    torch.cuda.synchronize()
    check(t, out, lse, mass)
    mass2 = None if mass is None else t["mass"].cuda()
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    B.attn_shared(p, out2, lse2, mass2, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert mass is None or torch.equal(mass, mass2)
    assert B.device_error() == 0


# many rows of a KV head over long caches: more than 48 MB of scores
LONG = [
    dict(B=2, T=4, Hq=64, n_kv=4, S=26001, lens=[26001, 13], mass=4, D=64, garbage=True),
    dict(B=2, T=3, Hq=56, n_kv=2, S=40003, P=70, mass=1, per_head_lens=True, garbage=True, dtype="f16", layout="bhsd"),
    dict(B=4, T=5, Hq=40, n_kv=4, S=16385, lens=[0, 3, 16385, 257], mass=1, D=64, layout="bhsd"),
]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_masses_of_long_caches_under_many_rows(B, case):
    t = make(300 + case, **LONG[case])
    out, lse, mass, p, ws = run(B, t)
    torch.cuda.synchronize()
    check(t, out, lse, mass)
    assert B.device_error() == 0


@pytest.mark.parametrize("rows,Hq,n_kv,P,D,dtype,plen", [
    (17, 8, 8, 5000, 128, "bf16", None),       # a part of one row tile
    (64, 4, 2, 40000, 64, "f16", None),        # one row tile, many key tiles
    (16, 64, 8, 9001, 128, "bf16", None),      # one whole row tile, a ragged last key tile
    (40, 32, 8, 4999, 128, "f16", None),       # two row tiles
    (150, 8, 4, 6500, 64, "bf16", None),       # two pairs of row tiles, the last one partly empty
    (33, 32, 4, 5000, 128, "bf16", [13 * i for i in range(33)]),           # nothing visible behind 416
    (40, 16, 2, 12000, 64, "bf16", [0] * 39 + [7777]),                     # one request sees anything
    (21, 16, 2, 12000, 128, "f16", [11000 - 517 * i for i in range(21)]),  # one row tile, ragged limits
])
def test_prefix_on_the_tensor_cores(B, rows, Hq, n_kv, P, D, dtype, plen):
    t, out, lse, p, ws = _prefix_only(B, rows, rows, Hq, n_kv, P, D, dtype, plen)
    # the 64-bit oracle on a few requests (rows are independent)
    pick = [0, rows // 2, rows - 1]
    few = dict(t, q=t["q"][pick])
    if plen is not None:
        few["prefix_len"] = t["prefix_len"][pick]
    check(few, out[pick], lse[pick], None)
    assert torch.isfinite(out.float()).all()


def test_strides_that_no_tensor_map_holds(B):
    # the heads share their memory: a head stride of zero is read by the streaming kernel
    g = torch.Generator().manual_seed(3)
    one = torch.randn(3000, 1, 128, generator=g).to(torch.bfloat16)
    t = {"q": torch.randn(40, 1, 16, 128, generator=g).to(torch.bfloat16), "scale": 0.1, "dtype": "bf16",
         "pk": one.expand(3000, 8, 128), "pv": one.expand(3000, 8, 128)}
    p = B.AttnProblem(t["q"].cuda(), 0.1, pk=one.cuda().expand(3000, 8, 128), pv=one.cuda().expand(3000, 8, 128))
    out, lse = torch.empty_like(p.q), torch.empty((40, 1, 16), device="cuda")
    ws = torch.empty(B.attn_shared_workspace_size(p, False), dtype=torch.uint8, device="cuda")
    B.attn_shared(p, out, lse, None, ws)
    few = dict(t, q=t["q"][::13])
    check(few, out[::13], lse[::13], None)


@pytest.mark.parametrize("rows,P", [(32, 8192), (24, 5000), (64, 6000)])
def test_many_repeats_agree(B, rows, P):
    """The pipeline of the tensor-core kernel, run often beside other work: no
    wait gives up and every run leaves the same bits."""
    t, out, lse, p, ws = _prefix_only(B, 50, rows, 32, 8, P, 128)
    other = torch.empty_like(out)
    noise = torch.zeros(1 << 26, device="cuda")
    for i in range(300):
        if i % 7 == 0:
            noise.add_(1.0)
        B.attn_shared(p, other, lse, None, ws)
        if i % 50 == 49:
            assert torch.equal(out, other)
    assert B.device_error() == 0


def test_wait_limit_is_reported(B):
    t, out, lse, p, ws = _prefix_only(B, 51, 64, 32, 8, 8192, 128)
    try:
        B.set_wait_limit_ns(0)
        B.attn_shared(p, torch.empty_like(out), None, None, ws)
        err = B.device_error()
    finally:
        B.set_wait_limit_ns(B.DEFAULT_WAIT_LIMIT_NS)
    assert err & B.DEVERR_WAIT_TIMEOUT
    again = torch.empty_like(out)
    B.attn_shared(p, again, lse, None, ws)
    assert B.device_error() == 0 and torch.equal(again, out)


@pytest.mark.parametrize("rows,Hq,n_kv,P,D,dtype", [(32, 32, 8, 8192, 128, "bf16"), (20, 8, 4, 12000, 64, "f16"),
                                                   (24, 16, 16, 5000, 128, "bf16"), (160, 16, 8, 3000, 128, "bf16")])
def test_steep_scores_on_the_tensor_cores(B, rows, Hq, n_kv, P, D, dtype):
    # The running maximum passes its reference over and over, at other tiles for
    # each row: the accumulator is rescaled while products are under way.
    t = make(60, B=rows, T=1, Hq=Hq, n_kv=n_kv, D=D, P=P, dtype=dtype)
    g = torch.Generator().manual_seed(61)
    ramp = torch.linspace(0, 6, P).view(P, 1, 1) * (1 + torch.rand(1, n_kv, 1, generator=g))
    t["pk"] = (ramp + 0.5 * t["pk"].float()).to(DT[dtype])
    t["q"] = (torch.rand(rows, 1, Hq, 1, generator=g) * 2 - 0.5 + 0.3 * t["q"].float()).to(DT[dtype])
    for _ in range(5):
        out, lse, mass, p, ws = run(B, t)
        pick = [0, 3, rows // 2, rows - 1]
        few = dict(t, q=t["q"][pick])
        check(few, out[pick], lse[pick], None)
    assert B.device_error() == 0


@pytest.mark.parametrize("P", [0, 500, 9000])
def test_copies_fills_and_forks_before_a_captured_call(B, P):
    """What comes right before a call in a graph need not be a kernel, nor one node."""
    t = make(71, B=20, T=1, Hq=16, n_kv=2, D=128, P=P, S=300, mass=1, lens=[300] * 20)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in t.items()}
    p = B.AttnProblem(d["q"], t["scale"], d["k"], d["v"], d["lens"], d.get("pk"), d.get("pv"))
    out, lse = torch.empty_like(d["q"]), torch.empty((20, 1, 16), device="cuda")
    ws = torch.empty(B.attn_shared_workspace_size(p, True), dtype=torch.uint8, device="cuda")
    lens = torch.full((20, 1), 300, dtype=torch.int32, device="cuda")
    e = B.EvictProblem(d["mass"], lens, 128, 2, 16, planes=(d["k"], d["v"]))
    src = torch.empty((20, 1, 128), dtype=torch.int32, device="cuda")
    start = [x.clone() for x in (d["mass"], d["k"], d["v"])]
    side = torch.cuda.Stream()

    def step():
        now = torch.cuda.current_stream()
        side.wait_stream(now)
        with torch.cuda.stream(side):
            d["k"].copy_(start[1])
        d["v"].copy_(start[2])
        d["mass"].copy_(start[0])
        ws.zero_()
        now.wait_stream(side)
        B.attn_shared(p, out, lse, d["mass"], ws)
        src.zero_()
        B.cache_evict(e, src)

    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (out, lse, d["mass"], src, d["k"], d["v"])]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.synchronize()
    for _ in range(3):
        for x in (out, lse, d["mass"], src, d["k"], d["v"]):
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip((out, lse, d["mass"], src, d["k"], d["v"]), want):
            assert torch.equal(x, y)
    assert B.device_error() == 0


def test_step_in_a_graph(B):
    """Attention and eviction captured once and replayed on new contents."""
    t = make(70, B=20, T=1, Hq=16, n_kv=2, D=128, P=9000, S=300, mass=1, lens=[300] * 20)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in t.items()}
    p = B.AttnProblem(d["q"], t["scale"], d["k"], d["v"], d["lens"], d["pk"], d["pv"])
    out, lse = torch.empty_like(d["q"]), torch.empty((20, 1, 16), device="cuda")
    ws = torch.empty(B.attn_shared_workspace_size(p, True), dtype=torch.uint8, device="cuda")
    lens = torch.full((20, 1), 300, dtype=torch.int32, device="cuda")
    e = B.EvictProblem(d["mass"], lens, 128, 2, 16, planes=(d["k"], d["v"]))
    src = torch.empty((20, 1, 128), dtype=torch.int32, device="cuda")

    def step():
        B.attn_shared(p, out, lse, d["mass"], ws)
        B.cache_evict(e, src)

    start = [x.clone() for x in (d["mass"], d["k"], d["v"])]
    step()
    want = [x.clone() for x in (out, lse, d["mass"], src, d["k"], d["v"])]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.synchronize()
    for _ in range(3):
        for x, y in zip((d["mass"], d["k"], d["v"]), start):
            x.copy_(y)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip((out, lse, d["mass"], src, d["k"], d["v"]), want):
            assert torch.equal(x, y)
    assert B.device_error() == 0
