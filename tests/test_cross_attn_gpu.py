"""vg_cross_attn_fwd / _bwd against attention in 64 bits (GPU).

Bounds, as relative Frobenius errors.  fp32: 1e-5, the library's bound for exact
fp32.  16 bits, u = half an ulp (2^-8 bf16, 2^-11 fp16): an output carries one
rounding of the result and one of each score's weight, both at most u and
independent, and a gradient one more of the score gradients: 2 u and 3 u.  lse is
fp32 everywhere: 1e-5.  Score gradients are differences, P (dP - delta), so two
errors do not shrink with them and are added to their bounds: scores and lse hold
2^-24 of their own size each, a few of which reach P (|dP| + |delta|), and delta
comes from `out`, which is rounded: u |dO| |O| P.
"""
import math

import pytest
import torch

from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
OUT_TOL = {"f32": 1e-5, "f16": 2 * U["f16"], "bf16": 2 * U["bf16"]}
GRAD_TOL = {"f32": 1e-5, "f16": 3 * U["f16"], "bf16": 3 * U["bf16"]}
NAMES = ("out", "lse", "grad_q", "grad_k", "grad_v")


def offsets(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32).cuda()


def strided(n, h, d, dt, layout):
    """An uninitialised [n, h, d] view: tokens first, heads first, or one half of a packed projection."""
    if layout == "heads":
        return torch.empty(h, max(n, 1), d, dtype=dt, device="cuda")[:, :n].transpose(0, 1)
    if layout == "packed":
        return torch.empty(n, 2, h, d, dtype=dt, device="cuda")[:, 1]
    return torch.empty(n, h, d, dtype=dt, device="cuda")


def make(lq, lk, hq, hk, d, dtype, valid=None, layout="rows", seed=0, q_scale=1.0, g_scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nq, nk, dt = sum(lq), sum(lk), DT[dtype]
    x = {}
    for name, n, h, s in (("q", nq, hq, q_scale), ("k", nk, hk, 1.0), ("v", nk, hk, 1.0), ("go", nq, hq, g_scale)):
        x[name] = strided(n, h, d, dt, layout)
        x[name].copy_(torch.randn(n, h, d, generator=g, device="cuda") * s)
    x.update(lq=lq, lk=lk, valid=list(lk) if valid is None else valid, q_off=offsets(lq), k_off=offsets(lk),
             k_lens=None if valid is None else torch.tensor(valid, dtype=torch.int32).cuda(), layout=layout,
             scale=d ** -0.5, dtype=dtype)
    return x


def call(x, backward=True, ws=None):
    """The operator's outputs, each written over NaN."""
    (nq, hq, d), (nk, hk, _), dt = x["q"].shape, x["k"].shape, x["q"].dtype
    if ws is None:
        ws = ops.cross_attn_workspace(nq, nk, len(x["lq"]), hq, hk, d, dt, backward=backward)
    r = {"out": strided(nq, hq, d, dt, x["layout"]), "lse": torch.empty(hq, nq, device="cuda"),
         "grad_q": strided(nq, hq, d, dt, x["layout"]), "grad_k": strided(nk, hk, d, dt, x["layout"]),
         "grad_v": strided(nk, hk, d, dt, x["layout"])}
    for t in r.values():
        t.fill_(math.nan)
    pos = (x["q"], x["k"], x["v"], x["q_off"], x["k_off"], x["k_lens"])
    ops.vg_cross_attn_fwd(*pos, r["out"], r["lse"], ws, scale=x["scale"])
    if backward:
        ops.vg_cross_attn_bwd(*pos, r["out"], r["lse"], x["go"], r["grad_q"], r["grad_k"], r["grad_v"], ws,
                              scale=x["scale"])
    r["status"] = ops.vg_cross_attn_status(ws)
    return r


def reference(x):
    """The formulas, sample by sample and head by head, in 64 bits."""
    q, k, v, go = (x[n].double() for n in ("q", "k", "v", "go"))
    group = q.shape[1] // k.shape[1]
    r = {"slack_q": 0.0, "slack_k": 0.0, "out": torch.zeros_like(q), "grad_q": torch.zeros_like(q),
         "grad_k": torch.zeros_like(k),
         "grad_v": torch.zeros_like(v),
         "lse": torch.full((q.shape[1], q.shape[0]), -math.inf, dtype=torch.float64, device="cuda")}
    a = b = 0
    for n, rows, m in zip(x["lq"], x["lk"], x["valid"]):
        for h in range(q.shape[1] if n and m else 0):
            qs, ks, vs, gs = q[a:a + n, h], k[b:b + m, h // group], v[b:b + m, h // group], go[a:a + n, h]
            s = qs @ ks.T * x["scale"]
            r["lse"][h, a:a + n] = s.logsumexp(1)
            p = s.softmax(1)
            o = p @ vs
            ds = p * (gs @ vs.T - (gs * o).sum(1, keepdim=True)) * x["scale"]
            r["out"][a:a + n, h] = o
            r["grad_q"][a:a + n, h] = ds @ ks
            r["grad_k"][b:b + m, h // group] += ds.T @ qs
            r["grad_v"][b:b + m, h // group] += p.T @ gs
            # what the cancellation in ds does not shrink
            e32 = 2.0 ** -22 * (1 + s.abs().nan_to_num(0, 0, 0).max())
            loose = e32 * p * ((gs @ vs.T).abs() + (gs * o).sum(1, keepdim=True).abs()) * x["scale"]
            turn = U.get(x["dtype"], 0.0) * (gs * o).abs().sum(1, keepdim=True) * x["scale"]
            r["slack_q"] += float((loose @ ks.abs()).norm() ** 2 + (turn * (p @ ks)).norm() ** 2)
            r["slack_k"] += float((loose.T @ qs.abs()).norm() ** 2 + (p.T @ (turn * qs)).norm() ** 2)
        a, b = a + n, b + rows
    return r


def rel(a, b, slack=0.0):
    """Relative error, of what is beyond the slack (2-norms)."""
    a, b = a.double(), b.double()
    fine = b.isfinite()
    assert torch.equal(fine, a.isfinite()) and torch.equal(a[~fine], b[~fine])
    n, err = b[fine].norm(), float((a[fine] - b[fine]).norm())
    return max(0.0, err - slack) / float(n if n > 0 else 1.0)


def compare(r, ref, dtype, names=NAMES):
    assert r["status"] == ops.VG_OK
    for n in names:
        tol = 1e-5 if n == "lse" else OUT_TOL[dtype] if n == "out" else GRAD_TOL[dtype]
        e = rel(r[n], ref[n], {"grad_q": ref["slack_q"], "grad_k": ref["slack_k"]}.get(n, 0.0) ** 0.5)
        assert e <= tol, (n, e, tol)


SHAPES = [
    # queries, key rows, query heads, key heads, width
    ([1], [1], 1, 1, 64),
    ([1, 1, 1], [77, 0, 5], 8, 8, 64),                 # single tokens, one sample without states
    ([0, 5, 130], [7, 0, 257], 4, 2, 64),              # no queries; no keys; ragged tails
    ([127, 128, 129], [63, 64, 65], 2, 1, 128),
    ([255, 256, 257], [127, 128, 129], 3, 3, 64),
    ([300], [1000], 6, 2, 40),                         # three heads a key head: not packed
    ([33, 65], [200, 31], 16, 1, 64),                  # sixteen heads a key head
    ([50], [90], 32, 1, 32),                           # more than sixteen
    ([70, 3], [150, 129], 4, 4, 8),
    ([70, 3], [150, 129], 4, 1, 24),
    ([200], [333], 2, 2, 72),
    ([200], [333], 2, 1, 96),
    ([2] * 70, [3] * 35 + [0] * 5 + [4] * 30, 2, 2, 64),   # more samples than a warp has lanes
    ([1000, 24], [1370, 1370], 2, 2, 64),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lq,lk,hq,hk,d", SHAPES)
def test_against_64_bits(dtype, lq, lk, hq, hk, d):
    x = make(lq, lk, hq, hk, d, dtype, seed=d + len(lq))
    compare(call(x), reference(x), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["heads", "packed"])
@pytest.mark.parametrize("d", [64, 80])
def test_layouts(dtype, layout, d):
    x = make([150, 40], [100, 300], 4, 2, d, dtype, layout=layout, seed=3)
    compare(call(x), reference(x), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lq,lk,hq,hk,d", [
    ([3, 1], [20001, 700], 4, 2, 64),          # few queries: the keys are cut into parts, some without keys
    ([1], [30000], 16, 4, 128),
    ([9000, 1], [10, 0], 2, 2, 64),            # few keys: the queries are cut
    ([7000], [130], 8, 2, 128),
])
def test_split_axes(dtype, lq, lk, hq, hk, d):
    x = make(lq, lk, hq, hk, d, dtype, seed=5)
    compare(call(x), reference(x), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_padded_rows_are_never_used(dtype, d):
    lk, valid = [300, 300, 300, 140], [1, 0, 300, 129]
    x = make([200, 5, 64, 129], lk, 4, 2, d, dtype, valid=valid, seed=7)
    at = 0
    for rows, m in zip(lk, valid):          # what lies past the valid rows is not a number
        x["k"][at + m:at + rows] = math.nan
        x["v"][at + m:at + rows] = math.inf
        at += rows
    compare(call(x), reference(x), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_samples_do_not_touch_one_another(dtype):
    """A sample of NaN between two others: the others get, bit for bit, what they get beside a clean one."""
    clean = make([100, 70, 45], [90, 33, 150], 4, 2, 64, dtype, seed=11)
    want = call(clean)
    dirty = dict(clean)
    for n in ("q", "k", "v", "go"):
        dirty[n] = clean[n].clone()
    dirty["q"][100:170] = dirty["go"][100:170] = math.nan
    dirty["k"][90:123] = dirty["v"][90:123] = math.nan
    got = call(dirty)
    keep_q, keep_k = [slice(0, 100), slice(170, 215)], [slice(0, 90), slice(123, 273)]
    for s in keep_q:
        for n in ("out", "grad_q"):
            assert torch.equal(got[n][s], want[n][s]), n
        assert torch.equal(got["lse"][:, s], want["lse"][:, s])
    for s in keep_k:
        for n in ("grad_k", "grad_v"):
            assert torch.equal(got[n][s], want[n][s]), n
    assert got["out"][100:170].isnan().all() and got["grad_q"][100:170].isnan().all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_growing_scores(dtype, d):
    """Keys whose scores grow along the sequence, by far more than exp can hold: the running maximum is replaced
    again and again, and the last key takes nearly all of the weight."""
    x = make([130], [700], 2, 2, d, dtype, seed=13)
    x["q"][:] = 0
    x["q"][:, :, 0] = torch.linspace(0.5, 8, 130, device="cuda")[:, None]
    x["k"][:, :, 0] = torch.linspace(-40, 40, 700, device="cuda")[:, None]
    x["scale"] = 1.0
    compare(call(x), reference(x), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_scores_of_minus_infinity(dtype):
    """Keys that no query can reach weigh nothing, wherever they stand; a row with no others is NaN, as in the
    formula."""
    x = make([40, 40], [300, 20], 2, 2, 64, dtype, seed=17)
    x["q"][:, :, 0] = 1.0
    x["k"][:200, :, 0] = -math.inf           # whole tiles of them first
    x["k"][300:, :, 0] = -math.inf           # the second sample has only such keys
    got, ref = call(x, backward=False), reference(x)
    assert got["status"] == ops.VG_OK
    assert rel(got["out"][:40], ref["out"][:40]) <= OUT_TOL[dtype]
    assert rel(got["lse"][:, :40], ref["lse"][:, :40]) <= 1e-5
    assert got["out"][40:].isnan().all() and (got["lse"][:, 40:] == -math.inf).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("g_scale", [1e-6, 1.0, 1e3])
def test_gradient_scales(dtype, g_scale):
    """Score gradients far from 1 (many keys, small or large incoming gradients) keep their precision in 16 bits."""
    x = make([40], [4096], 2, 1, 64, dtype, seed=19, q_scale=0.2, g_scale=g_scale)
    # results below fp16's normal range cannot hold their own rounding: compare what can
    ref = reference(x)
    names = [n for n in NAMES if dtype == "bf16" or n in ("out", "lse") or ref[n].abs().median() > 2.0 ** -11]
    assert dtype == "bf16" or g_scale < 1e3 or "grad_q" in names
    compare(call(x), ref, dtype, names)


def test_gradients_against_differences():
    """Central differences of sum(out * go) along random directions, in fp32: truncation h^2 and rounding
    1e-7 / h of values of order 1, so 1e-3 of the directional derivative's own scale at h = 1e-2."""
    x = make([40, 9], [70, 33], 4, 2, 64, "f32", seed=23)
    r = call(x)
    g = torch.Generator(device="cuda").manual_seed(1)
    for name in ("q", "k", "v"):
        for _ in range(3):
            dirn = torch.randn(x[name].shape, generator=g, device="cuda")
            sides = []
            for h in (1e-2, -1e-2):
                y = dict(x)
                y[name] = x[name] + h * dirn
                sides.append((call(y, backward=False)["out"].double() * x["go"].double()).sum())
            diff = float(sides[0] - sides[1]) / 2e-2
            grad = r["grad_" + name].double()
            want = float((grad * dirn.double()).sum())
            assert abs(diff - want) <= 1e-3 * float(grad.norm()) * math.sqrt(2) + 1e-3 * abs(want), (name, diff, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_same_from_run_to_run(dtype):
    for shape in (([500, 300], [700, 1100], 4, 2, 64), ([2], [9000], 8, 2, 64), ([4000], [70], 4, 2, 128)):
        x = make(*shape, dtype, seed=29)
        a, b = call(x), call(x)
        for n in NAMES:
            assert torch.equal(a[n], b[n]), (shape, n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_lse_and_on_another_stream(dtype):
    x = make([100, 3], [257, 40], 4, 2, 64, dtype, seed=31)
    want = call(x, backward=False)
    s = torch.cuda.Stream()
    out = torch.empty_like(want["out"])
    ws = ops.cross_attn_workspace(103, 297, 2, 4, 2, 64, DT[dtype])
    s.wait_stream(torch.cuda.current_stream())
    ops.vg_cross_attn_fwd(x["q"], x["k"], x["v"], x["q_off"], x["k_off"], None, out, None, ws, stream=s)
    assert ops.vg_cross_attn_status(ws, stream=s) == ops.VG_OK
    assert torch.equal(out, want["out"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["start", "end", "order", "keys end", "long", "negative"])
def test_bad_offsets_write_nothing(dtype, what):
    x = make([100, 60], [50, 90], 4, 2, 64, dtype, seed=37)
    good = call(x)
    y = dict(x)
    if what in ("start", "end", "order"):
        y["q_off"] = torch.tensor({"start": [1, 100, 160], "end": [0, 100, 170], "order": [0, 161, 160]}[what],
                                  dtype=torch.int32).cuda()
    elif what == "keys end":
        y["k_off"] = torch.tensor([0, 50, 139], dtype=torch.int32).cuda()
    else:
        y["k_lens"] = torch.tensor({"long": [51, 90], "negative": [50, -1]}[what], dtype=torch.int32).cuda()
    ws = ops.cross_attn_workspace(160, 140, 2, 4, 2, 64, DT[dtype], backward=True)
    got = call(y, ws=ws)
    assert got["status"] == ops.VG_ERR_INVALID_ARG
    for n in NAMES:
        assert got[n].isnan().all(), n
    again = call(x, ws=ws)                      # the record was cleared; the workspace serves the next call
    assert again["status"] == ops.VG_OK
    for n in NAMES:
        assert torch.equal(again[n], good[n]), n


@pytest.mark.parametrize("nq,nk", [(0, 40), (40, 0), (0, 0)])
def test_empty_sides(nq, nk):
    for dtype in ("f32", "bf16"):
        x = make([nq], [nk], 4, 2, 64, dtype)
        r = call(x)
        assert r["status"] == ops.VG_OK
        assert not r["out"].any() and not r["grad_q"].any() and not r["grad_k"].any() and not r["grad_v"].any()
        assert (r["lse"] == -math.inf).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_few_keys_keep_delta_exact(dtype, d):
    """Over few keys `out` is as large as V, and delta taken from the rounded `out` would add as much error as the
    rounding of dS.  Two independent roundings are left, of dS and of the result.  One has a relative root mean square
    of u 0.736 / sqrt(3) (uniform within half an ulp, mantissas m with E[1/m^2] = 3 / (8 ln 2)); 10 % for the sample.
    """
    x = make([403] * 5, [2, 3, 5, 17, 120], 8, 4, d, dtype, seed=5)
    r, ref = call(x), reference(x)
    bound = 1.1 * math.sqrt(2) * U[dtype] * 0.736 / math.sqrt(3)
    a = b = 0
    for n, m in zip(x["lq"], x["lk"]):
        assert rel(r["grad_q"][a:a + n], ref["grad_q"][a:a + n]) < bound
        assert rel(r["grad_k"][b:b + m], ref["grad_k"][b:b + m]) < bound
        a, b = a + n, b + m
