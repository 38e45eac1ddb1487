"""vg_cross_attn_fwd / _bwd where values are not finite, far apart or many (GPU).

Bounds not named here are those of test_cross_attn_gpu.py.
"""
import math

import pytest
import torch

import test_cross_attn_gpu as base
from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

make, call, reference, rel, compare = base.make, base.call, base.reference, base.rel, base.compare
TYPES = ["f32", "f16", "bf16"]


# ------------------------------------------------------------------ values that are not finite, in a cut axis
def key_parts(x):
    """Parts of the key axis in the forward pass, from the workspace: one output row and log-sum each."""
    (nq, hq, d), (nk, hk, _) = x["q"].shape, x["k"].shape
    nb = ops.cross_attn_workspace(nq, nk, len(x["lq"]), hq, hk, d, x["q"].dtype).numel() - 256
    return max(1, nb // (nq * hq * (d + 1) * 4))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lq,lk,hq,hk,least", [
    ([1] * 4, [20000] * 4, 8, 8, 9),         # one query a sample: one part for each lane of the join, and a few more
    ([1], [30000], 4, 2, 17),                # several parts for every lane
    ([100, 30], [450, 350], 4, 2, 2),        # few parts
])
@pytest.mark.parametrize("what", ["nan key", "inf key", "nan value far down", "inf value far down",
                                  "nan value at weight zero"])
def test_not_finite_in_a_part(dtype, lq, lk, hq, hk, least, what):
    """One key or value that is not finite, in each part in turn: the outputs that it belongs to are not finite either
    (a weight however small times it), all others the same bits as without it."""
    x = make(lq, lk, hq, hk, 64, dtype, seed=41)
    x["q"][:, :, 0] = 1.0                    # scores can be moved by channel 0 alone
    parts, n = key_parts(x), lk[0]
    assert parts >= least
    head, rows = hk - 1, slice(0, lq[0])
    heads = slice(head * (hq // hk), (head + 1) * (hq // hk))
    clean = call(x, backward=False)
    for p in range(min(parts, 40)):
        key = int((p + 0.5) * n / min(parts, 40))
        y = dict(x, k=x["k"].clone(), v=x["v"].clone())
        if what == "nan key":
            y["k"][key, head, 3] = math.nan
        elif what == "inf key":
            y["k"][key, head, 0] = math.inf
        else:                                # the keys around it, more than a part, weigh exp(-500) or nothing
            y["k"][max(0, key - n // 8):key + n // 8, head, 0] = -math.inf if what.endswith("zero") else -4000.0
            y["v"][key, head, 5] = math.inf if what.startswith("inf") else math.nan
        got, want = call(y, backward=False), clean
        assert got["status"] == ops.VG_OK
        if "value" in what:
            want = call(dict(y, v=x["v"]), backward=False)
            assert not got["out"][rows, heads, 5].isfinite().any(), key
            got["out"][rows, heads, 5] = want["out"][rows, heads, 5]
        else:
            assert got["out"][rows, heads].isnan().all() and got["lse"][heads, rows].isnan().all(), key
            got["out"][rows, heads], got["lse"][heads, rows] = want["out"][rows, heads], want["lse"][heads, rows]
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"]), key


@pytest.mark.parametrize("dtype", TYPES)
def test_no_keys_and_keys_of_weight_zero_in_cut_calls(dtype):
    """Beside a sample that is cut into parts: one without keys gives zeros, one with scores of -inf alone NaN."""
    x = make([2, 3, 1], [20000, 0, 5000], 4, 2, 64, dtype, seed=43)
    x["q"][:, :, 0] = 1.0
    x["k"][20000:, :, 0] = -math.inf
    assert key_parts(x) > 8
    r = call(x, backward=False)
    assert r["status"] == ops.VG_OK
    assert not r["out"][2:5].any() and (r["lse"][:, 2:5] == -math.inf).all()
    assert r["out"][5:].isnan().all() and (r["lse"][:, 5:] == -math.inf).all()
    assert r["out"][:2].isfinite().all() and r["lse"][:, :2].isfinite().all()


# ------------------------------------------------------------------ gradients of very different sizes
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("what", ["inf gradient", "large gradient", "inf value", "large value", "without keys"])
def test_a_sample_does_not_set_another_ones_scale(dtype, what):
    """Whatever stands in one sample, the gradients of the others are the same bits.  Beside something large the
    others are small (score gradients of 1e-3), beside something infinite large (of 10 and more)."""
    lk, size = [90, 0 if what == "without keys" else 200, 150], (0.1, 0.1) if "large" in what else (8.0, 1.0)
    clean = make([100, 70, 45], lk, 4, 2, 64, dtype, seed=47, g_scale=size[0])
    clean["v"].mul_(size[1])
    want = call(clean)
    dirty = dict(clean, go=clean["go"].clone(), v=clean["v"].clone())
    if what in ("inf gradient", "without keys"):
        dirty["go"][110, 1, 3] = math.inf
    elif what == "large gradient":
        dirty["go"][100:170] = 6e4
    elif what == "inf value":
        dirty["v"][100, 1, 7] = -math.inf
    else:
        dirty["v"][90:290] = 6e4
    got = call(dirty)
    assert got["status"] == want["status"] == ops.VG_OK
    k1 = 90 + lk[1]
    for s in (slice(0, 100), slice(170, 215)):
        for n in ("out", "grad_q"):
            assert torch.equal(got[n][s], want[n][s]), n
    for s in (slice(0, 90), slice(k1, k1 + 150)):
        for n in ("grad_k", "grad_v"):
            assert torch.equal(got[n][s], want[n][s]), n
    compare(want, reference(clean), dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("keys", [100, 4096])
def test_a_large_row_leaves_the_others_their_precision(dtype, keys):
    """A query whose incoming gradient is 3e6 times its neighbours': their gradients hold the bound among
    themselves.  (K is large, q small: results are far inside fp16's normal range and the weights are even.)"""
    x = make([130], [keys], 2, 1, 64, dtype, seed=53, q_scale=0.02, g_scale=1e-2)
    x["k"].mul_(16)
    x["go"][77] = 3e4
    r, ref = call(x), reference(x)
    assert r["status"] == ops.VG_OK
    others = torch.arange(130, device="cuda") != 77
    assert ref["grad_q"][others].abs().median() > 2.0 ** -11
    y = {n: (x[n][others].contiguous() if n in ("q", "go") else x[n]) for n in x}
    y.update(lq=[129], q_off=base.offsets([129]))
    slack = reference(y)["slack_q"] ** 0.5
    assert rel(r["grad_q"][others], ref["grad_q"][others], slack) <= base.GRAD_TOL[dtype]
    compare(r, ref, dtype, ("out", "lse", "grad_k", "grad_v"))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("g_scale", [1e-6, 1e-3, 1.0])
@pytest.mark.parametrize("name", ["grad_q", "grad_k"])
def test_small_gradients_over_many_keys(dtype, g_scale, name):
    """Score gradients of 1e-8 to 1e-2 (4,096 keys of even weight) keep their precision.  V, and the other operand
    of the product with them, are large, so that the result is a normal number of the type; q and K are balanced so
    that scores stay small."""
    x = make([40], [4096], 2, 1, 64, dtype, seed=59, g_scale=g_scale)
    x["v"].mul_(1e3 if g_scale < 1e-4 else 1.0)
    big, small = ("k", "q") if name == "grad_q" else ("q", "k")
    x[big].mul_(2e3 if g_scale < 1.0 else 2.0)
    x[small].mul_(1e-4 if g_scale < 1.0 else 0.1)
    ref = reference(x)
    assert ref["lse"].std() < 0.5                                # even weights
    assert 2.0 ** -11 < ref[name].abs().median() and ref[name].abs().max() < 3e4
    compare(call(x), ref, dtype, ("out", "lse", name))


# ------------------------------------------------------------------ sizes at which the plan changes
def plan(x):
    """What the sizes reach: SMs, blocks of two row tiles of queries, key tiles x heads, and the parts of the query
    axis in dK and dV, from the workspace (two fp32 gradients a part, beside the row statistics)."""
    (nq, hq, d), (nk, hk, _), batch = x["q"].shape, x["k"].shape, len(x["lq"])
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    group = hq // hk
    gp = group if group <= 16 and not group & (group - 1) else 1
    nb = ops.cross_attn_workspace(nq, nk, batch, hq, hk, d, x["q"].dtype, backward=True).numel()
    parts = max(1, (nb - 256 - 8 * nq * hq) // (2 * nk * hk * d * 4))
    return sms, (nq * gp // 256) * (hq // gp), (nk // 128) * hk, parts


ROUNDINGS = 1.1 * math.sqrt(2) * 0.736 / math.sqrt(3)
LARGE = [
    # queries, key rows, query heads, key heads, width, valid keys
    ([9101, 128, 3000, 1], [700, 1, 937, 65], 16, 16, 64, None),         # 6 and 8 key tiles, with tails
    ([6000, 4224, 2049], [900, 641, 768], 16, 8, 64, [900, 0, 651]),     # two heads a row; padded; one without keys
    ([12345], [1000], 8, 4, 40, None),
    ([3001, 4096], [700, 130], 8, 8, 128, None),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lq,lk,hq,hk,d,valid", LARGE)
def test_two_row_tiles_and_many_units(dtype, lq, lk, hq, hk, d, valid):
    """Calls whose forward blocks take two row tiles and whose blocks have several units each, so that every ring
    wraps and every accumulator is used again.  Two independent roundings (of the weights or score gradients, and of
    the result), of a relative root mean square of u 0.736 / sqrt(3) each; 10 % for the sample."""
    if valid:
        valid = [min(v, n) for v, n in zip(valid, lk)]
    x = make(lq, lk, hq, hk, d, dtype, valid=valid, seed=61)
    sms, row_units, key_units, _ = plan(x)
    assert row_units > 2 * sms or d == 128 and row_units > sms
    r, ref = call(x), reference(x)
    compare(r, ref, dtype)
    for n in ("out", "grad_q", "grad_k", "grad_v"):
        slack = {"grad_q": ref["slack_q"], "grad_k": ref["slack_k"]}.get(n, 0.0) ** 0.5
        assert rel(r[n], ref[n], slack) <= ROUNDINGS * base.U[dtype], n
    again = call(x)
    for n in base.NAMES:
        assert torch.equal(r[n], again[n]), n


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_growing_scores_in_two_row_tiles(dtype, d):
    """Scores that grow along the keys, by more than exp can hold, while both row tiles of a block are at work, and
    of which some row tiles have none."""
    x = make([5000, 130], [900, 300], 8, 8, d, dtype, seed=67)
    sms, row_units, _, _ = plan(x)
    assert row_units >= sms
    x["q"][:] = 0
    x["q"][:, :, 0] = torch.linspace(0.5, 8, 5130, device="cuda")[:, None]
    x["q"][2000:2100] = 0                       # rows whose maximum never moves, beside others'
    x["k"][:900, :, 0] = torch.linspace(-40, 40, 900, device="cuda")[:, None]
    x["scale"] = 1.0
    compare(call(x), reference(x), dtype)


@pytest.mark.parametrize("dtype,hq,hk", [("bf16", 16, 16), ("f16", 16, 16), ("bf16", 32, 16)])
def test_key_gradients_cut_to_even_waves(dtype, hq, hk):
    """So many steps that the query axis of dK and dV is cut although there are as many key tiles as SMs."""
    lq = [20011, 15000] if hq == hk else [10011, 7500]
    x = make(lq, [800, 571], hq, hk, 64, dtype, seed=71)
    sms, _, key_units, parts = plan(x)
    assert key_units >= sms and parts > 1
    r, ref = call(x), reference(x)
    compare(r, ref, dtype)
    for n in ("out", "grad_q", "grad_k", "grad_v"):
        slack = {"grad_q": ref["slack_q"], "grad_k": ref["slack_k"]}.get(n, 0.0) ** 0.5
        assert rel(r[n], ref[n], slack) <= ROUNDINGS * base.U[dtype], n


@pytest.mark.parametrize("dtype", TYPES)
def test_thousands_of_samples(dtype):
    """3,000 small samples, some without queries or without keys."""
    lq, lk = [(5 * i) % 7 for i in range(3000)], [(11 * i + 3) % 23 for i in range(3000)]
    x = make(lq, lk, 2, 1, 32, dtype, seed=73)
    r = call(x)
    # the samples side by side, padded: [sample, head, query, key]
    nq, nk, b = sum(lq), sum(lk), len(lq)
    rows = torch.full((b, max(lq)), nq, device="cuda")
    keys = torch.full((b, max(lk)), nk, device="cuda")
    for i in range(b):
        rows[i, :lq[i]] = torch.arange(int(x["q_off"][i]), int(x["q_off"][i]) + lq[i], device="cuda")
        keys[i, :lk[i]] = torch.arange(int(x["k_off"][i]), int(x["k_off"][i]) + lk[i], device="cuda")
    leaf = {n: x[n].double().requires_grad_() for n in ("q", "k", "v")}
    pad = lambda t: torch.cat([t, t.new_zeros(1, *t.shape[1:])])  # noqa: E731
    q, k, v = pad(leaf["q"])[rows], pad(leaf["k"])[keys][:, :, 0], pad(leaf["v"])[keys][:, :, 0]
    s = torch.einsum("bihd,bjd->bhij", q, k) * x["scale"]
    s = s.masked_fill((keys == nk)[:, None, None, :], -1e30)
    p = s.softmax(-1) * (keys < nk)[:, None, None, :]
    o = torch.einsum("bhij,bjd->bihd", p, v)
    out = torch.zeros(nq + 1, 2, 32, dtype=torch.float64, device="cuda").index_put((rows,), o)[:nq]
    out.backward(x["go"].double())
    assert r["status"] == ops.VG_OK
    # a sample's one key has no score gradient at all, and what rounding leaves is of the size of the others' error
    for n, want in (("out", out.detach()), ("grad_q", leaf["q"].grad), ("grad_k", leaf["k"].grad),
                    ("grad_v", leaf["v"].grad)):
        assert rel(r[n], want) <= (base.OUT_TOL if n == "out" else base.GRAD_TOL)[dtype], n


@pytest.mark.parametrize("dtype,size", [("bf16", 1e24), ("f32", 1e24), ("f16", 3e3)])
@pytest.mark.parametrize("queries", [3, 5000])
def test_large_values_under_growing_scores(dtype, size, queries):
    """Scores that pass the first tile's by up to 40, and values as large as the type's range allows sums of: weights
    are kept small enough for their products with them."""
    x = make([queries], [900], 8, 8, 64, dtype, seed=79)
    x["q"][:] = 0
    x["q"][:, :, 0] = 1
    x["k"][:, :, 0] = torch.linspace(0, 40, 900, device="cuda")[:, None]
    x["scale"] = 1.0
    x["v"].mul_(size)
    compare(call(x, backward=False), reference(x), dtype, ("out", "lse"))
