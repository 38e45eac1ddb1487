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
