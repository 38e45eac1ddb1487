"""vg_gated_scan_fwd / _bwd at lengths that give a warp 4, 8 and 16 runs of 16 tokens, and thousands of tiles, against the
recurrence in 64 bits (GPU).

Bounds, as relative Frobenius errors.  A gate's error moves a state by about twice its share, 3e-6 in all.  A state's own
roundings, two a token and 2^-24 each, are forgotten with its memory, here below 250 tokens on average: sqrt(500) 2^-24
of them if they are as good as random, 1.4e-6.  A token's map passes through the maps of its warp's tokens in the same way, 8 warps,
and 40 folded tiles or the join's 8 doublings and twice 9 tiles a thread, of which tiles beyond the memory no longer count: at
most 50 roundings, 3e-6.  Together below 1e-5; a gradient of the gate has both chains and two products, 2e-5.  A
16-bit result has one rounding more, u (the bounds of `compare`).
"""
import numpy as np
import pytest
import torch

from test_gated_scan_gpu import DT, F, R, call, compare, make, reference
from test_recurrent_edges_gpu import exact_ws, fenced

from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


def chain(a, b, place):
    """h of h <- a h + b from 0 at each sequence's place 0, by maps of 1, 2, 4 .. tokens."""
    d, far = 1, int(place.max()) + 1
    a, b = a.clone(), b.clone()
    while d < far:
        have = (place[d:] >= d)[:, None]
        nb = b[d:] + torch.where(have, a[d:] * b[:-d], 0.0)
        na = torch.where(have, a[d:] * a[:-d], a[d:])
        a[d:], b[d:] = na, nb
        d *= 2
    return b


def long_reference(x, flags):
    n, c = x["x"].shape
    lens = torch.tensor(x["lengths"], device="cuda")
    b = lens.numel()
    rows = torch.arange(n, device="cuda") if x["order"] is None else x["order"].long()
    seq = torch.repeat_interleave(torch.arange(b, device="cuda"), lens)
    at = torch.arange(n, device="cuda") - (lens.cumsum(0) - lens)[seq]
    left = lens[seq] - 1 - at
    if flags & R:                                # visits in the order of time: all reversed, sequences too
        rows, seq, at, left = rows.flip(0), seq.flip(0), left.flip(0), at.flip(0)
    gate, v, gy = (x[k].double()[rows] for k in ("gate", "x", "grad_out"))
    zero = torch.zeros(b, c, dtype=torch.float64, device="cuda")
    h0 = zero if x["first"] is None else x["first"].double()
    gl = zero if x["grad_last"] is None else x["grad_last"].double()
    a, s = torch.sigmoid(gate), torch.sigmoid(-gate)
    take = v if flags & F else s * v
    start, stop = (at == 0), (left == 0)
    take = take + torch.where(start[:, None], a * h0[seq], 0.0)
    h = chain(a, take, at)
    before = torch.cat([h[:1], h[:-1]])
    before[start] = h0[seq[start]]
    r = {k: torch.empty(n, c, dtype=torch.float64, device="cuda") for k in ("out", "grad_gate", "grad_x")}
    r["last"], r["grad_first"] = h0.clone(), gl.clone()
    r["out"][rows] = h
    r["last"][seq[stop]] = h[stop]
    up = gy + torch.where(stop[:, None], gl[seq], 0.0)
    lam = chain(torch.cat([a[1:], a[:1]]).flip(0), up.flip(0), left.flip(0)).flip(0)
    r["grad_first"][seq[start]] = (a * lam)[start]
    r["grad_x"][rows] = lam if flags & F else lam * s
    r["grad_gate"][rows] = lam * (before if flags & F else before - v) * a * s
    return r


@pytest.mark.parametrize("flags", [0, R, F, R | F])
def test_the_reference(flags):
    for lengths in ([300], [40, 0, 1, 77, 0]):
        x = make(lengths, 8, "f32", order=True, state=True, seed=1)
        want = reference(x, flags)
        for k, v in long_reference(x, flags).items():
            assert (v - want[k]).abs().max() <= 1e-12 * want[k].abs().max(), k


# runs a warp takes (152 SMs), forward and backward: 4; 8; 16; 16, ragged; 8 (fp32: 16), blocks of channels beside one another; 16 (8);
# 8 forward and 16 of more than 2048 tiles; 4, sequences of some tens of tokens
LONG = [([120_001], 8), ([250_001], 16), ([467_003], 8), ([300_007, 0, 160_000, 6_993, 1, 17], 24), ([60_000, 40_003], 136),
        ([199_999, 5, 130], 136), ([2_200_003], 8), ([4_300_001], 8), ([61, 3, 0, 17, 64, 1] * 900, 8)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("reverse", [0, R])
@pytest.mark.parametrize("lengths,c", LONG)
def test_long_scans(dtype, reverse, lengths, c):
    k = len(lengths) + c + (reverse > 0)
    flags = reverse | (F if k % 4 == 1 else 0)
    x = make(lengths, c, dtype, order=k % 3 != 0, state=k % 2 == 0, seed=k, memory=(0.0, 5.0) if flags & F else (0.0, 6.0))
    compare(call(x, flags), long_reference(x, flags), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,batch", [(5_000, 40, 3), (5_000, 16, 100), (70_001, 16, 3), (70_001, 16, 100), (300_000, 136, 40)])
@pytest.mark.parametrize("reverse", [0, R])
def test_bad_offsets_of_many_tiles_write_nothing(dtype, n, c, batch, reverse):
    """The maps' and the join's steps walk the offsets before the last step knows that they are bad."""
    x = make([n // batch] * (batch - 1) + [n - n // batch * (batch - 1)], c, dtype, state=True, seed=batch)
    good, dt = x["offsets"].tolist(), DT[dtype]
    rng = np.random.default_rng(n + batch)
    mid = batch // 2
    bads = [good[:mid] + [good[mid - 1] - 1] + good[mid + 1:], good[:-1] + [n - 1], [1] + good[1:], good[:-1] + [n + 7],
            good[:mid] + [-5] + good[mid + 1:], good[:mid] + [2 ** 31 - 1] + good[mid + 1:], [-2 ** 31] + good[1:],
            good[::-1], rng.permutation(good).tolist(), rng.integers(-2 ** 31, 2 ** 31, batch + 1).tolist()]
    ws, ws_ok = exact_ws(ops.gated_scan_workspace(n, c, batch, dt).numel())
    kept, kept_ok = fenced(tuple(ops.gated_scan_carries(n, c).shape), torch.float32, rows_before=4)
    want = call(x, reverse)
    for bad in bads:
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        outs = {k: fenced((n, c), dt) for k in ("out", "gg", "gx")}
        outs |= {k: fenced((batch, c), torch.float32, rows_before=4) for k in ("last", "gf")}
        o = {k: v[0] for k, v in outs.items()}
        kept.fill_(7)
        ops.vg_gated_scan_fwd(x["gate"], x["x"], off, None, x["first"], o["out"], o["last"], kept, ws, flags=reverse)
        assert ops.vg_gated_scan_status(ws) == ops.VG_ERR_INVALID_ARG
        ops.vg_gated_scan_bwd(x["gate"], x["x"], off, None, x["first"], kept, x["grad_out"], x["grad_last"], o["gg"], o["gx"],
                              o["gf"], ws, flags=reverse)
        assert ops.vg_gated_scan_status(ws) == ops.VG_ERR_INVALID_ARG
        for k, (t, around) in outs.items():
            assert (t == 7).all(), k
            around()
        assert (kept == 7).all()
        kept_ok()
        ws_ok()
    got = call(x, reverse, ws=ws)               # the workspace serves again
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_one_workspace_for_all_lengths():
    """A workspace of the most rows serves calls of fewer, some of which are cut into more parts."""
    c, dt = 64, torch.bfloat16
    ws, ws_ok = exact_ws(ops.gated_scan_workspace(467_000, c, 1, dt).numel())
    for n in (467_000, 389_000, 120_001, 40_000, 2_049, 1):
        x = make([n], c, "bf16", state=True, seed=n)
        want, got = call(x), call(x, ws=ws)
        for k in want:
            assert torch.equal(got[k], want[k]), (n, k)
    ws_ok()
