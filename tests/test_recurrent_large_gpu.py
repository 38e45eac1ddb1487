"""Sizes at which every thread or group of lanes takes several turns, outputs over inputs in long calls, rows beyond 4 GB (GPU)."""
import numpy as np
import pytest
import torch

import test_dropout_gpu as drop
import test_gated_scan_gpu as scan
import test_layer_norm_gpu as norm

from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


# the grids of 64 blocks an SM (152 of them) cover 19.9 M fp32 and 39.8 M 16-bit elements in a turn, 9.96 M where pointers are not aligned
@pytest.mark.parametrize("dtype,n,shift", [("f32", 45_000_003, 0), ("bf16", 85_000_001, 0), ("f16", 41_000_006, 0), ("f32", 23_000_001, 1),
                                           ("f16", 11_000_002, 1)])
def test_dropout_of_several_turns(dtype, n, shift):
    x, res, gy = drop.tensors(n, dtype, seed=3, shift=shift)
    rng, p = drop.state(drop.SEED, 7), 0.25
    keep = torch.from_numpy(drop.words(n, drop.SEED, 7, 5) >= np.uint64(2 ** 30)).cuda()
    out, gx = torch.empty_like(x), torch.empty_like(x)
    ops.vg_dropout_add_fwd(x, res, p, rng, 5, out)
    ops.vg_dropout_add_bwd(gy, p, rng, 5, gx)
    u, e = drop.U[dtype], 2.0 ** -24
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0         # half a step of fp16 below its normal numbers
    part = torch.where(keep, x.double() / (1 - p), 0.0)
    want = res.double() + part
    assert ((out.double() - want).abs() <= (u + e) * want.abs() + 2 * e * part.abs() + tiny).all()
    assert torch.equal(out[~keep], res[~keep])
    want = torch.where(keep, gy.double() / (1 - p), 0.0)
    assert ((gx.double() - want).abs() <= (u + 3 * e) * want.abs() + tiny).all()
    assert (gx[~keep] == 0).all()


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("n,c", [(100_003, 64), (50_001, 200), (30_001, 520), (20_001, 1024), (9_001, 2048), (5_003, 4096), (2_501, 8192)])
def test_norm_of_many_fp16_rows(n, c, skip):
    x = norm.make(n, c, "f16", skip=skip, seed=c)
    norm.compare(norm.call(x), norm.reference(x), "f16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,c", [([300], 40), ([5_000, 0, 3], 72), ([70_001], 16), ([60_000, 40_003], 136), ([250_001], 8)])
def test_scan_gradients_over_its_operands(dtype, lengths, c):
    """Each output in the place of an input, whichever."""
    x = scan.make(lengths, c, dtype, order=True, state=True, seed=c)
    want = scan.call(x)
    n, b, dt = sum(lengths), len(lengths), scan.DT[dtype]
    ws, kept = ops.gated_scan_workspace(n, c, b, dt), ops.gated_scan_carries(n, c)
    for over in ("gate", "x"):                                   # the forward's output
        t = {k: x[k].contiguous().clone() for k in ("gate", "x")}
        ops.vg_gated_scan_fwd(t["gate"], t["x"], x["offsets"], x["order"], x["first"], t[over], None, kept, ws)
        assert torch.equal(t[over], want["out"])
    for gg, gx in (("gate", "x"), ("x", "gate"), ("grad_out", "x"), ("gate", "grad_out")):
        t = {k: x[k].contiguous().clone() for k in ("gate", "x", "grad_out")}
        gf = x["grad_last"].clone()
        ops.vg_gated_scan_bwd(t["gate"], t["x"], x["offsets"], x["order"], x["first"], kept, t["grad_out"], x["grad_last"], t[gg],
                              t[gx], gf, ws)
        assert torch.equal(t[gg], want["grad_gate"]) and torch.equal(t[gx], want["grad_x"]), (gg, gx)
        assert torch.equal(gf, want["grad_first"])
    assert ops.vg_gated_scan_status(ws) == ops.VG_OK


def far_rows(n, c, columns, seed):
    """`columns` [n, c] views of one bf16 tensor whose rows reach beyond 4 GB, and contiguous copies of them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    stride = -(-(2 ** 32 + 2 ** 28) // (2 * n * 8)) * 8
    big = torch.empty(n, max(stride, columns * c), dtype=torch.bfloat16, device="cuda")
    views = [big[:, i * c:(i + 1) * c] for i in range(columns)]
    for v in views:
        v.copy_(torch.randn(n, c, generator=g, device="cuda"))
    return views, [v.contiguous() for v in views]


def test_rows_beyond_4_gb():
    n, c = 1_100_003, 16
    (gate, v, gy, out, gg, gx), (gate1, v1, gy1, out1, gg1, gx1) = far_rows(n, c, 6, 1)
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    order = torch.randperm(n, device="cuda").int()
    ws, kept = ops.gated_scan_workspace(n, c, 1, torch.bfloat16), ops.gated_scan_carries(n, c)
    for a, b, d, o, p, q in ((gate, v, gy, out, gg, gx), (gate1, v1, gy1, out1, gg1, gx1)):
        ops.vg_gated_scan_fwd(a, b, off, order, None, o, None, kept, ws)
        ops.vg_gated_scan_bwd(a, b, off, order, None, kept, d, None, p, q, None, ws)
    assert torch.equal(out, out1) and torch.equal(gg, gg1) and torch.equal(gx, gx1)
    state, state1 = (torch.zeros(n, c, device="cuda") for _ in range(2))
    ops.vg_gated_scan_step(gate, v, state, out)
    ops.vg_gated_scan_step(gate1, v1, state1, out1)
    assert torch.equal(out, out1) and torch.equal(state, state1)
    w, nws, r = torch.randn(c, device="cuda").bfloat16(), ops.layer_norm_workspace(n, c), []
    for a, d, o, p in ((v, gy, out, gx), (v1, gy1, out1, gx1)):
        stats, gw, gb = torch.empty(n, 2, device="cuda"), torch.empty_like(w), torch.empty_like(w)
        ops.vg_layer_norm_fwd(a, w, None, o, stats)
        ops.vg_layer_norm_bwd(a, w, stats, d, d, p, gw, gb, nws)
        r.append((o, p, gw, gb, stats))
    for s, t in zip(*r):
        assert torch.equal(s, t)
