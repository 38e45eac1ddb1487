"""Argument checks of the recurrent-block operators: refused on the host, before any launch (CPU only).

Pointers here are made-up addresses that a refused call never follows.
"""
import ctypes

import pytest
import torch

from test_binding_devices import gpu, refused

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def ops():
    from voxel_gemm_gb300 import build, ops
    build.build()
    return ops


def rows(ops, data=4096, stride=64):
    return ops.RowsStruct(data, stride)


def norm(ops, bwd, n=10, c=64, dtype=1, x="ok", w=4096, b=4096, eps=1e-5, y="ok", stats=4096, gy="ok", skip=None,
         gw=4096, gb=4096, ws=4096, nbytes=1 << 30):
    r = rows(ops, stride=max(c, 8))
    x, y, gy = (r if isinstance(t, str) else t for t in (x, y, gy))
    L = ops.lib()
    if not bwd:
        return L.vg_layer_norm_fwd(n, c, dtype, x, P(w), P(b), eps, y, P(stats), None)
    return L.vg_layer_norm_bwd(n, c, dtype, x, P(w), P(stats), gy, skip, y, P(gw), P(gb), P(ws), nbytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(c=0), 1), (dict(c=-8), 1), (dict(dtype=3), 1), (dict(c=60), 5),
    (dict(c=8200), 5), (dict(x=None), 1), (dict(y=None), 1), (dict(w=4100), 1), (dict(stats=4100), 1)])
def test_norm_refusals(ops, change, status):
    assert norm(ops, False, **change) == norm(ops, True, **change) == status


def test_norm_refusals_of_one_pass(ops):
    bad = ops.VG_ERR_INVALID_ARG
    for eps in (-1.0, float("nan"), float("inf")):
        assert norm(ops, False, eps=eps) == bad
    assert norm(ops, False, b=4104) == bad
    assert norm(ops, True, stats=None) == norm(ops, True, gy=None) == norm(ops, True, ws=None) == bad
    assert norm(ops, True, ws=4097) == norm(ops, True, gw=4104) == norm(ops, True, gb=4104) == bad
    need = ops.lib().vg_layer_norm_workspace_bytes(10, 64)
    assert need > 0 and norm(ops, True, nbytes=need - 1) == ops.VG_ERR_WORKSPACE_TOO_SMALL
    for r in (rows(ops, 4104), rows(ops, 0), rows(ops, stride=32), rows(ops, stride=68), rows(ops, stride=-64),
              rows(ops, stride=1 << 60)):
        assert norm(ops, False, x=r) == norm(ops, False, y=r) == bad
        assert norm(ops, True, x=r) == norm(ops, True, y=r) == norm(ops, True, gy=r) == norm(ops, True, skip=r) == bad
    assert norm(ops, False, n=0, x=None, y=None) == ops.VG_OK            # nothing is looked at or launched
    assert norm(ops, True, n=0, x=None, y=None, gy=None, gw=None, gb=None, ws=None) == ops.VG_OK
    for n, c in ((-1, 64), (10, 60), (10, 8200), (1 << 31, 64)):
        assert ops.lib().vg_layer_norm_workspace_bytes(n, c) == 0


def scan(ops, **kw):
    d = dict(n=10, channels=64, batch=2, dtype=2, flags=0, offsets=4096, order=None)
    d.update(kw)
    return ops.ScanStruct(*(d[f] for f, _ in ops.ScanStruct._fields_))


def scan_call(ops, s, bwd, gate="ok", x="ok", first=None, out="ok", last=1 << 20, kept=4096, gy="ok", gl=None, gg="ok",
              ws=4096, nbytes=1 << 30):
    r = rows(ops)
    gate, x, out, gy, gg = (r if isinstance(t, str) else t for t in (gate, x, out, gy, gg))
    L = ops.lib()
    if not bwd:
        return L.vg_gated_scan_fwd(s, gate, x, P(first), out, P(last), P(kept), P(ws), nbytes, None)
    return L.vg_gated_scan_bwd(s, gate, x, P(first), P(kept), gy, P(gl), gg, out, P(last), P(ws), nbytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(channels=0), 1), (dict(channels=60), 5), (dict(channels=65544), 5),
    (dict(batch=0), 1), (dict(batch=-1), 1), (dict(dtype=7), 1), (dict(flags=0x1), 5), (dict(offsets=None), 1),
    (dict(offsets=4098), 1), (dict(order=4098), 1)])
def test_scan_refusals(ops, change, status):
    s = scan(ops, **change)
    assert scan_call(ops, s, False) == scan_call(ops, s, True) == status
    if not {"offsets", "order"} & set(change):
        assert ops.lib().vg_gated_scan_workspace_bytes(s) == 0


def test_scan_operands(ops):
    bad, s, L = ops.VG_ERR_INVALID_ARG, scan(ops), ops.lib()
    for r in (None, rows(ops, 4104), rows(ops, 0), rows(ops, stride=32), rows(ops, stride=68)):
        for what in ("gate", "x", "out"):
            assert scan_call(ops, s, False, **{what: r}) == scan_call(ops, s, True, **{what: r}) == bad
        assert scan_call(ops, s, True, gy=r) == scan_call(ops, s, True, gg=r) == bad
    for kw in (dict(first=4104), dict(last=4104), dict(kept=4104), dict(ws=None), dict(ws=4097),
               dict(first=1 << 20), dict(first=(1 << 20) + 256), dict(first=(1 << 20) - 256)):  # over `last`
        assert scan_call(ops, s, False, **kw) == scan_call(ops, s, True, **kw) == bad, kw
    assert scan_call(ops, s, True, kept=None) == scan_call(ops, s, True, gl=4104) == bad
    assert scan_call(ops, s, True, gl=1 << 20) == bad                     # the states' gradients over one another
    big = scan(ops, n=100_000)
    need = L.vg_gated_scan_workspace_bytes(big)
    assert need > 256
    for bwd in (False, True):
        assert scan_call(ops, big, bwd, nbytes=need - 1) == ops.VG_ERR_WORKSPACE_TOO_SMALL
    assert L.vg_gated_scan_workspace_bytes(None) == 0 and L.vg_gated_scan_status(None, None) == bad
    assert [L.vg_gated_scan_carry_rows(n) for n in (-5, 0, 1, 16, 17, 1 << 30)] == [0, 0, 1, 1, 2, 1 << 26]


def test_step_refusals(ops):
    L, r, bad = ops.lib(), rows(ops), ops.VG_ERR_INVALID_ARG

    def step(n=4, c=64, dtype=1, flags=0, gate=r, x=r, state=4096, out=r):
        return L.vg_gated_scan_step(n, c, dtype, flags, gate, x, P(state), out, None)
    assert step(n=-1) == step(c=0) == step(dtype=5) == step(state=None) == step(state=4104) == bad
    assert step(gate=None) == step(x=rows(ops, 4104)) == step(out=rows(ops, stride=8)) == bad
    assert step(c=12) == step(flags=ops.VG_SCAN_REVERSE) == ops.VG_ERR_UNSUPPORTED
    assert step(n=0, gate=None, x=None, out=None, state=None) == ops.VG_OK


def test_dropout_refusals(ops):
    L, bad, nan = ops.lib(), ops.VG_ERR_INVALID_ARG, float("nan")

    def both(n=10, dtype=1, x=4096, p=0.5, rng=4096, out=4096):
        a = L.vg_dropout_add_fwd(n, dtype, P(x), None, p, P(rng), 0, P(out), None)
        assert a == L.vg_dropout_add_bwd(n, dtype, P(x), p, P(rng), 0, P(out), None)
        return a
    for kw in (dict(n=-1), dict(dtype=4), dict(x=None), dict(out=None), dict(rng=None), dict(p=-0.1), dict(p=1.0),
               dict(p=1 - 2.0 ** -33), dict(p=nan), dict(p=float("inf")), dict(x=4097), dict(out=4097),
               dict(rng=4100), dict(dtype=0, x=4098)):
        assert both(**kw) == bad, kw
    assert both(n=1 << 46) == ops.VG_ERR_UNSUPPORTED
    assert L.vg_dropout_add_fwd(10, 1, P(4096), P(4097), 0.5, P(4096), 0, P(4096), None) == bad
    assert both(n=0, x=None, out=None, rng=None) == ops.VG_OK


def test_binding_checks(ops):
    """Shapes and types that the binding turns down before it reaches the library; memory of another device."""
    x, w, st = torch.zeros(4, 64), torch.zeros(64), torch.zeros(4, 2)
    ws = torch.zeros(4096, dtype=torch.uint8)
    refused(lambda **t: ops.vg_layer_norm_fwd(**t), dict(x=x, weight=w, bias=w.clone(), y=x.clone(), stats=st))
    refused(lambda **t: ops.vg_layer_norm_bwd(**t), dict(
        x=x, weight=w, stats=st, grad_y=x.clone(), grad_skip=x.clone(), grad_x=x.clone(), grad_weight=w.clone(),
        grad_bias=w.clone(), ws=ws))
    off, order = torch.tensor([0, 4], dtype=torch.int32), torch.arange(4, dtype=torch.int32)
    h, kept = torch.zeros(1, 64), torch.zeros(1, 64)
    common = dict(gate=x, x=x.clone(), offsets=off, order=order, first=h, carries=kept, ws=ws)
    refused(lambda **t: ops.vg_gated_scan_fwd(**t), dict(common, out=x.clone(), last=h.clone()))
    refused(lambda **t: ops.vg_gated_scan_bwd(**t), dict(
        common, grad_out=x.clone(), grad_last=h.clone(), grad_gate=x.clone(), grad_x=x.clone(), grad_first=h.clone()))
    refused(lambda **t: ops.vg_gated_scan_step(**t), dict(gate=x, x=x.clone(), state=x.clone(), out=x.clone()))
    rng = torch.zeros(2, dtype=torch.int64)
    refused(lambda **t: ops.vg_dropout_add_fwd(p=0.5, call=0, **t),
            dict(x=x, residual=x.clone(), rng=rng, out=x.clone()))
    refused(lambda **t: ops.vg_dropout_add_bwd(p=0.5, call=0, **t), dict(grad_out=x, rng=rng, grad_x=x.clone()))

    g = {n: gpu(t) for n, t in dict(x=x, w=w, st=st, off=off, h=h, kept=kept, ws=ws, rng=rng, y=x.clone()).items()}
    for call in (
            lambda: ops.vg_layer_norm_fwd(g["w"], None, None, g["y"], None),
            lambda: ops.vg_layer_norm_fwd(g["x"], gpu(w[:8]), None, g["y"], None),
            lambda: ops.vg_layer_norm_fwd(g["x"], None, None, gpu(x.half()), None),
            lambda: ops.vg_layer_norm_fwd(g["x"], None, None, g["y"], gpu(st.double())),
            lambda: ops.vg_layer_norm_fwd(g["x"], None, None, gpu(torch.zeros(64, 4).t()), None),
            lambda: ops.vg_gated_scan_fwd(g["x"], g["y"], gpu(off.long()), None, None, g["y"], None, None, g["ws"]),
            lambda: ops.vg_gated_scan_fwd(g["x"], g["y"], g["off"], g["off"], None, g["y"], None, None, g["ws"]),
            lambda: ops.vg_gated_scan_fwd(g["x"], g["y"], g["off"], None, g["x"], g["y"], None, None, g["ws"]),
            lambda: ops.vg_gated_scan_fwd(g["x"], g["y"], g["off"], None, None, g["y"], None, g["x"], g["ws"]),
            lambda: ops.vg_gated_scan_step(g["x"], g["y"], g["h"], g["y"]),
            lambda: ops.vg_dropout_add_fwd(g["x"], gpu(w), 0.5, g["rng"], 0, g["y"]),
            lambda: ops.vg_dropout_add_fwd(g["x"], None, 0.5, gpu(rng.int()), 0, g["y"]),
            lambda: ops.vg_dropout_add_fwd(gpu(torch.zeros(64, 4).t()), None, 0.5, g["rng"], 0, g["y"])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ops.layer_norm_workspace(10, 12, device="cpu"),
                 lambda: ops.gated_scan_workspace(10, 64, 0, torch.float32, device="cpu")):
        with pytest.raises(ops.VGError):
            call()
