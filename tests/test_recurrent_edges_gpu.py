"""The recurrent-block operators at their edges: memory around the operands, exactly sized workspaces, captured training
passes, gates from one end of the sigmoid to the other, tensors of another GPU (GPU)."""
import pytest
import torch

from test_binding_devices import OnGpu1
from test_gated_scan_gpu import DT, F, R, U, call, compare, make, reference

from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


def fenced(shape, dtype, rows_before=3, rows_after=5):
    """A [rows, c] view inside of a buffer of sevens, and the check that nothing around it has changed."""
    n, c = shape
    buf = torch.full((n + rows_before + rows_after, c), 7.0, dtype=dtype, device="cuda")

    def check():
        assert (buf[:rows_before] == 7).all() and (buf[rows_before + n:] == 7).all()
    return buf[rows_before:rows_before + n], check


def exact_ws(nbytes):
    """A workspace of exactly so many bytes with a pattern behind it."""
    buf = torch.full((nbytes + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 256 == 0
    buf[:256] = 0

    def check():
        assert (buf[nbytes:] == 0x5A).all()
    return buf[:nbytes], check


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,c", [([1], 8), ([17], 72), ([127, 2, 500], 40), ([1025], 136), ([5000, 3], 64), ([40_001], 16),
                                       ([70_003], 520)])
def test_scan_stays_in_its_memory(dtype, lengths, c):
    x = make(lengths, c, dtype, order=True, state=True, seed=c)
    want = call(x)
    n, b, dt = sum(lengths), len(lengths), DT[dtype]
    ws, ws_ok = exact_ws(ops.gated_scan_workspace(n, c, b, dt).numel())
    kept, kept_ok = fenced(tuple(ops.gated_scan_carries(n, c).shape), torch.float32, rows_before=4)
    outs = {k: fenced((n, c), dt) for k in ("out", "grad_gate", "grad_x")}
    outs |= {k: fenced((b, c), torch.float32, rows_before=4) for k in ("last", "grad_first")}
    o = {k: v[0] for k, v in outs.items()}
    ops.vg_gated_scan_fwd(x["gate"], x["x"], x["offsets"], x["order"], x["first"], o["out"], o["last"], kept, ws)
    ops.vg_gated_scan_bwd(x["gate"], x["x"], x["offsets"], x["order"], x["first"], kept, x["grad_out"], x["grad_last"],
                          o["grad_gate"], o["grad_x"], o["grad_first"], ws)
    assert ops.vg_gated_scan_status(ws) == ops.VG_OK
    for k, v in outs.items():
        assert torch.equal(v[0], want[k]), k
        v[1]()
    ws_ok()
    kept_ok()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("n,c", [(1, 8), (257, 72), (1000, 1024), (33, 4096), (20_001, 64), (7, 8192)])
def test_norm_stays_in_its_memory(dtype, n, c):
    g = torch.Generator(device="cuda").manual_seed(n)
    dt = DT[dtype]
    x, gy = (torch.randn(n, c, generator=g, device="cuda").to(dt) for _ in range(2))
    w, b = (torch.randn(c, generator=g, device="cuda").to(dt) for _ in range(2))
    y, y_ok = fenced((n, c), dt)
    gx, gx_ok = fenced((n, c), dt)
    stats, stats_ok = fenced((n, 2), torch.float32, rows_before=4)
    gwb, gwb_ok = fenced((2, c), dt)
    ws, ws_ok = exact_ws(ops.layer_norm_workspace(n, c).numel())
    ops.vg_layer_norm_fwd(x, w, b, y, stats)
    ops.vg_layer_norm_bwd(x, w, stats, gy, None, gx, gwb[0], gwb[1], ws)
    torch.cuda.synchronize()
    for check in (y_ok, gx_ok, stats_ok, gwb_ok, ws_ok):
        check()
    assert y.isfinite().all() and gx.isfinite().all() and (gwb[1].double() - gy.double().sum(0)).norm() < 0.1 * (n * c) ** 0.5


@pytest.mark.parametrize("n", [1, 9, 4097, 300_001])
def test_dropout_stays_in_its_memory(n):
    rng = torch.tensor([5, 6], device="cuda")
    for shift in (0, 1):
        buf = torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[16 + shift:16 + shift + n]
        ops.vg_dropout_add_fwd(torch.randn(n, device="cuda").bfloat16(), None, 0.5, rng, 0, out)
        assert (buf[:16 + shift] == 7).all() and (buf[16 + shift + n:] == 7).all()


@pytest.mark.parametrize("lengths,c,flags", [([300], 64, 0), ([3000, 5, 0, 77], 72, R), ([50_000], 64, F)])
def test_a_captured_training_pass(lengths, c, flags):
    """Forward and backward in one graph, replayed over other inputs in the same memory."""
    xs = [make(lengths, c, "bf16", state=True, seed=s) for s in (1, 2, 3)]
    want = [call(x, flags) for x in xs]
    n, b = sum(lengths), len(lengths)
    mem = {k: torch.empty_like(xs[0][k]) for k in ("gate", "x", "first", "grad_out", "grad_last")}
    r = {k: torch.empty_like(v) for k, v in want[0].items()}
    ws, kept = ops.gated_scan_workspace(n, c, b, torch.bfloat16), ops.gated_scan_carries(n, c)
    off = xs[0]["offsets"]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.vg_gated_scan_fwd(mem["gate"], mem["x"], off, None, mem["first"], r["out"], r["last"], kept, ws, flags=flags)
        ops.vg_gated_scan_bwd(mem["gate"], mem["x"], off, None, mem["first"], kept, mem["grad_out"], mem["grad_last"],
                              r["grad_gate"], r["grad_x"], r["grad_first"], ws, flags=flags)
    for x, w in zip(xs, want):
        for k, t in mem.items():
            t.copy_(x[k])
        graph.replay()
        for k in r:
            assert torch.equal(r[k], w[k]), k


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_gates_from_end_to_end(dtype):
    """One token from a state of 1000, the input small beside it: out = a h + (1 - a) x element by element.  16-bit types
    find a h within 2^-23 of h (the rounding of 1 - a, and its reciprocal's), fp32 within its own size; the gate's
    exponential and reciprocal are good for 4e-6 at |g| < 40."""
    c, dt = 648, DT[dtype]
    gate = torch.linspace(-40, 40, c, device="cuda").to(dt)
    rows = torch.stack([gate, gate.flip(0)])
    x = make([1, 1], c, dtype, state=True, seed=3)
    x["gate"], x["x"] = rows.contiguous(), x["x"].contiguous()
    x["first"] = torch.full((2, c), 1000.0, device="cuda")
    r, ref = call(x), reference(x)
    a, s = torch.sigmoid(rows.double()), torch.sigmoid(-rows.double())
    parts = (a * 1000).abs() + (s * x["x"].double()).abs()
    left = 0 if dtype == "f32" else 2.0 ** -23 * 1000
    for name, u in (("out", U[dtype]), ("last", 0)):
        bound = u * ref[name].abs() + 4e-6 * parts + left + (2.0 ** -25 if dtype == "f16" else 0)
        assert ((r[name].double() - ref[name]).abs() <= bound).all(), name
    # the gradient of the gate keeps its size at both ends
    size = (a * s) * ((x["first"].double() - x["x"].double()) * (x["grad_out"].double() + x["grad_last"].double())).abs()
    tiny = 2.0 ** -25 if dtype == "f16" else 1e-30
    assert ((r["grad_gate"].double() - ref["grad_gate"]).abs() <= (U[dtype] + 1e-5) * size + tiny).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_gate_of_minus_infinity_lets_nothing_through(dtype):
    """What is far larger than the token's input leaves no trace: the state is the input, to the bit."""
    x = make([64], 32, dtype, state=True, seed=4)
    gate = x["gate"].contiguous()
    gate[20] = -float("inf")
    x["gate"], x["x"] = gate, x["x"].contiguous()
    x["x"][:20] = 30_000.0
    r = call(x)
    assert torch.equal(r["out"][20], x["x"][20])
    compare(r, reference(x), dtype)


def test_tensors_of_another_gpu_than_the_current_one():
    x = torch.zeros(4, 64, device="cuda").as_subclass(OnGpu1)
    w = torch.zeros(64, device="cuda").as_subclass(OnGpu1)
    rng = torch.zeros(2, dtype=torch.int64, device="cuda").as_subclass(OnGpu1)
    for f in (lambda: ops.vg_layer_norm_fwd(x, w, w, x, None), lambda: ops.vg_gated_scan_step(x, x, x, x),
              lambda: ops.vg_dropout_add_fwd(x, None, 0.5, rng, 0, x)):
        with pytest.raises(ValueError, match="current GPU"):
            f()
