"""vg_gated_scan_fwd / _bwd / _step against the recurrence, token by token in 64 bits (GPU).

Bounds, as relative Frobenius errors.  fp32: a gate's sigmoid is off by an exponential of about 2 units (arguments up
to 10 add 10 * 2^-24), a sum and a quotient, 1.5e-6 in all, and moves a state by about twice that share; a
state passes the roundings of at most 8 tokens, 32 joined maps and 7 siblings a level, each 2^-24, that is under 4e-6: 1e-5
with those of its memory.  A gradient of the gate has both chains and two products: 2e-5.  A 16-bit result has one rounding
more, u = half a step, 2^-8 (bf16) or 2^-11 (fp16).
"""
import numpy as np
import pytest
import torch

from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
R, F = ops.VG_SCAN_REVERSE, ops.VG_SCAN_FREE_INPUT


def offsets(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def make(lengths, c, dtype, order=False, state=False, seed=0, memory=(0.0, 5.0)):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, n, b = DT[dtype], int(sum(lengths)), len(lengths)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")
    packed = torch.cat([rnd(n, c) + torch.linspace(*memory, c, device="cuda"), rnd(n, c)], 1).to(dt)
    x = {"gate": packed[:, :c], "x": packed[:, c:], "offsets": offsets(lengths), "lengths": lengths, "order": None,
         "first": rnd(b, c) if state else None, "grad_last": rnd(b, c) if state else None,
         "grad_out": rnd(n, c).to(dt)}
    if order:  # a permutation of all rows: sequences' tokens anywhere
        x["order"] = torch.randperm(n, generator=g, device="cuda").int()
    return x


def call(x, flags=0, ws=None, stream=None):
    n, c = x["x"].shape
    b = len(x["lengths"])
    nan = float("nan")
    r = {"out": torch.full_like(x["x"], nan), "last": torch.full((b, c), nan, device="cuda"),
         "grad_gate": torch.full_like(x["x"], nan), "grad_x": torch.full_like(x["x"], nan),
         "grad_first": torch.full((b, c), nan, device="cuda")}
    if ws is None:
        ws = ops.gated_scan_workspace(n, c, b, x["x"].dtype)
    kept = ops.gated_scan_carries(n, c).fill_(nan)
    ops.vg_gated_scan_fwd(x["gate"], x["x"], x["offsets"], x["order"], x["first"], r["out"], r["last"], kept, ws,
                          flags=flags, stream=stream)
    ops.vg_gated_scan_bwd(x["gate"], x["x"], x["offsets"], x["order"], x["first"], kept, x["grad_out"], x["grad_last"],
                          r["grad_gate"], r["grad_x"], r["grad_first"], ws, flags=flags, stream=stream)
    assert ops.vg_gated_scan_status(ws, stream) == ops.VG_OK
    return r


def reference(x, flags=0):
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    gate, v, gy = d(x["gate"]), d(x["x"]), d(x["grad_out"])
    n, c = v.shape
    b = len(x["lengths"])
    order = np.arange(n) if x["order"] is None else x["order"].cpu().numpy()
    h0 = np.zeros((b, c)) if x["first"] is None else d(x["first"])
    gl = np.zeros((b, c)) if x["grad_last"] is None else d(x["grad_last"])
    r = {k: np.zeros((n, c)) for k in ("out", "grad_gate", "grad_x")}
    r["last"], r["grad_first"] = h0.copy(), gl.copy()
    at = 0
    for i, t in enumerate(x["lengths"]):
        rows = order[at:at + t]
        at += t
        if flags & R:
            rows = rows[::-1]
        with np.errstate(over="ignore"):
            a, s = 1 / (1 + np.exp(-gate[rows])), 1 / (1 + np.exp(gate[rows]))
        xs = v[rows]
        h, before, after = h0[i], np.empty((t, c)), np.empty((t, c))
        for k in range(t):
            before[k] = h
            h = a[k] * h + (xs[k] if flags & F else s[k] * xs[k])
            after[k] = h
        mu = gl[i]
        lam = np.empty((t, c))
        for k in range(t - 1, -1, -1):
            lam[k] = gy[rows[k]] + mu
            mu = a[k] * lam[k]
        r["out"][rows], r["last"][i], r["grad_first"][i] = after, h, mu
        r["grad_x"][rows] = lam if flags & F else lam * s
        r["grad_gate"][rows] = lam * (before if flags & F else before - xs) * a * s
    return {k: torch.from_numpy(w).cuda() for k, w in r.items()}


def compare(r, ref, dtype):
    for n, want in ref.items():
        err, u = (r[n].double() - want).norm(), U["f32" if n in ("last", "grad_first") else dtype]
        bound = ((2e-5 if n == "grad_gate" else 1e-5) + u) * want.norm() + 1e-30
        assert err <= bound, (n, float(err), float(bound))


# one token to several tiles; beginnings and ends inside tiles, at their borders, at every token; empty sequences
CASES = [([1], 8), ([2], 40), ([7], 64), ([8, 8], 64), ([300], 24), ([256, 256], 64), ([255, 2, 255], 136),
         ([0, 5, 0, 0, 300, 1, 0], 72), ([1] * 300, 16), ([0, 0], 8), ([128, 128, 1, 127], 200), ([129, 511, 3], 128),
         ([3, 2500, 1000, 77], 80), ([700] * 5, 520)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("flags", [0, R, F, R | F])
@pytest.mark.parametrize("lengths,c", CASES)
def test_against_the_recurrence(dtype, flags, lengths, c):
    k = len(lengths) + c
    x = make(lengths, c, dtype, order=k % 2 == 0, state=k % 3 == 0, seed=k)
    compare(call(x, flags), reference(x, flags), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,flags", [([20_000], 0), ([9_000, 1, 11_000], R), ([70_001], 0), ([33_000, 0, 40_007], R)])
def test_long_sequences(dtype, lengths, flags):
    """Three and four levels of the tree of tiles, states that live through hundreds of tokens."""
    x = make(lengths, 16, dtype, order=True, state=True, seed=3, memory=(2.0, 6.0))
    compare(call(x, flags), reference(x, flags), dtype)


def test_many_sequences():
    lengths = np.random.default_rng(0).integers(0, 9, 5_000).tolist()
    x = make(lengths, 24, "f32", state=True, seed=4)
    for flags in (0, R):
        compare(call(x, flags), reference(x, flags), "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_that_are_shut_and_open(dtype):
    """Gates of plus and minus infinity, and so large that one side of the sigmoid rounds to 0 or 1."""
    x = make([600, 20], 64, dtype, state=True, seed=5)
    gate = x["gate"].contiguous()
    gate[::7], gate[3::11], gate[5::13], gate[2::17] = float("inf"), -float("inf"), 60.0, -60.0
    gate[:, 0], gate[:, 1], gate[:, 2] = float("inf"), -float("inf"), 17.0
    x["gate"] = gate
    compare(call(x), reference(x), dtype)


def test_what_is_not_finite_stays_in_its_channel_and_sequence():
    """The states after it are infinite or NaN up to the end of its sequence; all else keeps its bits."""
    x = make([40, 500, 60, 3000, 9], 32, "f32", state=True, seed=6)
    want = call(x)
    x["x"] = x["x"].contiguous()
    rows, cols = [45, 700, 1200], [3, 4, 5]
    for r, c, v in zip(rows, cols, (float("nan"), float("inf"), -float("inf"))):
        x["x"][r, c] = v
    got = call(x)
    ends = [540, 3600, 3600]
    hit = torch.zeros_like(got["out"], dtype=torch.bool)
    for r, c, e in zip(rows, cols, ends):
        hit[r:e, c] = True
    assert torch.equal(got["out"][~hit], want["out"][~hit])
    assert not got["out"][hit].isfinite().any()
    assert torch.equal(got["last"].isfinite(), torch.tensor(
        [[not (i, c) in {(1, 3), (3, 4), (3, 5)} for c in range(32)] for i in range(5)], device="cuda"))
    # gradients: x does not enter its own, and the gate's are of the same channel and sequence
    assert torch.equal(got["grad_x"], want["grad_x"])
    same = torch.ones(32, dtype=torch.bool, device="cuda")
    same[3:6] = False
    assert torch.equal(got["grad_gate"][:, same], want["grad_gate"][:, same])
    assert torch.equal(got["grad_gate"][:40], want["grad_gate"][:40])
    # a gradient that is not finite goes the other way, up to the sequence's beginning
    x = make([40, 500, 60], 32, "f32", seed=7)
    want = call(x)
    x["grad_out"][300, 9] = float("nan")
    got = call(x)
    hit = torch.zeros_like(got["out"], dtype=torch.bool)
    hit[40:301, 9] = True
    for n in ("grad_x", "grad_gate"):
        assert torch.equal(got[n][~hit], want[n][~hit]) and not got[n][hit].isfinite().any(), n


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("free", [False, True])
def test_token_by_token(dtype, free):
    """Single-token steps against one scan: the states agree, so decoding can go on from a scan's last state."""
    steps, b, c = 40, 5, 72
    flags = F if free else 0
    x = make([steps] * b, c, dtype, state=True, seed=8)
    want = reference(x, flags)
    st = x["first"].clone()
    for t in range(steps):
        out = torch.empty(b, c, dtype=DT[dtype], device="cuda")
        ops.vg_gated_scan_step(x["gate"][t::steps], x["x"][t::steps], st, out, flags=flags)
        compare({"out": out}, {"out": want["out"][t::steps]}, dtype)
    compare({"last": st}, {"last": want["last"]}, dtype)


def test_steps_of_odd_batches():
    for n, c in ((1, 8), (3, 520), (1001, 1024), (0, 16)):
        x = make([1] * n, c, "bf16", state=True, seed=n)
        st, out = x["first"].clone(), torch.empty(n, c, dtype=torch.bfloat16, device="cuda")
        ops.vg_gated_scan_step(x["gate"], x["x"], st, out)
        ref = reference(x)
        compare({"out": out, "last": st}, {"out": ref["out"], "last": ref["last"]}, "bf16")


def test_outputs_that_are_not_wanted():
    x = make([300, 200], 64, "f16", seed=9)
    want = call(x)
    ws = ops.gated_scan_workspace(500, 64, 2, torch.float16)
    out, gg, gx = (torch.empty_like(want["out"]) for _ in range(3))
    ops.vg_gated_scan_fwd(x["gate"], x["x"], x["offsets"], None, None, out, None, None, ws)
    assert torch.equal(out, want["out"])
    kept = ops.gated_scan_carries(500, 64)
    ops.vg_gated_scan_fwd(x["gate"], x["x"], x["offsets"], None, None, out, None, kept, ws)
    ops.vg_gated_scan_bwd(x["gate"], x["x"], x["offsets"], None, None, kept, x["grad_out"], None, gg, gx, None, ws)
    assert torch.equal(gg, want["grad_gate"]) and torch.equal(gx, want["grad_x"])


def test_in_place_strided_and_neighbours():
    """The output over the input, gradients over the packed projection's halves, columns beside them untouched."""
    x = make([500, 0, 77], 40, "bf16", order=True, state=True, seed=10)
    want = call(x)
    ws = ops.gated_scan_workspace(577, 40, 3, torch.bfloat16)
    packed = torch.full((577, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    gg, gx = packed[:, :40], packed[:, 48:88]
    kept, last = ops.gated_scan_carries(577, 40), torch.empty(3, 40, device="cuda")
    y = x["x"].contiguous()
    ops.vg_gated_scan_fwd(x["gate"], y, x["offsets"], x["order"], x["first"], y, last, kept, ws)
    assert torch.equal(y, want["out"]) and torch.equal(last, want["last"])
    ops.vg_gated_scan_bwd(x["gate"], x["x"], x["offsets"], x["order"], x["first"], kept, x["grad_out"], x["grad_last"],
                          gg, gx, None, ws)
    assert torch.equal(gg, want["grad_gate"]) and torch.equal(gx, want["grad_x"])
    assert (packed[:, 40:48] == 7).all() and (packed[:, 88:] == 7).all()


def test_the_same_from_run_to_run():
    x = make([60_000, 50_000], 128, "bf16", seed=11)
    a = call(x)
    for _ in range(3):
        b = call(x)
        for n in a:
            assert torch.equal(a[n], b[n]), n


def test_two_calls_at_once_and_graphs_that_share_a_workspace():
    xs = [make([40_000], 64, "f32", seed=s) for s in (1, 2)]
    want = [call(x) for x in xs]
    wss = [ops.gated_scan_workspace(40_000, 64, 1, torch.float32) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    kept = [ops.gated_scan_carries(40_000, 64) for _ in range(2)]
    out = [torch.empty_like(w["out"]) for w in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, ws, s, k, o in zip(xs, wss, streams, kept, out):
            ops.vg_gated_scan_fwd(x["gate"], x["x"], x["offsets"], None, None, o, None, k, ws, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(out, want):
        assert torch.equal(o, w["out"])
    graphs = []
    for x, o in zip(xs, out):                      # both on the first workspace, one after the other
        o.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.vg_gated_scan_fwd(x["gate"], x["x"], x["offsets"], None, None, o, None, None, wss[0])
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(out, want):
        assert torch.equal(o, w["out"])
    assert ops.vg_gated_scan_status(wss[0]) == ops.VG_OK


def test_a_workspace_full_of_anything():
    """What a workspace held before does not matter, past its error record."""
    x = make([5_000], 64, "bf16", seed=12)
    want = call(x)
    for fill in (0, 0xFF, 0x5A):
        ws = ops.gated_scan_workspace(5_000, 64, 1, torch.bfloat16)
        ws[4:] = fill
        got = call(x, ws=ws)
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["grad_gate"], want["grad_gate"])


def test_bad_offsets_write_nothing():
    for bad in ([0, 30, 20, 50], [1, 10, 20, 50], [0, 10, 20, 49], [0, 10, 60, 50], [0, -5, 20, 50]):
        x = make([10, 10, 30], 16, "f32", seed=13)
        ws = ops.gated_scan_workspace(50, 16, 3, torch.float32)
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        out, last = torch.full((50, 16), 7.0, device="cuda"), torch.full((3, 16), 7.0, device="cuda")
        kept = ops.gated_scan_carries(50, 16)
        ops.vg_gated_scan_fwd(x["gate"], x["x"], off, None, None, out, last, kept, ws)
        assert ops.vg_gated_scan_status(ws) == ops.VG_ERR_INVALID_ARG
        ops.vg_gated_scan_bwd(x["gate"], x["x"], off, None, None, kept, x["grad_out"], None, out, out.clone(), last, ws)
        assert ops.vg_gated_scan_status(ws) == ops.VG_ERR_INVALID_ARG
        assert (out == 7).all() and (last == 7).all()
        # the workspace serves again
        ops.vg_gated_scan_fwd(x["gate"], x["x"], x["offsets"], None, None, out, last, kept, ws)
        assert ops.vg_gated_scan_status(ws) == ops.VG_OK
        compare({"out": out}, {"out": reference(x)["out"]}, "f32")


def test_an_order_that_leaves_the_rows_is_reported():
    """The token's row is left out; sequences without such tokens keep their results."""
    x = make([300, 400], 16, "f32", seed=14)
    want = call(x)
    order = torch.arange(700, dtype=torch.int32, device="cuda")
    order[10], order[20], order[30] = -1, 700, 2 ** 31 - 1
    out = torch.full((700, 16), 7.0, device="cuda")
    ws = ops.gated_scan_workspace(700, 16, 2, torch.float32)
    kept = ops.gated_scan_carries(700, 16)
    ops.vg_gated_scan_fwd(x["gate"], x["x"], x["offsets"], order, None, out, None, kept, ws)
    assert ops.vg_gated_scan_status(ws) == ops.VG_ERR_INVALID_ARG
    assert torch.equal(out[300:], want["out"][300:]) and (out[[10, 20, 30]] == 7).all()
    gg, gx = torch.full_like(out, 7.0), torch.full_like(out, 7.0)
    ops.vg_gated_scan_bwd(x["gate"], x["x"], x["offsets"], order, None, kept, x["grad_out"], None, gg, gx, None, ws)
    assert ops.vg_gated_scan_status(ws) == ops.VG_ERR_INVALID_ARG
    assert (gg[[10, 20, 30]] == 7).all() and torch.equal(gx[300:], want["grad_x"][300:])


def test_gradients_against_differences():
    """Central differences of sum(out g) + sum(last gl) in fp32 at h = 1e-2: truncation h^2 of third derivatives of
    order 1 and rounding 1e-7 sqrt(size) / h: 1e-3 of the gradient's norm."""
    x = make([90, 300, 7], 24, "f32", order=True, state=True, seed=15, memory=(-1.0, 2.0))
    g = torch.Generator(device="cuda").manual_seed(3)
    for flags in (0, R, F):
        r = call(x, flags)
        for what, grad in (("gate", "grad_gate"), ("x", "grad_x"), ("first", "grad_first")):
            dirn = torch.randn(x[what].shape, generator=g, device="cuda")
            side = []
            for h in (1e-2, -1e-2):
                y = dict(x)
                y[what] = (x[what] + h * dirn).contiguous()
                z = call(y, flags)
                side.append((z["out"].double() * x["grad_out"].double()).sum() +
                            (z["last"].double() * x["grad_last"].double()).sum())
            diff = float(side[0] - side[1]) / 2e-2
            have = float((r[grad].double() * dirn.double()).sum())
            assert abs(diff - have) <= 3e-3 * float(r[grad].double().norm()), (flags, what)
