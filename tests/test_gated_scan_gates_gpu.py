"""What a gate keeps of a state, element by element, from one end of the sigmoid to the other (GPU).

Inputs are zero and free, or a sequence is one token, so that results are products of a = sigmoid(gate) alone:
nothing hides what a nearly closed gate lets through.

Bounds.  exp(gate) is exp2 of the rounded product with log2(e): |gate| (2^-24 + 1.3e-8) and the instruction's 2^-22, at |gate| <= 40
together 3.2e-6; sum, reciprocal and the products that make a of them are within 7 units of 2^-24 more: 3.6e-6 of a for every
16-bit gate, and of 1 - a.  fp32 gates: exp of 2 units, a sum, a quotient: 2^-21.  A state then passes two roundings a token.
"""
import pytest
import torch

from test_gated_scan_gpu import DT, F, R, U, call, make, reference

from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

A_ERR = {"f32": 2.0 ** -21, "f16": 3.6e-6, "bf16": 3.6e-6}


def closed_gates(dtype, rows, c, lo=-40.0, hi=40.0):
    g = torch.linspace(lo, hi, rows * c, device="cuda").view(rows, c)
    return g[torch.arange(rows, device="cuda") * 7 % rows].to(DT[dtype]).contiguous()


def near(got, want, rel, what):
    err = (got.double() - want).abs() / want.abs()
    assert err.max() <= rel, (what, float(err.max()), rel)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("b,flags", [(2, 0), (300, F), (300, R)])
def test_one_token_keeps_its_share(dtype, b, flags):
    """grad_first = a lam, and with no input last = a first; from one tile and from many."""
    c = 136
    x = make([1] * b, c, dtype, state=True, seed=b)
    x["gate"] = closed_gates(dtype, b, c)
    x["x"] = torch.zeros_like(x["gate"])
    r, ref = call(x, flags), reference(x, flags)
    a = torch.sigmoid(x["gate"].double())
    near(r["last"], a * x["first"].double(), A_ERR[dtype] + 2 * 2.0 ** -24, "last")
    lam = x["grad_out"].double() + x["grad_last"].double()   # its sum may cancel: one rounding of 2^-24 of it
    near(r["grad_first"], a * lam, A_ERR[dtype] + 3 * 2.0 ** -24, "grad_first")
    tiny = {"f32": 1e-30, "bf16": 1e-30, "f16": 2.0 ** -25}[dtype]
    assert ((r["out"].double() - ref["out"]).abs() <= (U[dtype] + 4e-6) * ref["out"].abs() + tiny).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lengths,c,lo,hi", [([9] * 40, 64, -8.0, 0.0), ([600, 3, 700], 24, 0.5, 6.0), ([5000], 16, 4.0, 9.0),
                                             ([2, 3] * 60, 136, -20.0, -9.0)])
@pytest.mark.parametrize("flags", [F, F | R])
def test_what_is_left_after_many_tokens(dtype, lengths, c, lo, hi, flags):
    """first times all of a sequence's gates, and grad_last's way back; the tokens' own inputs and gradients are zero."""
    n = sum(lengths)
    x = make(lengths, c, dtype, state=True, seed=n)
    x["gate"] = closed_gates(dtype, n, c, lo, hi)
    x["x"], x["grad_out"] = torch.zeros_like(x["gate"]), torch.zeros_like(x["gate"])
    r = call(x, flags)
    a, at = torch.sigmoid(x["gate"].double()), 0
    s = torch.sigmoid(-x["gate"].double())
    for i, t in enumerate(lengths):
        left = a[at:at + t].log().sum(0)
        # each gate's error moves a state by that share of a, or (open gates) that share of 1 - a and a rounding
        share = torch.minimum(s[at:at + t] * A_ERR[dtype] + 2.0 ** -24, torch.tensor(A_ERR[dtype], device="cuda").double())
        rel = float((share + 2 * 2.0 ** -24).sum(0).max()) * 1.01
        at += t
        want = left.exp()
        assert float(left.min()) > -80
        near(r["last"][i], want * x["first"][i].double(), rel, ("last", i))
        near(r["grad_first"][i], want * x["grad_last"][i].double(), rel, ("grad_first", i))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,c,flags,lo,hi", [(2_900, 72, F, -11.0, -3.0), (2_900, 72, F | R, -11.0, -3.0),
                                             (2_900, 72, F, -3.0, -0.5), (40_000, 8, F, -11.0, 0.0), (40_000, 8, F | R, -3.0, 0.0)])
def test_a_nearly_closed_gate_here_and_there(dtype, n, c, flags, lo, hi):
    """Whole runs of tokens in which a few gates, or none, are nearly closed, within one long sequence."""
    x = make([n], c, dtype, order=True, state=True, seed=n)
    gate = torch.full((n, c), 80.0, device="cuda")           # keeps a state as it is
    gate[::16] = torch.linspace(11.0, 12.0, c, device="cuda")
    gate[5::n // 7] = torch.linspace(lo, hi, c, device="cuda")
    x["gate"] = gate.to(DT[dtype])
    x["x"], x["grad_out"] = torch.zeros_like(x["gate"]), torch.zeros_like(x["gate"])
    r = call(x, flags)
    d = x["gate"].double()
    left = torch.nn.functional.logsigmoid(d).sum(0)
    share = torch.where(d > 0, torch.sigmoid(-d) * A_ERR[dtype] + 2.0 ** -24 * (d < 80), torch.tensor(A_ERR[dtype], device="cuda").double())
    rel = float(share.sum(0).max()) + 2 * 2.0 ** -24 * n
    for name, of in (("last", "first"), ("grad_first", "grad_last")):
        near(r[name][0], left.exp() * x[of][0].double(), rel, name)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_steps_keep_their_share(dtype):
    n, c = 33, 136
    gate = closed_gates(dtype, n, c)
    first = torch.randn(n, c, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    st, out = first.clone(), torch.empty_like(gate)
    ops.vg_gated_scan_step(gate, torch.zeros_like(gate), st, out, flags=F)
    near(st, torch.sigmoid(gate.double()) * first.double(), A_ERR[dtype] + 2 * 2.0 ** -24, "state")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gates_beyond_the_exponentials_range(dtype):
    """Gates of 80 and more in size: nothing turns into NaN, open gates keep a state to the bit, shut ones leave the input."""
    ends = torch.tensor([-float("inf"), -1000.0, -200.0, -100.0, 87.0, 88.0, 89.0, 90.0, 127.0, 128.0, 1000.0, float("inf")],
                        device="cuda").to(DT[dtype])
    c = 96
    x = make([1, 40, 3000], c, dtype, state=True, seed=7)
    x["gate"] = ends[torch.arange(x["x"].numel(), device="cuda") * 5 % 12].view(-1, c).contiguous()
    x["x"] = x["x"].contiguous()
    for flags in (0, R):
        r, at = call(x, flags), 0
        for i, t in enumerate(x["lengths"]):
            rows = range(at + t - 1, at - 1, -1) if flags else range(at, at + t)
            at += t
            h = x["first"][i].clone()
            for k in rows:
                h = torch.where(x["gate"][k] > 0, h, x["x"][k].float())
                assert torch.equal(r["out"][k], h.to(DT[dtype])), (i, k)
            assert torch.equal(r["last"][i], h)
        for name in ("grad_gate", "grad_x", "grad_first"):
            assert r[name].isfinite().all(), name
        shut = x["gate"] < 0
        assert (r["grad_gate"].float().abs() <= 1e-30).all() and (r["grad_x"][~shut].float().abs() <= 1e-30).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lengths,shift", [([40, 500, 60, 3000, 9], 0.0), ([40, 500, 60, 3000, 9], -4.0), ([900, 70_000], 2.0)])
def test_16_bit_tokens_that_are_not_finite(dtype, lengths, shift):
    """They reach their channel's later states of their sequence and the gradients of its gates, and nothing else."""
    c, ends = 72, torch.tensor(lengths).cumsum(0).tolist()
    x = make(lengths, c, dtype, state=True, seed=6, memory=(shift, shift + 4.0))
    want = call(x)
    x["x"] = x["x"].contiguous()
    hit = torch.zeros_like(want["out"], dtype=torch.bool)
    for row, col, v in ((45, 3, float("nan")), (ends[0] + 100, 4, float("inf")), (ends[-1] - 5, 71, -float("inf"))):
        x["x"][row, col] = v
        hit[row:next(e for e in ends if e > row), col] = True
    got = call(x)
    assert torch.equal(got["out"][~hit], want["out"][~hit]) and not got["out"][hit].isfinite().any()
    assert torch.equal(got["grad_x"], want["grad_x"]) and torch.equal(got["grad_first"], want["grad_first"])
    assert torch.equal(got["grad_gate"][~hit], want["grad_gate"][~hit])
    y = make(lengths, c, dtype, state=True, seed=6, memory=(shift, shift + 4.0))
    row, start = ends[0] + 300, ends[0]
    y["grad_out"][row, 9] = float("nan")
    got, hit = call(y), torch.zeros_like(hit)
    hit[start:row + 1, 9] = True
    assert torch.equal(got["out"], want["out"])
    for name in ("grad_x", "grad_gate"):
        assert torch.equal(got[name][~hit], want[name][~hit]) and not got[name][hit].isfinite().any(), name
