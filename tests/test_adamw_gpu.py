"""vg_adamw_step and vg_adamw_decode against the step in 64 bits (GPU).

Bounds come from counting fp32 roundings (e = 2^-24 each, half an ulp): m is three
of them on its terms' sizes, v four, the parameter three on its own size and about
twelve on the step's.  8-bit moments are held to half a step of their format around
the 64-bit value (plus those roundings), and to the nearest code where it is clear.
"""
import math

import pytest
import torch

from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
H = dict(lr=1e-2, beta1=0.9, beta2=0.98, eps=1e-8)


def make(sizes, dtype, bits, master, seed=0, shift=0, wd=0.1):
    """Tensors of the given sizes; with `shift`, views that start `shift` elements into their storage."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda n: torch.randn(n, generator=g, device="cuda")  # noqa: E731

    def put(x, dt):
        s = torch.empty(x.numel() + shift, dtype=dt, device="cuda")[shift:]
        s.copy_(x)
        return s
    dts = [DT[d] for d in (dtype if isinstance(dtype, list) else [dtype] * len(sizes))]
    masters = [put(rnd(n), torch.float32) for n in sizes]
    params = [put(m, dt) for m, dt in zip(masters, dts)]
    grads = [put(rnd(n) * 0.01, dt) for n, dt in zip(sizes, dts)]
    decay = [wd if i % 2 == 0 else 0.0 for i in range(len(sizes))]
    st = ops.AdamWState(params, grads, masters if master else None, bits=bits, weight_decay=decay)
    return dict(params=params, grads=grads, masters=masters if master else None, decay=decay, st=st, bits=bits)


def moments(t):
    """The moments of each tensor as fp32."""
    st = t["st"]
    if t["bits"] == 32:
        flat = (st.m, st.v)
    else:
        flat = (torch.empty(st.m.numel(), device="cuda"), torch.empty(st.m.numel(), device="cuda"))
        ops.vg_adamw_decode(st.m, st.m_scale, flat[0], second=False)
        ops.vg_adamw_decode(st.v, st.v_scale, flat[1], second=True)
    return [[f[o:o + p.numel()].double() for p, o in zip(t["params"], st.offsets)] for f in flat]


def check_step(t, step, gs=1.0, h=H):
    m0, v0 = moments(t)
    p0 = [(x if t["masters"] is None else y).double().clone()
          for x, y in zip(t["params"], t["masters"] or t["params"])]
    ops.vg_adamw_step(t["st"], step, h["lr"], h["beta1"], h["beta2"], h["eps"], grad_scale=gs)
    m1, v1 = moments(t)
    for i, grad in enumerate(t["grads"]):
        g = grad.double() * gs
        m = h["beta1"] * m0[i] + (1 - h["beta1"]) * g
        v = h["beta2"] * v0[i] + (1 - h["beta2"]) * g * g
        em = 4 * E * (h["beta1"] * m0[i].abs() + (1 - h["beta1"]) * g.abs()) + 1e-44
        ev = 6 * E * v + 1e-44
        upd = h["lr"] / (1 - h["beta1"] ** step) / ((v / (1 - h["beta2"] ** step)).sqrt() + h["eps"])
        p = p0[i] * (1 - h["lr"] * t["decay"][i]) - upd * m
        ep = 4 * E * p0[i].abs() + upd * (em + 12 * E * m.abs())
        new = (t["params"] if t["masters"] is None else t["masters"])[i]
        dt = t["params"][i].dtype
        u = {torch.float32: 0.0, torch.float16: 2.0 ** -12 * 2, torch.bfloat16: 2.0 ** -9 * 2}[dt]
        tiny = 0.0 if dt != torch.float16 else 2.0 ** -25
        if t["masters"] is not None:
            assert ((new.double() - p).abs() <= ep + 1e-44).all()
            assert torch.equal(t["params"][i], new.to(dt))
        else:
            assert ((new.double() - p).abs() <= ep + u * p.abs() + tiny + 1e-44).all()
        if t["bits"] == 32:
            assert ((m1[i] - m).abs() <= em).all() and ((v1[i] - v).abs() <= ev).all()
            continue
        n, st, o = m.numel(), t["st"], t["st"].offsets[i]
        nb = -(-n // 256)
        ms = st.m_scale[o // 256:o // 256 + nb].double().repeat_interleave(256)[:n]
        vs = st.v_scale[o // 256:o // 256 + nb].double().repeat_interleave(256)[:n]
        # half a step: 2^-4 of a value's power of two (2^-5 for the root), or half of 2^-9 below 2^-6
        assert ((m1[i] - m).abs() <= em + torch.maximum(m.abs() / 16, ms * 2.0 ** -10)).all()
        root = v.sqrt()
        small = root < vs
        err = (v1[i].sqrt() - root).abs()
        assert (err[~small] <= root[~small] / 32 * (1 + 1e-5)).all()
        assert (v1[i].sqrt()[small & (v > 1e-40)] == vs[small & (v > 1e-40)]).all()
        assert (v1[i][v == 0] == 0).all()
        for s, top, x in ((ms, 7, m), (vs, 14, root)):
            lead = torch.zeros(nb * 256, dtype=torch.float64, device="cuda")
            lead[:n] = x.abs()
            big = lead.view(nb, 256).amax(1)
            sc = s[::256]
            fine = big > 1e-30
            ratio = (big / sc)[fine]
            assert ((ratio >= 2.0 ** top * (1 - 1e-5)) & (ratio <= 2.0 ** (top + 1) * (1 + 1e-5))).all()
            assert (torch.frexp(sc)[0] == 0.5).all()          # powers of two


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype,master", [("f32", False), ("f16", True), ("bf16", True), ("bf16", False),
                                          ("f16", False), ("f32", True)])
def test_steps(bits, dtype, master):
    t = make([1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 5000, 0, 30_001], dtype, bits, master, seed=bits)
    for step in (1, 2, 3, 1000):
        check_step(t, step, gs=0.5 if step == 2 else 1.0)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("shift", [1, 3])
def test_unaligned_tensors(bits, shift):
    t = make([1000, 13, 4096], "bf16", bits, True, seed=1, shift=shift)
    u = make([1000, 13, 4096], "bf16", bits, True, seed=1)
    for step in (1, 2):
        check_step(t, step)
        check_step(u, step)
    for a, b in zip(t["params"] + t["masters"], u["params"] + u["masters"]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("count", [33, 384, 385, 900])
def test_many_tensors(count):
    sizes = [1 + (i * 37) % 600 for i in range(count)]
    t = make(sizes, [["f32", "f16", "bf16"][i % 3] for i in range(count)], 8 if count % 2 else 32, True, seed=count)
    check_step(t, 1)


@pytest.mark.parametrize("bits", [8, 32])
def test_zero_gradients(bits):
    t = make([600], "f32", bits, False)
    t["grads"][0].zero_()
    before = t["params"][0].clone()
    ops.vg_adamw_step(t["st"], 1, 0.1)
    assert torch.equal(t["params"][0], before * torch.tensor(1 - 0.1 * 0.1, dtype=torch.float64).float())
    m, v = moments(t)
    assert not m[0].any() and not v[0].any()


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_values_that_are_not_finite(value):
    """They stay where they are: in 8 bits a block's other states keep their scale, and the bad one is NaN."""
    for bits in (8, 32):
        t, u = make([700], "f32", bits, False, seed=5), make([700], "f32", bits, False, seed=5)
        t["grads"][0][300] = value
        u["grads"][0][300] = 0
        ops.vg_adamw_step(t["st"], 1, 1e-2)
        ops.vg_adamw_step(u["st"], 1, 1e-2)
        keep = torch.arange(700, device="cuda") != 300
        (mt, vt), (mu, vu) = moments(t), moments(u)
        assert torch.equal(mt[0][keep], mu[0][keep]) and torch.equal(vt[0][keep], vu[0][keep])
        assert torch.equal(t["params"][0][keep], u["params"][0][keep])
        assert t["params"][0][300].isnan()
        if bits == 8:
            assert mt[0][300].isnan() and vt[0][300].isnan()


def test_every_code():
    """The 256 codes of both formats, as the header defines them."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    scale = torch.tensor([2.0 ** -5], device="cuda")
    m, v = torch.empty(256, device="cuda"), torch.empty(256, device="cuda")
    ops.vg_adamw_decode(codes, scale, m, second=False)
    ops.vg_adamw_decode(codes, scale, v, second=True)
    for c in range(256):
        a = c & 127
        x = a / 512 if a < 8 else (1 + (a & 7) / 8) * 2.0 ** ((a >> 3) - 7)
        want = math.nan if a == 127 else math.copysign(x, -1 if c & 128 else 1) / 32
        assert m[c].item() == want or (math.isnan(want) and m[c].isnan()), c
        y = 0.0 if c == 0 else (1 + ((c - 1) & 15) / 16) * 2.0 ** ((c - 1) >> 4)
        want = math.nan if c == 255 else (y / 32) ** 2
        assert v[c].item() == want or (math.isnan(want) and v[c].isnan()), c


def test_scale_range():
    """Gradients from 1e-30 to 1e15: the scale exponent is held to what fp32 can invert."""
    for s in (1e-30, 1e-12, 1.0, 1e15):
        t = make([512], "f32", 8, False, seed=6)
        t["grads"][0].mul_(s)
        ops.vg_adamw_step(t["st"], 1, 1e-3)
        m, v = moments(t)
        assert m[0].isfinite().all() and v[0].isfinite().all()
        if s >= 1e-12:
            want = 0.1 * t["grads"][0].double()
            assert float((m[0] - want).norm() / want.norm()) < 1 / 16


def test_on_another_stream():
    t, u = make([3000], "bf16", 8, True, seed=7), make([3000], "bf16", 8, True, seed=7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ops.vg_adamw_step(t["st"], 1, 1e-2, stream=s)
    s.synchronize()
    ops.vg_adamw_step(u["st"], 1, 1e-2)
    assert torch.equal(t["masters"][0], u["masters"][0]) and torch.equal(t["st"].m, u["st"].m)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_each_operation_is_rounded_by_itself(dtype, bits):
    """A step from zero moments, then another one, bit for bit as single fp32 operations (each a pass of its own here)
    give it; with bits = 8 the second step starts from the decoded codes."""
    t = make([70001], dtype, bits, master=True, seed=3)
    p, grad = t["masters"][0].clone(), t["grads"][0].float()
    f32 = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    b1, omb1, b2, omb2 = (f32(x) for x in (H["beta1"], 1 - H["beta1"], H["beta2"], 1 - H["beta2"]))
    for step in (1, 2):
        m, v = (x[0].float() for x in moments(t))
        ops.vg_adamw_step(t["st"], step, H["lr"], H["beta1"], H["beta2"], H["eps"])
        m = m * b1 + grad * omb1
        v = v * b2 + (grad * grad) * omb2
        den = v.sqrt() * f32((1 - H["beta2"] ** step) ** -0.5) + f32(H["eps"])
        p = p * f32(1 - H["lr"] * t["decay"][0]) - (m / den) * f32(H["lr"] / (1 - H["beta1"] ** step))
        assert torch.equal(t["masters"][0], p) and torch.equal(t["params"][0], p.to(DT[dtype]))
