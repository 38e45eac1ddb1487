"""vg_qk_norm_rope_fwd / _bwd against the formulas in 64 bits (GPU).

Angles are one fp32 product, (float)coord * freq; the reference takes that
product's fp32 value and goes on in 64 bits.  Bounds, as relative Frobenius
errors: fp32 sums of at most 256 squares, a square root and a handful of products
stay within 3e-6; a 16-bit result has one rounding more, at most u = half an ulp,
2^-8 (bf16) or 2^-11 (fp16).  A weight gradient is a sum over the rows: 3e-6 of the sum of its
terms' sizes, and its own rounding.
"""
import pytest
import torch

from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TOL = {"f32": 3e-6, "f16": 3e-6 + 2.0 ** -11, "bf16": 3e-6 + 2.0 ** -8}


def make(n, hq, hk, d, dtype, weights="heads", turn=True, pairs=None, seed=0, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    packed = (rnd(n, hq + hk + 1, d) * spread).to(dt)                 # strided views of a projection
    x = {"q": packed[:, :hq] if hq else None, "k": packed[:, hq:hq + hk] if hk else None}
    for name, h in (("q", hq), ("k", hk)):
        shape = (d,) if weights == "shared" else (h, d)
        x[name + "_weight"] = (1 + 0.3 * rnd(*shape)).to(dt) if h and weights else None
        x["g" + name] = rnd(n, h, d).to(dt) if h else None
    x["coords"] = x["freqs"] = x["pairs"] = None
    if turn:
        x["pairs"] = (d // 6, d // 6, d // 6) if pairs is None else pairs
        x["coords"] = torch.randint(-20, 1024, (n, 4), generator=g, device="cuda", dtype=torch.int32)
        x["freqs"] = torch.rand(sum(x["pairs"]), generator=g, device="cuda")
    return x


def call(x, flags=0, eps=1e-6, ws=None):
    pos = (x["q_weight"], x["k_weight"], x["coords"], x["freqs"], x["pairs"])

    def like(t):
        return None if t is None else torch.full(t.shape, float("nan"), dtype=t.dtype, device="cuda")
    r = {"q": like(x["q"]), "k": like(x["k"])}
    ops.vg_qk_norm_rope_fwd(x["q"], x["k"], *pos, r["q"], r["k"], eps=eps, flags=flags)
    r["grad_q"], r["grad_k"] = like(x["q"]), like(x["k"])
    r["grad_q_weight"], r["grad_k_weight"] = like(x["q_weight"]), like(x["k_weight"])
    some = x["q"] if x["q"] is not None else x["k"]
    hq, hk = (0 if x[n] is None else x[n].shape[1] for n in ("q", "k"))
    if ws is None:
        ws = ops.qk_norm_rope_workspace(some.shape[0], hq, hk, some.shape[2])
    ops.vg_qk_norm_rope_bwd(x["q"], x["k"], *pos, x["gq"], x["gk"], r["grad_q"], r["grad_k"], r["grad_q_weight"],
                            r["grad_k_weight"], ws, eps=eps, flags=flags)
    return r


def reference(x, flags=0, eps=1e-6):
    r = {}
    for name in ("q", "k"):
        if x[name] is None:
            continue
        v, d = x[name].double(), x[name].shape[2]
        w = torch.ones(d, dtype=torch.float64, device="cuda") if x[name + "_weight"] is None \
            else x[name + "_weight"].double()
        ang = torch.zeros(v.shape[0], d // 2, dtype=torch.float64, device="cuda")
        if x["coords"] is not None:
            axis = torch.repeat_interleave(torch.arange(3), torch.tensor(x["pairs"])).cuda()
            ang[:, :axis.numel()] = (x["coords"][:, 1 + axis].float() * x["freqs"]).double()
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        halves = flags & ops.VG_ROPE_HALVES
        i0 = torch.arange(d // 2, device="cuda") if halves else torch.arange(0, d, 2, device="cuda")
        i1 = i0 + d // 2 if halves else i0 + 1

        def turn(t, sign):
            y = torch.empty_like(t)
            y[..., i0] = t[..., i0] * c - sign * t[..., i1] * s
            y[..., i1] = sign * t[..., i0] * s + t[..., i1] * c
            return y
        g = turn(x["g" + name].double(), -1)
        if flags & ops.VG_QK_NO_NORM:
            r[name], r["grad_" + name] = turn(v, 1), g
            continue
        rms = (v.square().mean(2, keepdim=True) + eps).sqrt()
        r[name] = turn(v / rms * w, 1)
        r["grad_" + name] = g * w / rms - v * (g * w * v).mean(2, keepdim=True) / rms ** 3
        terms = g * v / rms
        over = (0, 1) if w.dim() == 1 else 0
        r[f"grad_{name}_weight"], r[f"size_{name}_weight"] = terms.sum(over), terms.abs().sum(over)
    return r


def compare(r, ref, dtype):
    for n, want in ref.items():
        if n.startswith("size") or r[n] is None:
            continue
        err = (r[n].double() - want).norm()
        if n.endswith("weight"):
            bound = 3e-6 * ref[n.replace("grad", "size")].norm() + (TOL[dtype] - 3e-6) * want.norm() + 1e-30
            if dtype == "f32":
                bound = bound + 1e-7 * want.norm()
        else:
            bound = TOL[dtype] * want.norm()
        assert err <= bound, (n, float(err), float(bound))


SHAPES = [
    (1, 16, 4, 128), (1, 1, 0, 8), (5, 0, 2, 24), (1000, 3, 1, 48), (37, 16, 4, 64), (700, 6, 2, 80), (513, 5, 5, 96),
    (129, 40, 8, 128), (33, 2, 1, 256), (300, 1, 1, 32), (9, 100, 30, 64),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("n,hq,hk,d", SHAPES)
def test_against_64_bits(dtype, halves, n, hq, hk, d):
    x = make(n, hq, hk, d, dtype, weights="shared" if n % 2 else "heads", seed=n + d)
    flags = ops.VG_ROPE_HALVES if halves else 0
    compare(call(x, flags), reference(x, flags), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(dtype):
    x = make(40_001, 4, 2, 64, dtype, seed=2)
    compare(call(x), reference(x), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("halves", [False, True])
def test_parts_alone(dtype, halves):
    """No weights; norm without rotation; rotation without norm; axes of unequal shares."""
    flags = ops.VG_ROPE_HALVES if halves else 0
    x = make(70, 4, 2, 64, dtype, weights=None)
    compare(call(x, flags), reference(x, flags), dtype)
    x = make(70, 4, 2, 64, dtype, turn=False)
    compare(call(x, flags), reference(x, flags), dtype)
    x = make(70, 4, 2, 64, dtype, weights=None)
    f = flags | ops.VG_QK_NO_NORM
    compare(call(x, f), reference(x, f), dtype)
    for pairs in ((0, 3, 1), (32, 0, 0), (0, 0, 32), (0, 0, 0)):
        x = make(70, 4, 2, 64, dtype, pairs=pairs)
        compare(call(x, flags), reference(x, flags), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_zero_rows_and_empty_calls(dtype):
    x = make(50, 2, 1, 64, dtype, seed=4)
    x["q"][7] = 0                                       # the row's norm is sqrt(eps) alone
    compare(call(x, eps=1e-3), reference(x, eps=1e-3), dtype)
    x = make(0, 2, 1, 64, dtype)
    r = call(x)
    assert not r["grad_q_weight"].any() and not r["grad_k_weight"].any()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_in_place_and_on_another_stream(dtype):
    x = make(333, 4, 2, 64, dtype, seed=6)
    want = call(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ops.vg_qk_norm_rope_fwd(x["q"], x["k"], x["q_weight"], x["k_weight"], x["coords"], x["freqs"], x["pairs"], x["q"],
                            x["k"], stream=s)
    s.synchronize()
    assert torch.equal(x["q"], want["q"]) and torch.equal(x["k"], want["k"])


def test_heads_first_layout():
    x = make(150, 4, 2, 64, "bf16", seed=8)
    want = call(x)
    for n in ("q", "k", "gq", "gk"):
        x[n] = x[n].transpose(0, 1).contiguous().transpose(0, 1)
    got = call(x)
    for n in ("q", "k", "grad_q", "grad_k", "grad_q_weight", "grad_k_weight"):
        assert torch.equal(got[n], want[n]), n


def test_the_same_from_run_to_run():
    x = make(20_000, 8, 4, 64, "bf16", weights="shared", seed=9)
    a, b = call(x), call(x)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_gradients_against_differences():
    """Central differences of sum(y * g) in fp32 at h = 1e-2: truncation h^2 of third derivatives of order 1, and
    rounding 1e-7 * sqrt(size) / h: 1e-3 of the gradient's norm."""
    x = make(60, 3, 1, 48, "f32", seed=10, spread=1.0)
    r = call(x)
    g = torch.Generator(device="cuda").manual_seed(3)
    for name in ("q", "k"):
        for what in (name, name + "_weight"):
            dirn = torch.randn(x[what].shape, generator=g, device="cuda")
            side = []
            for h in (1e-2, -1e-2):
                y = dict(x)
                y[what] = (x[what] + h * dirn).contiguous()
                side.append((call(y)[name].double() * x["g" + name].double()).sum())
            diff = float(side[0] - side[1]) / 2e-2
            grad = r["grad_" + what].double()
            assert abs(diff - float((grad * dirn.double()).sum())) <= 3e-3 * float(grad.norm()), what
