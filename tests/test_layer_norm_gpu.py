"""vg_layer_norm_fwd / _bwd against the formulas in 64 bits (GPU).

Bounds, as relative Frobenius errors: an fp32 sum of C <= 8192 terms is taken as at most 32 in a lane, then pairs:
some 45 roundings of 2^-24 each, and a square root and a handful of products stay within 3e-6; a 16-bit result has
one rounding more, at most u = half a step, 2^-8 (bf16) or 2^-11 (fp16).  A weight gradient is a sum over the rows: 3e-6 of
the sum of its terms' sizes, and its own rounding.
"""
import pytest
import torch

from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
EPS = 1e-5


def make(n, c, dtype, affine=True, skip=False, seed=0, wide=False, offset=0.0):
    """wide: rows of a packed tensor, strides beyond the channel count."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")

    def rows():
        t = rnd(n, 2 * c + 8 if wide else c).to(dt)
        return t[:, 8:8 + c] if wide else t
    x = {"x": rows(), "grad_y": rows(), "grad_skip": rows() if skip else None}
    if offset:
        x["x"] = x["x"] + offset
    x["weight"] = (1 + 0.3 * rnd(c)).to(dt) if affine else None
    x["bias"] = (0.5 * rnd(c)).to(dt) if affine else None
    return x


def call(x, eps=EPS, ws=None):
    n, c = x["x"].shape

    def like(t):
        return None if t is None else torch.full(t.shape, float("nan"), dtype=t.dtype, device="cuda")
    r = {"y": like(x["x"]), "stats": torch.full((n, 2), float("nan"), device="cuda"), "grad_x": like(x["x"]),
         "grad_weight": like(x["weight"]), "grad_bias": like(x["bias"])}
    ops.vg_layer_norm_fwd(x["x"], x["weight"], x["bias"], r["y"], r["stats"], eps=eps)
    if ws is None and x["weight"] is not None:
        ws = ops.layer_norm_workspace(n, c)
    ops.vg_layer_norm_bwd(x["x"], x["weight"], r["stats"], x["grad_y"], x["grad_skip"], r["grad_x"], r["grad_weight"],
                          r["grad_bias"], ws)
    return r


def reference(x, eps=EPS):
    v, g = x["x"].double(), x["grad_y"].double()
    mean = v.mean(1, keepdim=True)
    rstd = 1 / ((v - mean).square().mean(1, keepdim=True) + eps).sqrt()
    z = (v - mean) * rstd
    r = {"stats": torch.cat([mean, rstd], 1), "y": z}
    if x["weight"] is not None:
        r["y"] = z * x["weight"].double() + x["bias"].double()
        r["grad_weight"], r["size_weight"] = (g * z).sum(0), (g * z).abs().sum(0)
        r["grad_bias"], r["size_bias"] = g.sum(0), g.abs().sum(0)
        g = g * x["weight"].double()
    r["grad_x"] = (g - g.mean(1, keepdim=True) - z * (g * z).mean(1, keepdim=True)) * rstd
    if x["grad_skip"] is not None:
        r["grad_x"] = r["grad_x"] + x["grad_skip"].double()
    return r


def compare(r, ref, dtype):
    for n, want in ref.items():
        if n.startswith("size"):
            continue
        err, u = (r[n].double() - want).norm(), U["f32" if n == "stats" else dtype]
        bound = (3e-6 + u) * want.norm() + 1e-30
        if n in ("grad_weight", "grad_bias"):
            bound = 3e-6 * ref[n.replace("grad", "size")].norm() + u * want.norm() + 1e-30
        assert err <= bound, (n, float(err), float(bound))


# rows of one lane to eight warps, of one to eight vectors a lane, some with idle places
SHAPES = [(1, 8), (2, 1024), (5, 16), (1000, 24), (513, 40), (333, 72), (700, 96), (129, 128), (77, 200), (300, 256),
          (65, 264), (50, 512), (41, 520), (33, 776), (2013, 64), (9, 1032), (12, 1536), (7, 2048), (31, 4096),
          (3, 4104), (21, 8192), (10, 6152)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,c", SHAPES)
def test_against_64_bits(dtype, n, c):
    x = make(n, c, dtype, affine=n % 3 != 0, skip=n % 2 == 0, seed=n + c, wide=n % 5 == 0)
    compare(call(x), reference(x), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,skip", [(40_001, 64, True), (10_001, 1024, False), (5_003, 1024, True), (3_001, 4096, True)])
def test_many_rows(dtype, n, c, skip):
    x = make(n, c, dtype, skip=skip, seed=2)
    compare(call(x), reference(x), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_without_spread(dtype):
    """A row of equal values has variance zero: y is the bias, rstd 1 / sqrt(eps)."""
    x = make(50, 64, dtype, seed=4)
    x["x"][7] = 3.0
    x["x"][8] = 0.0
    compare(call(x, eps=1e-3), reference(x, eps=1e-3), dtype)


@pytest.mark.parametrize("c", [64, 1024, 4096])
def test_a_mean_far_from_zero(c):
    """Values around 1000 of spread 1: the mean is known to about 8 roundings of 1000 2^-24 = 5e-4, which is the
    error of z; a variance from the difference of squares would be off by 1000^2 2^-24 = 0.06."""
    x = make(100, c, "f32", seed=5, offset=1000.0)
    r, ref = call(x), reference(x)
    for n in ("y", "grad_x", "grad_weight"):
        assert (r[n].double() - ref[n]).norm() <= 5e-4 * ref[n].norm(), n
    assert (r["stats"][:, 1].double() - ref["stats"][:, 1]).norm() <= 1e-5 * ref["stats"][:, 1].norm()


def test_values_that_are_not_finite_stay_in_their_row():
    x = make(70, 200, "f32", seed=6)
    want = call(x)
    x["x"][11, 5], x["x"][20, 0], x["x"][33, 7] = float("inf"), float("nan"), -float("inf")
    got = call(x)
    bad = torch.tensor([11, 20, 33], device="cuda")
    good = torch.ones(70, dtype=torch.bool, device="cuda").index_fill(0, bad, False)
    for n in ("y", "grad_x", "stats"):
        assert torch.equal(got[n][good], want[n][good]), n
        assert not got[n][bad].isfinite().all(1).any(), n


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_no_rows(dtype):
    r = call(make(0, 64, dtype))
    assert not r["grad_weight"].any() and not r["grad_bias"].any()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("c", [64, 1032])
def test_in_place_and_on_another_stream(dtype, c):
    x = make(333, c, dtype, skip=True, seed=6)
    want = call(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, stats, ws = x["x"].clone(), torch.empty(333, 2, device="cuda"), ops.layer_norm_workspace(333, c)
    s.wait_stream(torch.cuda.current_stream())
    ops.vg_layer_norm_fwd(y, x["weight"], x["bias"], y, stats, eps=EPS, stream=s)
    gw, gb = torch.empty_like(x["weight"]), torch.empty_like(x["bias"])
    ops.vg_layer_norm_bwd(x["x"], x["weight"], stats, x["grad_y"], x["grad_skip"], x["grad_y"], gw, gb, ws, stream=s)
    s.synchronize()
    assert torch.equal(y, want["y"]) and torch.equal(stats, want["stats"])
    assert torch.equal(x["grad_y"], want["grad_x"])
    assert torch.equal(gw, want["grad_weight"]) and torch.equal(gb, want["grad_bias"])


def test_outputs_that_are_not_wanted():
    x = make(90, 96, "bf16", seed=7)
    want = call(x)
    y, gx, gb = torch.empty_like(x["x"]), torch.empty_like(x["x"]), torch.empty_like(x["bias"])
    ops.vg_layer_norm_fwd(x["x"], x["weight"], x["bias"], y, None, eps=EPS)
    assert torch.equal(y, want["y"])
    ops.vg_layer_norm_bwd(x["x"], x["weight"], want["stats"], x["grad_y"], None, gx, None, None, None)
    assert torch.equal(gx, want["grad_x"])
    ops.vg_layer_norm_bwd(x["x"], x["weight"], want["stats"], x["grad_y"], None, gx, None, gb,
                          ops.layer_norm_workspace(90, 96))
    assert torch.equal(gb, want["grad_bias"])
    # a weight without a bias, and the other way round
    ref = reference({**x, "bias": torch.zeros_like(x["bias"])})
    ops.vg_layer_norm_fwd(x["x"], x["weight"], None, y, None, eps=EPS)
    compare({"y": y}, {"y": ref["y"]}, "bf16")
    ref = reference({**x, "weight": torch.ones_like(x["weight"])})
    ops.vg_layer_norm_fwd(x["x"], None, x["bias"], y, None, eps=EPS)
    compare({"y": y}, {"y": ref["y"]}, "bf16")


def test_neighbouring_columns_are_left_alone():
    base = torch.full((100, 96), 7.0, device="cuda")
    x = make(100, 64, "f32", seed=8)
    ops.vg_layer_norm_fwd(x["x"], x["weight"], x["bias"], base[:, 16:80], None)
    assert (base[:, :16] == 7).all() and (base[:, 80:] == 7).all()
    assert torch.equal(base[:, 16:80], call(x)["y"])


def test_the_same_from_run_to_run_and_in_a_graph():
    x = make(20_000, 128, "bf16", skip=True, seed=9)
    a, b = call(x), call(x)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    ws = ops.layer_norm_workspace(20_000, 128)
    for t in a.values():
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.vg_layer_norm_fwd(x["x"], x["weight"], x["bias"], a["y"], a["stats"], eps=EPS)
        ops.vg_layer_norm_bwd(x["x"], x["weight"], a["stats"], x["grad_y"], x["grad_skip"], a["grad_x"],
                              a["grad_weight"], a["grad_bias"], ws)
    graph.replay()
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_gradients_against_differences():
    """Central differences of sum(y * g) in fp32 at h = 1e-2: truncation h^2 of third derivatives of order 1, and
    rounding 1e-7 * sqrt(size) / h: 1e-3 of the gradient's norm."""
    x = make(60, 48, "f32", seed=10)
    r = call(x)
    g = torch.Generator(device="cuda").manual_seed(3)
    for what, grad in (("x", "grad_x"), ("weight", "grad_weight"), ("bias", "grad_bias")):
        dirn = torch.randn(x[what].shape, generator=g, device="cuda")
        side = []
        for h in (1e-2, -1e-2):
            y = dict(x)
            y[what] = (x[what] + h * dirn).contiguous()
            side.append((call(y)["y"].double() * x["grad_y"].double()).sum())
        diff = float(side[0] - side[1]) / 2e-2
        assert abs(diff - float((r[grad].double() * dirn.double()).sum())) <= 3e-3 * float(r[grad].double().norm()), what
