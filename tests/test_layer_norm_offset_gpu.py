"""vg_layer_norm_bwd where a row's mean is far larger than its spread, or its spread tiny (GPU).

Whole numbers, times a power of two, around a mean that fp32 holds exactly, so that x - mean has no rounding and
z = (x - mean) rstd has one, 2^-24 of z.  Everything after it is fp32 sums; only what the mean could add is kept apart from them.
"""
import pytest
import torch

from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.mark.parametrize("n,c,mean,unit", [(257, 64, 70_001.0, 1.0), (33, 72, 99_991.0, 1.0), (5, 1024, 1_000_003.0, 1.0),
                                           (9, 4096, 70_001.0, 1.0), (3, 8192, 5_003.0, 1.0), (65, 128, 0.0, 2.0 ** -60)])
@pytest.mark.parametrize("skip", [False, True])
def test_a_mean_far_above_the_spread(n, c, mean, unit, skip):
    g = torch.Generator(device="cuda").manual_seed(c)
    half = torch.randint(1, 4, (n, c // 2), generator=g, device="cuda").float()
    off = torch.cat([half, -half], 1)
    x = mean + off * unit
    gy = torch.randn(n, c, generator=g, device="cuda")
    rstd = off.square().mean(1).rsqrt() / unit
    stats = torch.stack([torch.full((n,), mean, device="cuda"), rstd], 1)
    k = torch.randn(n, c, generator=g, device="cuda") if skip else None
    gx, gw, gb = torch.empty_like(x), torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    ops.vg_layer_norm_bwd(x, None, stats, gy, k, gx, gw, gb, ops.layer_norm_workspace(n, c))
    r, gd = stats[:, 1:].double(), gy.double()
    z = off.double() * unit * r
    # a column's sum: products and running sums of n terms
    assert ((gw.double() - (gd * z).sum(0)).abs() <= (n + 4) * E * (gd * z).abs().sum(0)).all()
    along, m = (gd * z).mean(1, keepdim=True), gd.mean(1, keepdim=True)
    want = (gd - m - z * along) * r + (k.double() if skip else 0.0)
    # the row's sums: at most 64 terms a lane in two chains, 8 exchanges, three factors
    size = (gd.abs() + 50 * (gd.abs().mean(1, keepdim=True) + z.abs() * (gd * z).abs().mean(1, keepdim=True))) * r
    assert ((gx.double() - want).abs() <= 4 * E * size + E * want.abs()).all()
