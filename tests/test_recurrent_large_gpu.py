"""Dropout and layer norm at sizes at which every thread or group of lanes takes several turns (GPU)."""
import numpy as np
import pytest
import torch

import test_dropout_gpu as drop
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
