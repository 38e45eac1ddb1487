"""examples/train_block.py in 16 bits at sums that are large (GPU)."""
import pytest

from test_train_block_gpu import example
from voxel_gemm_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_sums_over_many_voxels_stay_in_range(dtype):
    """A weight's gradient is a sum over the voxels, here of some 6,000 values of 50 and more: the step has to keep it
    below fp16's 65,504, and the loss has to fall."""
    ex, lengths = example(), [20, 33]
    wl = synth.Workload("train_block", 2, 40, 2, ("sphere", "torus"), 64, 64, dtype, 5, 2.0)
    coords, x, context, target = ex.make_inputs(wl, lengths, 40)
    target = target * 64
    block = ex.VoxelBlock(coords, wl.grid, wl.cin, x.dtype, lengths, 4, 2, 40, 32)
    losses = [float(block.train_step(x, context, target, step, 3e-2)) for step in range(1, 21)]
    block.check()
    assert all(g.isfinite().all() for g in block.grads)
    assert all(p.isfinite().all() for p in block.params)
    assert losses[-1] < losses[0]
