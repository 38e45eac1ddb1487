"""Numbers that the C entry points would take only in part are refused (CPU only; no call here is complete)."""
from types import SimpleNamespace

import pytest
import torch

from test_binding_devices import gpu

from voxel_gemm_gb300 import ops


@pytest.fixture(scope="module", autouse=True)
def built():
    from voxel_gemm_gb300 import build
    build.build()


@pytest.mark.parametrize("call", [-1, 2 ** 32, 2 ** 32 + 3, 2 ** 64])
def test_a_call_number_beyond_32_bits(call):
    """Its mask would be another call's.  (On the CPU: what is on the GPU only by name would be refused later.)"""
    x, rng = gpu(torch.zeros(64)), gpu(torch.zeros(2, dtype=torch.int64))
    bad = torch.zeros(64)                       # were the number taken, this operand would be refused by name of the GPU
    with pytest.raises(ValueError, match="32 bits"):
        ops.vg_dropout_add_fwd(x, None, 0.5, rng, call, bad)
    with pytest.raises(ValueError, match="32 bits"):
        ops.vg_dropout_add_bwd(x, 0.5, rng, call, bad)


@pytest.mark.parametrize("flags", [-1, 2 ** 32, 2 ** 32 + ops.VG_SCAN_REVERSE])
def test_flags_beyond_32_bits(flags):
    x, off = gpu(torch.zeros(4, 64)), gpu(torch.tensor([0, 4], dtype=torch.int32))
    ws, bad = gpu(torch.zeros(4096, dtype=torch.uint8)), torch.zeros(4, 64)
    for f in (lambda: ops.vg_gated_scan_fwd(x, x, off, None, None, bad, None, None, ws, flags=flags),
              lambda: ops.vg_gated_scan_bwd(x, x, off, None, None, None, x, None, x, bad, None, ws, flags=flags),
              lambda: ops.vg_gated_scan_step(x, x, x, bad, flags=flags)):
        with pytest.raises(ValueError, match="32 bits"):
            f()


def test_no_workspace():
    """The library's status, as for any other argument that is missing."""
    x, off = gpu(torch.zeros(4, 64)), gpu(torch.tensor([0, 4], dtype=torch.int32))
    h, kept = gpu(torch.zeros(1, 64)), gpu(torch.zeros(1, 64))
    s = SimpleNamespace(cuda_stream=0, device_index=0)
    for f in (lambda: ops.vg_gated_scan_fwd(x, x, off, None, None, x, h, kept, None, stream=s),
              lambda: ops.vg_gated_scan_bwd(x, x, off, None, None, kept, x, None, x, x, h, None, stream=s)):
        with pytest.raises(ops.VGError) as e:
            f()
        assert e.value.status == ops.VG_ERR_INVALID_ARG
