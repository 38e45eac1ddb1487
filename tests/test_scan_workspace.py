"""One workspace of the gated scan serves every call of fewer tokens (CPU only)."""
import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from voxel_gemm_gb300 import build, ops
    build.build()
    return ops


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("c", [8, 16, 64, 72, 256, 520, 1024, 4096])
def test_a_workspace_serves_fewer_tokens(ops, dtype, c):
    """Steps of 1.3 % from nothing to a few million tokens, with the rows around multiples of whole tiles."""
    n, sizes = 1, [0]
    while n < 8_000_000:
        sizes += [n, n // 2048 * 2048, n // 2048 * 2048 + 1]
        n += max(1, n // 77)
    before = 0
    for n in sorted(set(sizes)):
        need = ops.lib().vg_gated_scan_workspace_bytes(ops.ScanStruct(n, c, 3, ops._DT[dtype], 0, None, None))
        assert need >= before, (n, need, before)
        before = need


def test_a_workspace_stays_small_beside_the_tokens(ops):
    """No more than a 16-bit operand of the call itself, or than 8 tiles."""
    for n in (1, 2048, 25_179, 467_000, 602_492, 4_915_386):
        for c in (8, 64, 512):
            need = ops.lib().vg_gated_scan_workspace_bytes(ops.ScanStruct(n, c, 1, ops.VG_BF16, 0, None, None))
            assert need <= max(n, 8 * 76) * c * 2 + 512, (n, c, need)
