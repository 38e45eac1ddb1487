"""vg_dropout_add_fwd / _bwd against the generator's definition in whole numbers and the sum in 64 bits (GPU).

The mask has to be equal.  Values: one fp32 product and one fp32 sum, 2^-24 of each one's size, and the rounding to
the type, u of the result.
"""
import numpy as np
import pytest
import torch

from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def philox(counter, key):
    """Words [groups, 4] of counters [groups, 4] under a key of two 32-bit numbers (whole numbers of any size)."""
    c = [counter[:, i].astype(np.uint64) for i in range(4)]
    k0, k1, m = key[0], key[1], np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        s = np.uint64(32)
        c = [(q >> s) ^ c[1] ^ np.uint64(k0), q & m, (p >> s) ^ c[3] ^ np.uint64(k1), p & m]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1)


def words(n, seed, step, call):
    g = np.arange((n + 3) // 4, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    ctr = np.stack([g & low, g >> np.uint64(32), np.full_like(g, step & 0xFFFFFFFF), np.full_like(g, call)], 1)
    return philox(ctr, (seed & 0xFFFFFFFF, seed >> 32)).reshape(-1)[:n]


def test_generator_answers():
    """The answers published with the generator for all zeros, all ones, and the digits of pi."""
    for ctr, key, want in [
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]:
        assert tuple(int(v) for v in philox(np.array([ctr], dtype=np.uint64), key)[0]) == want


def state(seed, step):
    return torch.tensor(np.array([seed, step], dtype=np.uint64).view(np.int64)).cuda()


def tensors(n, dtype, seed=0, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(n + shift, generator=g, device="cuda").to(DT[dtype])[shift:] for _ in range(3)]


SEED = 0xFEDCBA9876543210


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])       # 1: pointers that are not aligned
@pytest.mark.parametrize("n,p", [(1, 0.5), (3, 0.1), (7, 0.9), (8, 0.5), (31, 0.0), (1025, 0.25), (99_999, 0.1),
                                 (1_300_003, 0.5)])
def test_against_the_definition(dtype, shift, n, p):
    x, res, grad = tensors(n, dtype, seed=n, shift=shift)
    step, call = 0x1234567890, 0xFFFFFFFE
    rng = state(SEED, step)
    keep = torch.from_numpy(words(n, SEED, step, call) >= round(p * 2 ** 32)).cuda()
    out, alone, gx = (torch.full_like(x, float("nan")) for _ in range(3))
    ops.vg_dropout_add_fwd(x, res, p, rng, call, out)
    ops.vg_dropout_add_fwd(x, None, p, rng, call, alone)
    ops.vg_dropout_add_bwd(grad, p, rng, call, gx)
    u = U[dtype]
    for got, of, add in ((out, x, res), (alone, x, None), (gx, grad, None)):
        part = torch.where(keep, of.double() / (1 - p), 0.0)
        want = part if add is None else part + add.double()
        size = part.abs() + (0 if add is None else add.double().abs())
        # 2^-24: the rounded factor, the product and the sum; half of fp16's smallest step at the bottom
        assert ((got.double() - want).abs() <= u * want.abs() + 3 * 2.0 ** -24 * size + 2.0 ** -25).all()
    assert torch.equal(alone[~keep], torch.zeros_like(alone[~keep]))
    assert torch.equal(out[~keep], res[~keep])
    assert torch.equal((gx != 0), keep & (grad != 0))


def test_dropped_values_do_not_matter():
    """A dropped element is zero whatever x holds."""
    n, p, rng = 4096, 0.5, state(7, 1)
    x, res, _ = tensors(n, "f32")
    keep = torch.from_numpy(words(n, 7, 1, 0) >= 2 ** 31).cuda()
    want = torch.empty_like(x)
    ops.vg_dropout_add_fwd(x, res, p, rng, 0, want)
    x[~keep] = torch.tensor([float("nan"), float("inf")], device="cuda").repeat(n)[:int((~keep).sum())]
    out = torch.empty_like(x)
    ops.vg_dropout_add_fwd(x, res, p, rng, 0, out)
    assert torch.equal(out, want)


def test_share_and_separate_calls():
    """The share kept is 1 - p within five standard deviations; calls, steps and seeds have masks of their own, which
    agree at about the chance share."""
    n, p = 1 << 20, 0.3
    x = torch.ones(n, device="cuda")
    masks = []
    for seed, step, call in ((1, 0, 0), (1, 0, 1), (1, 1, 0), (2, 0, 0), (1 + (1 << 40), 0, 0)):
        out = torch.empty_like(x)
        ops.vg_dropout_add_fwd(x, None, p, state(seed, step), call, out)
        masks.append(out != 0)
        assert abs(float(masks[-1].double().mean()) - (1 - p)) < 5 * (p * (1 - p) / n) ** 0.5
    same = (1 - p) ** 2 + p ** 2
    for i in range(len(masks)):
        for j in range(i):
            assert abs(float((masks[i] == masks[j]).double().mean()) - same) < 5 * (same * (1 - same) / n) ** 0.5


def test_the_mask_does_not_depend_on_type_or_shape():
    n, p, rng = 24_000, 0.4, state(99, 5)
    masks = []
    for dtype in DT:
        x = torch.ones(n, dtype=DT[dtype], device="cuda").view(4, 100, -1)
        out = torch.empty_like(x)
        ops.vg_dropout_add_fwd(x, None, p, rng, 2, out)
        masks.append((out != 0).view(-1))
    assert torch.equal(masks[0], masks[1]) and torch.equal(masks[0], masks[2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_another_stream_and_a_graph_that_counts(dtype):
    x, res, _ = tensors(50_001, dtype)
    rng, p = state(3, 10), 0.1
    want = []
    for step in (10, 11, 12):
        out = torch.empty_like(x)
        ops.vg_dropout_add_fwd(x, res, p, state(3, step), 4, out)
        want.append(out)
    s = torch.cuda.Stream()
    a, b = x.clone(), res.clone()
    s.wait_stream(torch.cuda.current_stream())
    ops.vg_dropout_add_fwd(a, res, p, rng, 4, a, stream=s)
    ops.vg_dropout_add_fwd(x, b, p, rng, 4, b, stream=s)
    s.synchronize()
    assert torch.equal(a, want[0]) and torch.equal(b, want[0])
    out, graph = torch.empty_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.vg_dropout_add_fwd(x, res, p, rng, 4, out)
        rng[1] += 1
    for w in want:
        graph.replay()
        assert torch.equal(out, w)


def test_nothing_to_drop():
    x = torch.empty(0, device="cuda")
    ops.vg_dropout_add_fwd(x, None, 0.5, state(1, 1), 0, x)
    ops.vg_dropout_add_bwd(x, 0.5, state(1, 1), 0, x)
