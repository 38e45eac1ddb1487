"""The recurrent-block operators together, and examples/train_block.py with its recurrent part (GPU)."""
import numpy as np
import pytest
import torch

from test_dropout_gpu import words
from test_train_block_gpu import example, reference as block_reference

from voxel_gemm_gb300 import ops, synth

pytestmark = pytest.mark.gpu


def curve_reference(scan, z, w, b, proj):
    """The recurrent part's formulas in 64 bits from torch's own operations, for autograd."""
    n = (z - z.mean(1, keepdim=True)) / (z.var(1, correction=0, keepdim=True) + 1e-5).sqrt() * w + b
    gate, u = (n @ proj).chunk(2, 1)
    a = torch.sigmoid(gate)
    order, off, h = scan.order.tolist(), scan.off.tolist(), [None] * z.shape[0]
    for lo, hi in zip(off, off[1:]):
        state = torch.zeros_like(z[0])
        for row in order[lo:hi]:
            state = a[row] * state + (1 - a[row]) * u[row]
            h[row] = state
    seed, step = scan.rng.tolist()
    keep = torch.from_numpy(words(z.numel(), seed, step, scan.CALL) >= round(scan.p * 2 ** 32)).cuda().view(z.shape)
    return z + torch.stack(h) * keep / (1 - scan.p)


def close(pairs, bound):
    for name, got, want in pairs:
        err = (got.double() - want).norm() / want.norm()
        assert err < bound, (name, float(err))


def make_part(dtype, p, n_per=(70, 0, 151), grid=(3, 9, 9, 9), c=48, seed=3):
    ex = example()
    rng = np.random.default_rng(seed)
    coords = []
    for i, n in enumerate(n_per):
        cells = rng.choice(grid[1] * grid[2] * grid[3], n, replace=False)
        coords += [(i, v // 81, v // 9 % 9, v % 9) for v in cells]
    coords = torch.tensor(coords, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
    part = ex.CurveScan(coords, grid, c, dtype, ex.offsets(list(n_per)), p, randn, seed=seed)
    for t in part.params[:2]:
        t.add_(randn(c, std=0.3))
    part.rng[1] = 7
    return part, randn(sum(n_per), c), randn(sum(n_per), c)


def test_the_order_follows_the_curve():
    """Each sample's voxels in a row of the codes, the samples one after another."""
    part, _, _ = make_part(torch.float32, 0.1)
    assert sorted(part.order.tolist()) == list(range(221))
    assert sorted(part.order[:70].tolist()) == list(range(70))


@pytest.mark.parametrize("p", [0.0, 0.25])
def test_part_against_autograd(p):
    """fp32: each operator is within 2e-5 and a gradient passes three of them and two matrix products: 1e-4."""
    part, z, grad = make_part(torch.float32, p)
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    out = part.forward(z)
    grads = [torch.empty_like(t) for t in part.params]
    d_z = part.backward(grad, grads)
    torch.backends.cuda.matmul.allow_tf32 = old
    assert ops.vg_gated_scan_status(part.scan_ws) == ops.VG_OK
    leaf = [t.double().requires_grad_() for t in (z, *part.params)]
    ref = curve_reference(part, *leaf)
    ref.backward(grad.double())
    close([("out", out, ref.detach()), *zip(("z", "norm weight", "norm bias", "projection"), [d_z, *grads],
                                            [t.grad for t in leaf])], 1e-4)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_part_in_16_bits(dtype):
    """Roundings on the way, half a step each: the norm's output, the product's, the scan's and the sum's forwards (the
    first three pass through slopes of about one); backwards those again and as many of gradients: 8 of them, each
    at most u, and a share of the values that is about one."""
    u = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    part, z, grad = make_part(dtype, 0.25)
    out = part.forward(z)
    grads = [torch.empty_like(t) for t in part.params]
    d_z = part.backward(grad, grads)
    leaf = [t.double().requires_grad_() for t in (z, *part.params)]
    ref = curve_reference(part, *leaf)
    ref.backward(grad.double())
    close([("out", out, ref.detach())], 4 * u)
    close(zip(("z", "norm weight", "norm bias", "projection"), [d_z, *grads], [t.grad for t in leaf]), 8 * u)


def test_step_against_autograd():
    """The whole block with its recurrent part; bounds as for the block alone, with three operators more."""
    ex, lengths, width, c = example(), [7, 0, 12], 24, 32
    coords = synth.random_coords(3, 300, 3, 9, 9, 9)
    coords = torch.from_numpy(coords[np.argsort(coords[:, 0], kind="stable")]).cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    x, grad = (torch.randn(coords.shape[0], c, generator=g, device="cuda") for _ in range(2))
    context = torch.randn(sum(lengths), width, generator=g, device="cuda")
    block = ex.VoxelBlock(coords, (3, 9, 9, 9), c, torch.float32, lengths, heads=4, kv_heads=2, state_width=width,
                          scan=True, dropout=0.2)
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    out = block.forward(x, context)
    d_x = block.backward(x, context, grad.view(out.shape))
    torch.backends.cuda.matmul.allow_tf32 = old
    block.check()
    params, block.params = block.params, block.params[:5]
    first, leaf = block_reference(block, x, context, lengths)
    more = [t.double().requires_grad_() for t in params[5:]]
    ref = curve_reference(block.scan, first.reshape(x.shape), *more)
    ref.backward(grad.double())
    names = ("x", "conv weight", "conv bias", "q weight", "k weight", "kv weight", "norm weight", "norm bias", "projection")
    close([("out", out, ref.detach().view(out.shape)),
           *zip(names, [d_x, *block.grads], [t.grad for t in (*leaf, *more)])], 1.5e-4)


@pytest.mark.parametrize("dtype,bits", [("f32", 32), ("f16", 8), ("bf16", 32)])
def test_steps_run_and_repeat(dtype, bits):
    ex, lengths = example(), [20, 33]
    wl = synth.Workload("train_block", 2, 24, 2, ("sphere", "torus"), 64, 64, dtype, 5, 2.0)
    runs = []
    for _ in range(2):
        coords, x, context, target = ex.make_inputs(wl, lengths, 40)
        block = ex.VoxelBlock(coords, wl.grid, wl.cin, x.dtype, lengths, 4, 2, 40, bits, scan=True, dropout=0.1)
        runs.append([float(block.train_step(x, context, target, step, 3e-3)) for step in range(1, 11)])
        assert block.scan.rng.tolist() == [0, 10]
        block.check()
    assert runs[0] == runs[1] and np.isfinite(runs[0]).all()


def test_command(capsys):
    example().main(["--workload", "sphere16_c32_f32", "--steps", "3", "--states", "9", "--scan", "--dropout", "0.2"])
    assert capsys.readouterr().out.count("loss") == 3


def test_serving_goes_on_from_a_scan():
    """A scan over the first tokens of each sequence leaves the states from which single steps go on."""
    b, t0, t1, c = 3, 100, 20, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    gate, x = (torch.randn(b, t0 + t1, c, generator=g, device="cuda") + 1 for _ in range(2))

    def scan(gate, x, t):
        off = torch.arange(b + 1, dtype=torch.int32, device="cuda") * t
        out, last = torch.empty(b * t, c, device="cuda"), torch.empty(b, c, device="cuda")
        ws = ops.gated_scan_workspace(b * t, c, b, torch.float32)
        ops.vg_gated_scan_fwd(gate.reshape(-1, c), x.reshape(-1, c), off, None, None, out, last, None, ws)
        return out.view(b, t, c), last
    whole, _ = scan(gate, x, t0 + t1)
    out, state = scan(gate[:, :t0], x[:, :t0], t0)
    assert (out - whole[:, :t0]).abs().max() < 1e-5
    for t in range(t0, t0 + t1):
        y = torch.empty(b, c, device="cuda")
        ops.vg_gated_scan_step(gate[:, t], x[:, t], state, y)
        assert (y - whole[:, t]).abs().max() < 1e-5
