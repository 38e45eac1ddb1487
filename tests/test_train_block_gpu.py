"""examples/train_block.py: the operators together, as a training step (GPU)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from voxel_gemm_gb300 import synth

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def reference(block, x, context, lengths):
    """The block's formulas in 64 bits from torch's own operations, for autograd: out and its leaves."""
    leaf = [t.double().requires_grad_() for t in (x, *block.params)]
    xs, w, b, qw, kw, kvw = leaf
    nbr = block.map.nbr.long()
    rows = torch.cat([xs, xs.new_zeros(1, xs.shape[1])])  # the last one: no neighbour
    y = b + sum(rows[torch.where(nbr[:, k] < 0, xs.shape[0], nbr[:, k])] @ w[k] for k in range(27))
    n, (h, d), hk = xs.shape[0], qw.shape, kw.shape[0]
    y = y.view(n, h, d)

    def norm(t, weight):
        return t * (t.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * weight
    q = norm(y, qw)
    axis = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(block.pairs, device="cuda"))
    angle = (block.coords[:, 1:].float()[:, axis] * block.freqs).double()[:, None, :]
    turned = 2 * axis.numel()
    a, c = q[..., 0:turned:2], q[..., 1:turned:2]
    pairs = torch.stack([a * angle.cos() - c * angle.sin(), a * angle.sin() + c * angle.cos()], -1)
    q = torch.cat([pairs.flatten(-2), q[..., turned:]], -1)
    kv = (context.double() @ kvw).view(-1, 2, hk, d)
    k, v = norm(kv[:, 0], kw), kv[:, 1]
    out = []
    sizes = torch.bincount(block.coords[:, 0], minlength=len(lengths)).tolist()
    for qs, ks, vs in zip(q.split(sizes), k.split(lengths), v.split(lengths)):
        ks, vs = (t.repeat_interleave(h // hk, 1) for t in (ks, vs))
        p = torch.einsum("ihd,jhd->hij", qs, ks).mul(d ** -0.5).softmax(-1) if ks.shape[0] else None
        out.append(torch.zeros_like(qs) if p is None else torch.einsum("hij,jhd->ihd", p, vs))
    return y + torch.cat(out), leaf


def test_step_against_autograd():
    """fp32, one sample without states.  Each operator is within 1e-5 (the library's fp32 bound) and a gradient passes
    at most ten of them, forward and backward."""
    ex, lengths, width, c = example(), [7, 0, 12], 24, 32
    coords = synth.random_coords(3, 400, 3, 9, 9, 9)
    coords = torch.from_numpy(coords[np.argsort(coords[:, 0], kind="stable")]).cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    x, grad = (torch.randn(coords.shape[0], c, generator=g, device="cuda") for _ in range(2))
    context = torch.randn(sum(lengths), width, generator=g, device="cuda")
    block = ex.VoxelBlock(coords, (3, 9, 9, 9), c, torch.float32, lengths, heads=4, kv_heads=2, state_width=width)
    for p in block.params[1:4]:
        p.add_(0.3 * torch.randn(p.shape, generator=g, device="cuda"))
    grad = grad.view(coords.shape[0], 4, c // 4)
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    out = block.forward(x, context)
    d_x = block.backward(x, context, grad)
    torch.backends.cuda.matmul.allow_tf32 = old
    block.check()
    ref, leaf = reference(block, x, context, lengths)
    ref.backward(grad.double())
    names = ("x", "conv weight", "conv bias", "q weight", "k weight", "kv weight")
    for name, got, want in [("out", out, ref.detach()), *zip(names, [d_x, *block.grads], [t.grad for t in leaf])]:
        err = (got.double() - want).norm() / want.norm()
        assert err < 1e-4, (name, float(err))


@pytest.mark.parametrize("dtype,bits", [("f32", 32), ("f16", 8), ("bf16", 8), ("bf16", 32)])
def test_loss_falls_and_steps_repeat(dtype, bits):
    ex, lengths = example(), [20, 33]
    wl = synth.Workload("train_block", 2, 24, 2, ("sphere", "torus"), 64, 64, dtype, 5, 2.0)
    runs = []
    for _ in range(2):
        coords, x, context, target = ex.make_inputs(wl, lengths, 40)
        block = ex.VoxelBlock(coords, wl.grid, wl.cin, x.dtype, lengths, 4, 2, 40, bits)
        runs.append([float(block.train_step(x, context, target, step, 3e-3)) for step in range(1, 21)])
        block.check()
    assert runs[0] == runs[1]
    assert runs[0][-1] < 0.8 * runs[0][0]


def test_command(capsys):
    example().main(["--workload", "sphere16_c32_f32", "--steps", "3", "--states", "9"])
    assert capsys.readouterr().out.count("loss") == 3
