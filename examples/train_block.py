"""Train one block of voxel tokens that read an encoder's states: convolution, attention, optimizer.

    y   = submanifold convolution of the voxel features x
    q   = norm(y) turned by the voxels' x, y, z;  k = norm(context Wk);  v = context Wv
    out = y + softmax(scale q k^T) v over the states of the voxel's own sample
    loss = mean((out - target)^2) / 2

With --scan a recurrent part follows, which mixes each sample's voxels along a Hilbert curve:

    [g, u] = layer norm(out) W,  h_t = sigmoid(g_t) h_{t-1} + (1 - sigmoid(g_t)) u_t,  out += dropout(h)

Forward, backward and the AdamW step run on the library (the products of the context with
[Wk, Wv], of the norm with W, and their gradients are plain matrix products).  Seeded synthetic inputs:

    python examples/train_block.py [--workload NAME] [--heads H] [--states M] [--steps K] [--bits 8|32] [--lr LR]
                                   [--scan] [--dropout P]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from voxel_gemm_gb300 import ops, synth  # noqa: E402


def offsets(lengths):
    """int32 [B + 1] on the GPU: 0 and the running sums."""
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


class CurveScan:
    """out = z + dropout(scan(layer norm(z) W)) for tokens z [N, channels], along a Hilbert curve through each sample's
    voxels; params are the norm's weight and bias, and W [channels, 2 channels].  A step's dropout masks are
    those of rng = (seed, step)."""

    CALL = 0  # the number of this dropout among those of a step

    def __init__(self, coords, grid, channels, dtype, q_off, dropout, randn, seed):
        n = coords.shape[0]
        bits = max(max(grid[1:]) - 1, 1).bit_length()
        codes = torch.empty(n, dtype=torch.int64, device="cuda")
        ops.vg_encode_seq(coords, bits, ops.VG_CURVE_HILBERT, codes)
        self.order, self.off, self.p = torch.argsort(codes).int(), q_off, dropout
        self.rng = torch.tensor([seed, 0], device="cuda")

        def empty(*shape, dt=dtype):
            return torch.empty(*shape, dtype=dt, device="cuda")
        self.params = [empty(channels).fill_(1), empty(channels).zero_(), randn(channels, 2 * channels, std=channels ** -0.5)]
        self.norm, self.h, self.out, self.d_h, self.d_z = (empty(n, channels) for _ in range(5))
        self.stats, self.d_gu = empty(n, 2, dt=torch.float32), empty(n, 2 * channels)
        self.carries = ops.gated_scan_carries(n, channels)
        self.norm_ws = ops.layer_norm_workspace(n, channels)
        self.scan_ws = ops.gated_scan_workspace(n, channels, q_off.numel() - 1, dtype)

    def forward(self, z):
        self.z, (w, b, proj) = z, self.params
        ops.vg_layer_norm_fwd(z, w, b, self.norm, self.stats)
        self.gate, self.u = (self.norm @ proj).chunk(2, 1)
        ops.vg_gated_scan_fwd(self.gate, self.u, self.off, self.order, None, self.h, None, self.carries, self.scan_ws)
        ops.vg_dropout_add_fwd(self.h, z, self.p, self.rng, self.CALL, self.out)
        return self.out

    def backward(self, grad_out, grads):
        """Gradients of params into `grads`; of z, returned."""
        d_w, d_b, d_proj = grads
        ops.vg_dropout_add_bwd(grad_out, self.p, self.rng, self.CALL, self.d_h)
        d_gate, d_u = self.d_gu.chunk(2, 1)
        ops.vg_gated_scan_bwd(self.gate, self.u, self.off, self.order, None, self.carries, self.d_h, None, d_gate, d_u,
                              None, self.scan_ws)
        torch.matmul(self.norm.t(), self.d_gu, out=d_proj)
        ops.vg_layer_norm_bwd(self.z, self.params[0], self.stats, self.d_gu @ self.params[2].t(), grad_out, self.d_z,
                              d_w, d_b, self.norm_ws)
        return self.d_z


class VoxelBlock:
    """The block over a fixed set of voxels, its buffers, parameters and optimizer state.

    coords [N, 4] (batch element, x, y, z), rows of a batch element together; state_lengths, the encoder states of
    each batch element; heads query heads share kv_heads key and value heads; scan adds the recurrent part."""

    def __init__(self, coords, grid, channels, dtype, state_lengths, heads, kv_heads, state_width, bits=32, seed=0,
                 weight_decay=0.0, scan=False, dropout=0.0):
        n, m, d = coords.shape[0], int(sum(state_lengths)), channels // heads
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

        def empty(*shape):
            return torch.empty(*shape, dtype=dtype, device="cuda")
        self.coords = coords
        self.map = ops.NbrMap.alloc(n, grid).build(coords)
        self.conv_ws = ops.conv_workspace(n, channels, channels, dtype)
        self.q_off = offsets(np.bincount(coords[:, 0].cpu().numpy(), minlength=grid[0]))
        self.k_off = offsets(state_lengths)
        self.freqs, self.pairs = ops.rope_freqs(d)
        self.conv_w, self.conv_b = randn(27, channels, channels, std=(27 * channels) ** -0.5), empty(channels).zero_()
        self.q_w, self.k_w = empty(heads, d).fill_(1), empty(kv_heads, d).fill_(1)
        self.kv_w = randn(state_width, 2 * kv_heads * d, std=state_width ** -0.5)
        self.params = [self.conv_w, self.conv_b, self.q_w, self.k_w, self.kv_w]
        self.scan = CurveScan(coords, grid, channels, dtype, self.q_off, dropout, randn, seed) if scan else None
        self.params += self.scan.params if scan else []
        self.grads = [torch.empty_like(p) for p in self.params]
        masters = None if dtype == torch.float32 else [p.float() for p in self.params]
        self.opt = ops.AdamWState(self.params, self.grads, masters=masters, bits=bits, weight_decay=weight_decay)
        self.y, self.qn, self.att = (empty(n, heads, d) for _ in range(3))
        self.kn = empty(m, kv_heads, d)
        self.lse = torch.empty(heads, n, device="cuda")
        self.attn_ws = ops.cross_attn_workspace(n, m, len(state_lengths), heads, kv_heads, d, dtype, backward=True)
        self.q_ws = ops.qk_norm_rope_workspace(n, heads, 0, d)
        self.k_ws = ops.qk_norm_rope_workspace(m, 0, kv_heads, d)
        self.d_qn, self.d_y = torch.empty_like(self.qn), torch.empty_like(self.y)
        self.d_kn, self.d_kv = torch.empty_like(self.kn), empty(m, 2, kv_heads, d)
        self.d_x = empty(n, channels)

    def forward(self, x, context):
        """out [N, heads, head_dim]."""
        ops.vg_subm_conv3d_fwd(self.map.ws, self.map.nbr, self.map.mask, x, self.conv_w, self.conv_b,
                               self.y.view(x.shape), self.conv_ws)
        self.kv = (context @ self.kv_w).view(self.d_kv.shape)
        ops.vg_qk_norm_rope_fwd(self.y, None, self.q_w, None, self.coords, self.freqs, self.pairs, self.qn, None)
        ops.vg_qk_norm_rope_fwd(None, self.kv[:, 0], None, self.k_w, None, None, None, None, self.kn)
        ops.vg_cross_attn_fwd(self.qn, self.kn, self.kv[:, 1], self.q_off, self.k_off, None, self.att, self.lse,
                              self.attn_ws)
        out = self.y + self.att
        return out if self.scan is None else self.scan.forward(out.view(x.shape)).view(out.shape)

    def backward(self, x, context, grad_out):
        """Gradients of the parameters into self.grads; of x, returned."""
        d_w, d_b, d_qw, d_kw, d_kvw = self.grads[:5]
        if self.scan is not None:
            grad_out = self.scan.backward(grad_out.reshape(x.shape), self.grads[5:]).view(grad_out.shape)
        ops.vg_cross_attn_bwd(self.qn, self.kn, self.kv[:, 1], self.q_off, self.k_off, None, self.att, self.lse,
                              grad_out, self.d_qn, self.d_kn, self.d_kv[:, 1], self.attn_ws)
        ops.vg_qk_norm_rope_bwd(None, self.kv[:, 0], None, self.k_w, None, None, None, None, self.d_kn, None,
                                self.d_kv[:, 0], None, d_kw, self.k_ws)
        ops.vg_qk_norm_rope_bwd(self.y, None, self.q_w, None, self.coords, self.freqs, self.pairs, self.d_qn, None,
                                self.d_y, None, d_qw, None, self.q_ws)
        torch.matmul(context.t(), self.d_kv.view(context.shape[0], -1), out=d_kvw)
        d_y = (self.d_y + grad_out).view(x.shape)
        ops.vg_subm_conv3d_bwd(self.map.ws, self.map.nbr, self.map.mask, d_y, x, self.conv_w, self.d_x, d_w, d_b,
                               self.conv_ws)
        return self.d_x

    def train_step(self, x, context, target, step, lr):
        """One step of the loss against target [N, channels] (step counts from 1); returns the loss, on the GPU."""
        diff = self.forward(x, context) - target.view(self.y.shape)
        # The loss's gradient is diff / diff.numel().  In 16 bits the backward pass carries diff / 2^k, with 4^k about
        # the number of voxels, and the step divides by the rest: the weights' gradients, sums over the voxels, stay
        # far below 65,504, and the values that they are sums of far above fp16's smallest.
        scale = 1 / diff.numel() if diff.dtype == torch.float32 else 2.0 ** -round(math.log2(diff.shape[0]) / 2)
        self.backward(x, context, diff * scale)
        ops.vg_adamw_step(self.opt, step, lr, grad_scale=1 / (diff.numel() * scale))
        if self.scan is not None:
            self.scan.rng[1] += 1
        return diff.float().square().mean() / 2

    def check(self):
        """Raise if a kernel recorded an error."""
        status = [("neighbour map", self.map.status()), ("convolution", ops.vg_conv_status(self.conv_ws)),
                  ("attention", ops.vg_cross_attn_status(self.attn_ws))]
        if self.scan is not None:
            status.append(("scan", ops.vg_gated_scan_status(self.scan.scan_ws)))
        for name, st in status:
            if st != ops.VG_OK:
                raise ops.VGError(st, name)


def make_inputs(wl, state_lengths, state_width, seed=0):
    """coords (rows of a batch element together), x, context and target of a seeded workload."""
    coords = synth.make_coords(wl)
    coords = torch.from_numpy(coords[np.argsort(coords[:, 0], kind="stable")]).cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = synth.torch_dtype(wl.dtype)
    x = torch.randn(coords.shape[0], wl.cin, generator=g, device="cuda")
    target = x @ torch.randn(wl.cin, wl.cin, generator=g, device="cuda") * wl.cin ** -0.5
    context = torch.randn(int(sum(state_lengths)), state_width, generator=g, device="cuda")
    return coords, x.to(dt), context.to(dt), target.to(dt)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--workload", default="b4_r64_spheres_c64_f16", choices=sorted(synth.WORKLOADS))
    ap.add_argument("--heads", type=int, default=4)
    ap.add_argument("--kv-heads", type=int, default=2)
    ap.add_argument("--states", type=int, default=77, help="encoder states of each batch element")
    ap.add_argument("--state-width", type=int, default=128)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32), help="bits of the optimizer's moments")
    ap.add_argument("--lr", type=float, default=3e-3)
    ap.add_argument("--scan", action="store_true", help="add the recurrent part along a Hilbert curve")
    ap.add_argument("--dropout", type=float, default=0.1, help="of the recurrent part")
    a = ap.parse_args(argv)
    wl = synth.WORKLOADS[a.workload]
    lengths = [a.states] * wl.B
    coords, x, context, target = make_inputs(wl, lengths, a.state_width)
    block = VoxelBlock(coords, wl.grid, wl.cin, x.dtype, lengths, a.heads, a.kv_heads, a.state_width, a.bits,
                       scan=a.scan, dropout=a.dropout)
    print(f"{a.workload}: {coords.shape[0]} voxels, {sum(lengths)} states")
    for step in range(1, a.steps + 1):
        loss = block.train_step(x, context, target, step, a.lr)
        print(f"step {step}: loss {float(loss):.5f}")
    block.check()


if __name__ == "__main__":
    main()
