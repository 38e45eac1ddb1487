"""Tensors that are not on the call's GPU are refused before the library sees their addresses (CPU only).

The tensors here lie on the CPU and say that they are on a GPU; in each call one does not, and no call is complete
without it, so none reaches a launch."""
import pytest
import torch

from voxel_gemm_gb300 import ops


class OnGpu(torch.Tensor):
    """A CPU tensor that gives itself out as one on GPU 0 (or `index`)."""
    index = 0

    def get_device(self):
        return self.index

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", self.index)

    __torch_function__ = torch._C._disabled_torch_function_impl


class OnGpu1(OnGpu):
    index = 1


def gpu(t, kind=OnGpu):
    return t.as_subclass(kind)


@pytest.fixture(scope="module", autouse=True)
def built():
    from voxel_gemm_gb300 import build
    build.build()


def refused(call, tensors):
    """call(**tensors) with each of them in turn on the CPU, and on another GPU."""
    for name, t in tensors.items():
        for elsewhere in (t, gpu(t, OnGpu1)):
            moved = {n: gpu(x) for n, x in tensors.items()}
            moved[name] = elsewhere
            with pytest.raises(ValueError, match="GPU"):
                call(**moved)


def test_attention():
    q, k = torch.zeros(4, 2, 64), torch.zeros(6, 2, 64)
    off = torch.tensor([0, 3, 6], dtype=torch.int32)
    common = dict(q=q, k=k, v=k.clone(), q_offsets=off, k_offsets=off.clone(), k_lens=torch.ones(2, dtype=torch.int32),
                  out=q.clone(), lse=torch.zeros(2, 4), ws=torch.zeros(4096, dtype=torch.uint8))
    refused(ops.vg_cross_attn_fwd, common)
    refused(ops.vg_cross_attn_bwd, dict(common, grad_out=q.clone(), grad_q=q.clone(), grad_k=k.clone(),
                                        grad_v=k.clone()))


@pytest.mark.parametrize("shared", [False, True])
def test_norm_and_rotation(shared):
    q, k = torch.zeros(4, 2, 64), torch.zeros(4, 1, 64)
    qw, kw = (torch.zeros(64), torch.zeros(64)) if shared else (torch.zeros(2, 64), torch.zeros(1, 64))
    freqs, pairs = ops.rope_freqs(64, device="cpu")
    common = dict(q=q, k=k, q_weight=qw, k_weight=kw, coords=torch.zeros(4, 4, dtype=torch.int32), freqs=freqs)
    refused(lambda **t: ops.vg_qk_norm_rope_fwd(axis_pairs=pairs, **t), dict(common, q_out=q.clone(), k_out=k.clone()))
    refused(lambda **t: ops.vg_qk_norm_rope_bwd(axis_pairs=pairs, **t), dict(
        common, grad_q_out=q.clone(), grad_k_out=k.clone(), grad_q=q.clone(), grad_k=k.clone(),
        grad_q_weight=qw.clone(), grad_k_weight=kw.clone(), ws=torch.zeros(4096, dtype=torch.uint8)))


def test_decoded_moments():
    refused(lambda **t: ops.vg_adamw_decode(second=False, **t),
            dict(codes=torch.zeros(300, dtype=torch.uint8), scales=torch.zeros(2), out=torch.zeros(300)))


def test_parameters_on_two_gpus():
    """One state is one table and one launch: parameters of two GPUs cannot share it."""
    a, b = torch.zeros(300), torch.zeros(5)
    for kinds in ((OnGpu, OnGpu1), (OnGpu1, OnGpu)):
        p = [gpu(t, kind) for t, kind in zip((a, b), kinds)]
        with pytest.raises(ValueError, match="one GPU"):
            ops.AdamWState(p, [gpu(t.clone(), kind) for t, kind in zip((a, b), kinds)])
