"""AdamWState's table and the tensors that it was made of (GPU)."""
import pytest
import torch

from voxel_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


def make():
    g = torch.Generator(device="cuda").manual_seed(1)
    params = [torch.randn(n, generator=g, device="cuda").requires_grad_() for n in (300, 1000)]
    (sum((p * p).sum() for p in params)).backward()
    return params, ops.AdamWState(params, [p.grad for p in params])


def refused(params, st):
    before = [p.detach().clone() for p in params]
    with pytest.raises(ValueError, match="AdamWState"):
        ops.vg_adamw_step(st, 2, 1e-2)
    assert all(torch.equal(a, b) for a, b in zip(before, params)) and not st.m.any()


def test_a_replaced_gradient_is_noticed():
    """zero_grad(set_to_none=True) and a new backward pass give a parameter another gradient tensor: the step would
    go on reading the old one."""
    params, st = make()
    for p in params:
        p.grad = None
    refused(params, st)
    (sum((p ** 4).sum() for p in params)).backward()
    refused(params, st)


@pytest.mark.parametrize("what", ["param", "grad", "master"])
def test_memory_that_moved_is_noticed(what):
    param = torch.randn(500, device="cuda").requires_grad_()
    (param * param).sum().backward()
    x = {"param": param, "grad": param.grad, "master": param.detach().clone()}
    st = ops.AdamWState([param], [param.grad], masters=[x["master"]])
    x[what].data = x[what].detach().clone()
    refused([param], st)


@pytest.mark.parametrize("what", ["param", "grad", "master"])
def test_the_state_keeps_the_memory_that_it_writes(what):
    """Buffers of the caller's own that get other memory: the step goes on with the old, which nothing else gets."""
    x = {n: torch.randn(500_000, device="cuda") for n in ("param", "grad", "master")}
    st = ops.AdamWState([x["param"]], [x["grad"]], masters=[x["master"]])
    x[what].data = torch.empty(0, device="cuda")
    others = [torch.zeros(500_000, device="cuda") for _ in range(8)]
    ops.vg_adamw_step(st, 1, 1e-2)
    assert not any(t.any() for t in others)


def test_gradients_that_stay_are_followed():
    """Gradients accumulated in place, zeroed and filled again are read where they lie; buffers of the caller's own
    have nothing to do with .grad."""
    params, st = make()
    want = [p.detach().clone() for p in params]
    grads = [p.grad.clone() for p in params]
    st2 = ops.AdamWState(want, grads)
    ops.vg_adamw_step(st, 1, 1e-2)
    ops.vg_adamw_step(st2, 1, 1e-2)
    opt = torch.optim.SGD(params, lr=0.0)
    opt.zero_grad(set_to_none=False)
    (sum((p ** 4).sum() for p in params)).backward()
    for p, g in zip(params, grads):
        g.copy_(p.grad)
    ops.vg_adamw_step(st, 2, 1e-2)
    ops.vg_adamw_step(st2, 2, 1e-2)
    assert all(torch.equal(p, w) for p, w in zip(params, want))
    own = torch.zeros(300, device="cuda")
    st3 = ops.AdamWState([params[0]], [own])
    params[0].grad = None
    ops.vg_adamw_step(st3, 1, 1e-2)
