"""Argument checks of the attention-block operators: refused on the host, before any launch (CPU only).

Pointers here are made-up addresses that a refused call never follows.
"""
import ctypes

import pytest
import torch

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def ops():
    from voxel_gemm_gb300 import build, ops
    build.build()
    return ops


def heads(ops, data=4096, row=128, head=64):
    return ops.HeadsStruct(data, row, head)


def rope_fwd(ops, n=10, hq=2, hk=0, d=64, dtype=1, q="ok", qw=4096, coords=4096, freqs=4096, pairs=(10, 10, 10),
             eps=1e-6, flags=0, out="ok"):
    h = heads(ops)
    pick = lambda x: h if isinstance(x, str) else x  # noqa: E731
    pp = None if pairs is None else (ctypes.c_int * 3)(*pairs)
    return ops.lib().vg_qk_norm_rope_fwd(n, hq, hk, d, dtype, pick(q), None, P(qw), None, P(coords), P(freqs), pp, eps,
                                         flags, pick(out), None, None)


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(hq=0, hk=0), 1), (dict(hq=-2, hk=3), 1), (dict(d=0), 1),
    (dict(dtype=3), 1), (dict(d=60), 5), (dict(d=264), 5), (dict(hq=5000), 1), (dict(flags=0x1), 5),
    (dict(q=None), 1), (dict(out=None), 1), (dict(qw=4100), 1), (dict(coords=None), 1), (dict(freqs=None), 1),
    (dict(pairs=None), 1), (dict(pairs=(-1, 2, 3)), 1), (dict(pairs=(11, 11, 11)), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(flags=0x400), 1),                                      # a weight without a norm
    (dict(flags=0x400, qw=None, coords=None, freqs=None), 1),    # nothing to do
])
def test_rope_refusals(ops, change, status):
    assert rope_fwd(ops, **change) == status


def test_rope_strides(ops):
    H = ops.HeadsStruct
    for bad in (H(4104, 128, 64), H(0, 128, 64), H(4096, 32, 64), H(4096, 128, 32), H(4096, 132, 64),
                H(4096, -128, 64), H(4096, 0, 64), H(4096, 128, 68), H(4096, 1 << 60, 64)):
        assert rope_fwd(ops, q=bad) == ops.VG_ERR_INVALID_ARG, (bad.data, bad.row_stride, bad.head_stride)
    # an output whose heads lie on one another's rows
    assert rope_fwd(ops, out=H(4096, 64, 64)) == ops.VG_ERR_INVALID_ARG
    # no rows: nothing is looked at or launched
    assert rope_fwd(ops, n=0, q=None, out=None) == ops.VG_OK


def test_rope_backward_refusals(ops):
    h, L = heads(ops), ops.lib()
    pp = (ctypes.c_int * 3)(10, 10, 10)
    need = L.vg_qk_norm_rope_workspace_bytes(10, 2, 0, 64)
    assert need > 0
    assert L.vg_qk_norm_rope_workspace_bytes(10, 2, 0, 60) == 0
    assert L.vg_qk_norm_rope_workspace_bytes(-1, 2, 0, 64) == 0

    def bwd(flags=0, qw=4096, gy=h, gx=h, gw=4096, gkw=None, ws=4096, nbytes=need):
        return L.vg_qk_norm_rope_bwd(10, 2, 0, 64, 1, h, None, P(qw), None, P(4096), P(4096), pp, 1e-6, flags, gy, None,
                                     gx, None, P(gw), P(gkw), P(ws), nbytes, None)
    assert bwd(nbytes=need - 1) == ops.VG_ERR_WORKSPACE_TOO_SMALL
    assert bwd(ws=None) == bwd(ws=4097) == ops.VG_ERR_INVALID_ARG
    assert bwd(gy=None) == bwd(gx=None) == bwd(gkw=4096) == bwd(gw=4100) == ops.VG_ERR_INVALID_ARG
    assert bwd(flags=ops.VG_QK_NO_NORM, qw=None) == ops.VG_ERR_INVALID_ARG   # a weight gradient without a norm


def attn(ops, **kw):
    d = dict(n_q=100, n_k=50, batch=2, heads_q=4, heads_k=2, head_dim=64, dtype=2, scale=0.125, q_offsets=4096,
             k_offsets=4096, k_lens=None)
    d.update(kw)
    return ops.AttnStruct(*(d[f] for f, _ in ops.AttnStruct._fields_))


@pytest.mark.parametrize("change,status", [
    (dict(n_q=-1), 1), (dict(n_k=1 << 31), 1), (dict(batch=0), 1), (dict(heads_q=0), 1), (dict(heads_k=0), 1),
    (dict(heads_q=3), 1), (dict(head_dim=0), 1), (dict(dtype=9), 1), (dict(head_dim=60), 5), (dict(head_dim=136), 5),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(q_offsets=None), 1), (dict(k_offsets=None), 1), (dict(q_offsets=4098), 1), (dict(k_lens=4098), 1),
])
def test_attn_refusals(ops, change, status):
    L, q, k = ops.lib(), heads(ops, row=256), heads(ops)
    a = attn(ops, **change)
    assert L.vg_cross_attn_fwd(a, q, k, k, q, None, P(4096), 1 << 40, None) == status
    assert L.vg_cross_attn_bwd(a, q, k, k, q, P(4096), q, q, k, k, P(4096), 1 << 40, None) == status
    if "scale" not in change and not {"q_offsets", "k_offsets", "k_lens"} & set(change):
        assert L.vg_cross_attn_workspace_bytes(a, 1) == 0


def test_attn_operands(ops):
    L, H = ops.lib(), ops.HeadsStruct
    q, k, a = heads(ops, row=256), heads(ops), attn(ops)
    need = L.vg_cross_attn_workspace_bytes(a, 1)
    assert need >= L.vg_cross_attn_workspace_bytes(a, 0) > 0

    def fwd(q=q, k=k, v=k, o=q, ws=4096, nbytes=need, lse=4096):
        return L.vg_cross_attn_fwd(a, q, k, v, o, P(lse), P(ws), nbytes, None)

    def bwd(g=q, gq=q, gk=k, gv=k, lse=4096, nbytes=need):
        return L.vg_cross_attn_bwd(a, q, k, k, q, P(lse), g, gq, gk, gv, P(4096), nbytes, None)
    bad = ops.VG_ERR_INVALID_ARG
    for x in (None, H(0, 256, 64), H(4104, 256, 64), H(4096, 260, 64), H(4096, 0, 64), H(4096, 256, 0)):
        assert fwd(q=x) == fwd(o=x) == bad
        assert bwd(g=x) == bwd(gq=x) == bad
    for x in (None, H(4104, 128, 64), H(4096, 132, 64), H(4096, 32, 64)):
        assert fwd(k=x) == fwd(v=x) == bwd(gk=x) == bwd(gv=x) == bad
    assert fwd(o=H(4096, 64, 64)) == bwd(gq=H(4096, 64, 64)) == bwd(gk=H(4096, 64, 64)) == bad   # overlapping rows
    assert fwd(ws=None) == fwd(ws=4097) == fwd(lse=4097) == bwd(lse=None) == bad
    small = L.vg_cross_attn_workspace_bytes(a, 0) - 1
    assert fwd(nbytes=small) == bwd(nbytes=need - 1) == ops.VG_ERR_WORKSPACE_TOO_SMALL
    assert L.vg_cross_attn_status(None, None) == bad
    assert L.vg_cross_attn_workspace_bytes(None, 0) == 0


def test_adamw_refusals(ops):
    T, L = ops.AdamWTensorStruct, ops.lib()
    good = dict(param=4096, grad=4096, master=None, m=4096, v=4096, m_scale=4096, v_scale=4096, n=10,
                weight_decay=0.0, dtype=0)

    def step(count=1, bits=32, step=1, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, gs=1.0, table=True, **kw):
        t = (T * 1)(T(*({**good, **kw}[f] for f, _ in T._fields_)))
        return L.vg_adamw_step(t if table else None, count, bits, step, lr, b1, b2, eps, gs, None)
    nan, inf, bad = float("nan"), float("inf"), ops.VG_ERR_INVALID_ARG
    for kw in (dict(count=-1), dict(table=False), dict(step=0), dict(lr=-1.0), dict(lr=nan), dict(lr=inf),
               dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=nan), dict(eps=-1.0), dict(gs=nan), dict(gs=inf),
               dict(n=-1), dict(dtype=5), dict(weight_decay=-1.0), dict(weight_decay=nan), dict(param=None),
               dict(grad=None), dict(m=None), dict(v=None), dict(param=4097), dict(grad=4098), dict(master=4098),
               dict(m=4098), dict(bits=8, m_scale=None), dict(bits=8, v_scale=4097)):
        assert step(**kw) == bad, kw
    assert step(bits=16) == ops.VG_ERR_UNSUPPORTED
    assert step(count=0) == step(n=0, param=None) == ops.VG_OK       # nothing to do, nothing launched
    d = L.vg_adamw_decode
    assert d(P(1), P(4), -1, 0, P(4), None) == d(P(1), P(4), 1, 2, P(4), None) == bad
    assert d(None, P(4), 1, 0, P(4), None) == d(P(1), P(6), 1, 0, P(4), None) == d(P(1), P(4), 1, 0, P(5), None) == bad
    assert d(None, None, 0, 0, None, None) == ops.VG_OK


def test_binding_checks(ops):
    """Shapes and dtypes that the binding turns down before it reaches the library."""
    q, w = torch.zeros(4, 2, 64), torch.zeros(2, 64)
    c = torch.zeros(4, 4, dtype=torch.int32)
    f, pairs = ops.rope_freqs(64, device="cpu")
    assert pairs == (10, 10, 10) and f.shape == (30,) and f[0] == 1 and f[10] == 1 and f[9] < f[8]

    def call(q=q, w=w, c=c, f=f, o=q):
        ops.vg_qk_norm_rope_fwd(q, None, w, None, c, f, pairs, o, None)
    for kw in (dict(q=None), dict(q=q[0]), dict(w=w[:1]), dict(w=w.half()), dict(c=c.long()), dict(c=c[:3]),
               dict(f=None), dict(f=f[:5]), dict(f=f.double()), dict(o=q.half()), dict(o=q[:3]),
               dict(o=q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError):
        ops.AdamWState([torch.zeros(3)], [torch.zeros(3)])           # not on the GPU
    with pytest.raises(ValueError):
        ops.AdamWState([torch.zeros(3)], [])
    with pytest.raises(ops.VGError):
        ops.AdamWState([], [], bits=16)
    with pytest.raises(ValueError):
        ops.vg_adamw_decode(torch.zeros(300, dtype=torch.uint8), torch.zeros(1), torch.zeros(300), True)
    with pytest.raises(ops.VGError):
        ops.cross_attn_workspace(10, 10, 1, 4, 3, 64, torch.float16, device="cpu")
