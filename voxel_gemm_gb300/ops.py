"""Thin ctypes binding of include/vg.h: argument marshalling only.

Each ``vg_*`` function has the C name and takes torch CUDA tensors (device
memory comes from torch; the library allocates nothing).  Status codes other
than VG_OK raise ``VGError``.  All computation happens inside
``libvoxelgemm.so``; if that library is missing the first call raises, there
is no fallback.

The small ``NbrMap`` / ``ConvWorkspace`` helpers only allocate the caller-owned
buffers with torch and keep the pointers together.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass

import torch

VG_OK, VG_ERR_INVALID_ARG, VG_ERR_COORD_OUT_OF_RANGE, VG_ERR_DUPLICATE_COORD = 0, 1, 2, 3
VG_ERR_HASH_FULL, VG_ERR_UNSUPPORTED, VG_ERR_WORKSPACE_TOO_SMALL, VG_ERR_CUDA = 4, 5, 6, 7
VG_ERR_DEVICE_TIMEOUT = 8
VG_F32, VG_F16, VG_BF16 = 0, 1, 2
VG_KEY32, VG_KEY64, VG_ORDER_HILBERT, VG_MAP_HASH, VG_MAP_COLUMNS = 0x1, 0x2, 0x4, 0x8, 0x40
VG_TEST_SMALL_HASH = 0x100
VG_CURVE_ZORDER, VG_CURVE_HILBERT = 0, 1
VG_ALLOW_TF32, VG_NO_SMALL_N_SPLIT = 0x10, 0x20
VG_NONE = 0xFFFFFFFF
VG_TILE_ROWS = 128
VG_ROPE_HALVES, VG_QK_NO_NORM, VG_QK_SHARED_WEIGHT = 0x200, 0x400, 0x800
VG_ADAMW_BLOCK = 256
VG_SCAN_REVERSE, VG_SCAN_FREE_INPUT, VG_SCAN_CARRY_ROWS = 0x1000, 0x2000, 16

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libvoxelgemm.so")
_lock = threading.Lock()
_lib = None

_DT = {torch.float32: VG_F32, torch.float16: VG_F16, torch.bfloat16: VG_BF16}


class SparseMapStruct(ctypes.Structure):
    """Mirror of vg_sparse_map (include/vg.h)."""
    _fields_ = [("n_in", ctypes.c_int64), ("n_out", ctypes.c_int64), ("kernel", ctypes.c_int),
                ("stride", ctypes.c_int), ("taps", ctypes.c_int), ("out_grid", ctypes.c_int * 4),
                ("side_in", ctypes.c_void_p), ("side_out", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("down_mask", ctypes.c_void_p), ("up", ctypes.c_void_p), ("up_mask", ctypes.c_void_p),
                ("coords_out", ctypes.c_void_p)]


class HeadsStruct(ctypes.Structure):
    """Mirror of vg_heads (include/vg.h)."""
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class AttnStruct(ctypes.Structure):
    """Mirror of vg_attn (include/vg.h)."""
    _fields_ = [("n_q", ctypes.c_int64), ("n_k", ctypes.c_int64), ("batch", ctypes.c_int), ("heads_q", ctypes.c_int),
                ("heads_k", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float), ("q_offsets", ctypes.c_void_p), ("k_offsets", ctypes.c_void_p),
                ("k_lens", ctypes.c_void_p)]


class AdamWTensorStruct(ctypes.Structure):
    """Mirror of vg_adamw_tensor (include/vg.h)."""
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("weight_decay", ctypes.c_double),
                ("dtype", ctypes.c_int)]


class RowsStruct(ctypes.Structure):
    """Mirror of vg_rows (include/vg.h)."""
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64)]


class ScanStruct(ctypes.Structure):
    """Mirror of vg_scan (include/vg.h)."""
    _fields_ = [("n", ctypes.c_int64), ("channels", ctypes.c_int), ("batch", ctypes.c_int), ("dtype", ctypes.c_int),
                ("flags", ctypes.c_uint), ("offsets", ctypes.c_void_p), ("order", ctypes.c_void_p)]


class VGError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {vg_strerror(status)} (status {status})")
        self.status = status


def lib():
    """The loaded libvoxelgemm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m voxel_gemm_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64, U, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint, ctypes.c_size_t
        D, H = ctypes.c_double, ctypes.POINTER(HeadsStruct)
        R, SC = ctypes.POINTER(RowsStruct), ctypes.POINTER(ScanStruct)
        sig = {
            "vg_strerror": ([I], ctypes.c_char_p),
            "vg_version": ([], I),
            "vg_nbrmap_workspace_bytes": ([I64, I, I, I, I, U], SZ),
            "vg_nbrmap_build": ([P, I64, I, I, I, I, U, P, SZ, P, P, P], I),
            "vg_nbrmap_status": ([P, P], I),
            "vg_nbrmap_sorted_idx": ([P], P),
            "vg_nbrmap_tile_mask": ([P, I64], P),
            "vg_nbrmap_sorted_nbr": ([P, I64], P),
            "vg_conv_workspace_bytes": ([I64, I, I, I, U], SZ),
            "vg_subm_conv3d_fwd": ([P, P, P, I64, I, P, P, P, P, I, I, U, P, SZ, P], I),
            "vg_subm_conv3d_bwd": ([P, P, P, I64, I, P, P, P, P, P, P, I, I, U, P, SZ, P], I),
            "vg_conv_status": ([P, P], I),
            "vg_nbrmap_describe": ([I64, I, I, I, I, U, I, ctypes.POINTER(ctypes.c_int)], I),
            "vg_conv_describe": ([I64, I, I, I, U, I, ctypes.POINTER(ctypes.c_int)], I),
            "vg_subm_conv3d_fwd_noalloc": ([P, P, P, I64, I, P, P, P, P, I, I, U, P], I),
            "vg_subm_conv3d_fwd_noalloc_status": ([P], I),
            "vg_sum_ordered": ([P, I, I64, I, P, P], I),
            "vg_encode_seq": ([P, I64, I, I, P, P], I),
            "vg_sparse_map_workspace_bytes": ([I64, I, I, I, I, I, I, U], SZ),
            "vg_sparse_map_build": ([P, I64, I, I, I, I, I, I, U, P, SZ, ctypes.POINTER(SparseMapStruct), P], I),
            "vg_sparse_conv_workspace_bytes": ([ctypes.POINTER(SparseMapStruct), I, I, I, I, U], SZ),
            "vg_sparse_conv3d_fwd": ([ctypes.POINTER(SparseMapStruct), I, I, P, P, P, P, I, I, U, P, SZ, P], I),
            "vg_sparse_conv3d_bwd": ([ctypes.POINTER(SparseMapStruct), I, I, P, P, P, P, P, P, I, I, U, P, SZ, P],
                                     I),
            "vg_decode_seq": ([P, I64, I, I, P, P], I),
            "vg_qk_norm_rope_fwd": ([I64, I, I, I, I, H, H, P, P, P, P, ctypes.POINTER(I), D, U, H, H, P], I),
            "vg_qk_norm_rope_workspace_bytes": ([I64, I, I, I], SZ),
            "vg_qk_norm_rope_bwd": ([I64, I, I, I, I, H, H, P, P, P, P, ctypes.POINTER(I), D, U, H, H, H, H, P, P, P,
                                     SZ, P], I),
            "vg_cross_attn_workspace_bytes": ([ctypes.POINTER(AttnStruct), I], SZ),
            "vg_cross_attn_fwd": ([ctypes.POINTER(AttnStruct), H, H, H, H, P, P, SZ, P], I),
            "vg_cross_attn_bwd": ([ctypes.POINTER(AttnStruct), H, H, H, H, P, H, H, H, H, P, SZ, P], I),
            "vg_cross_attn_status": ([P, P], I),
            "vg_adamw_step": ([ctypes.POINTER(AdamWTensorStruct), I, I, I64, D, D, D, D, D, P], I),
            "vg_adamw_decode": ([P, P, I64, I, P, P], I),
            "vg_layer_norm_fwd": ([I64, I, I, R, P, P, D, R, P, P], I),
            "vg_layer_norm_workspace_bytes": ([I64, I], SZ),
            "vg_layer_norm_bwd": ([I64, I, I, R, P, P, R, R, R, P, P, P, SZ, P], I),
            "vg_gated_scan_workspace_bytes": ([SC], SZ),
            "vg_gated_scan_carry_rows": ([I64], I64),
            "vg_gated_scan_fwd": ([SC, R, R, P, R, P, P, P, SZ, P], I),
            "vg_gated_scan_bwd": ([SC, R, R, P, P, R, P, R, R, P, P, SZ, P], I),
            "vg_gated_scan_step": ([I64, I, I, U, R, R, P, R, P], I),
            "vg_gated_scan_status": ([P, P], I),
            "vg_dropout_add_fwd": ([I64, I, P, P, D, P, ctypes.c_uint32, P, P], I),
            "vg_dropout_add_bwd": ([I64, I, P, D, P, ctypes.c_uint32, P, P], I),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
        return L


def _p(t):
    return None if t is None else t.data_ptr()


def _s(stream):
    if stream is not None:
        return stream.cuda_stream
    if torch.cuda.is_initialized():  # the current stream's handle without an object around it: 0.3 us instead of 3
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


def _check(st: int, where: str):
    if st != VG_OK:
        raise VGError(st, where)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def vg_strerror(status: int) -> str:
    return lib().vg_strerror(int(status)).decode()


def vg_version() -> int:
    return lib().vg_version()


def vg_nbrmap_workspace_bytes(N: int, B: int, X: int, Y: int, Z: int, flags: int = 0) -> int:
    return int(lib().vg_nbrmap_workspace_bytes(N, B, X, Y, Z, flags))


def vg_nbrmap_build(coords, B, X, Y, Z, flags, ws, nbr, mask, stream=None) -> None:
    N = coords.shape[0]
    _check(lib().vg_nbrmap_build(_p(coords), N, B, X, Y, Z, flags, _p(ws), ws.numel() * ws.element_size(),
                                 _p(nbr), _p(mask), _s(stream)), "vg_nbrmap_build")


def vg_nbrmap_status(ws, stream=None) -> int:
    return lib().vg_nbrmap_status(_p(ws), _s(stream))


def vg_nbrmap_sorted_idx(ws, N: int) -> torch.Tensor:
    """View of the workspace's sorted_idx [N] (int32 storage of uint32 values)."""
    off = lib().vg_nbrmap_sorted_idx(_p(ws)) - ws.data_ptr()
    return ws.view(torch.uint8)[off: off + 4 * N].view(torch.int32)


def vg_nbrmap_tile_mask(ws, N: int) -> torch.Tensor:
    """View of the workspace's per-tile masks [ceil(N/128)] (int32 storage of uint32 values)."""
    off = lib().vg_nbrmap_tile_mask(_p(ws), N) - ws.data_ptr()
    T = (N + VG_TILE_ROWS - 1) // VG_TILE_ROWS
    return ws.view(torch.uint8)[off: off + 4 * T].view(torch.int32)


def vg_nbrmap_sorted_nbr(ws, N: int) -> torch.Tensor:
    """View of the workspace's neighbour lists in processing order [ceil(N/128)*128, 27]."""
    off = lib().vg_nbrmap_sorted_nbr(_p(ws), N) - ws.data_ptr()
    R = (N + VG_TILE_ROWS - 1) // VG_TILE_ROWS * VG_TILE_ROWS
    return ws.view(torch.uint8)[off: off + 4 * 27 * R].view(torch.int32).view(R, 27)


def vg_conv_workspace_bytes(N: int, Cin: int, Cout: int, dtype, flags: int = 0) -> int:
    code = dtype if isinstance(dtype, int) else _DT[dtype]
    return int(lib().vg_conv_workspace_bytes(N, Cin, Cout, code, flags))


def vg_subm_conv3d_fwd(nbr_ws, nbr, mask, feats, weight, bias, out, conv_ws, flags=0, stream=None) -> None:
    N, Cin = feats.shape
    Cout = weight.shape[2]
    _check(lib().vg_subm_conv3d_fwd(_p(nbr_ws), _p(nbr), _p(mask), N, _dtype_code(feats), _p(feats),
                                    _p(weight), _p(bias), _p(out), Cin, Cout, flags, _p(conv_ws),
                                    conv_ws.numel() * conv_ws.element_size(), _s(stream)),
           "vg_subm_conv3d_fwd")


def vg_subm_conv3d_fwd_noalloc(nbr_ws, nbr, mask, feats, weight, bias, out, flags=0, stream=None) -> None:
    """Forward without a workspace argument (scratch is a fixed array inside the library)."""
    N, Cin = feats.shape
    Cout = weight.shape[2]
    _check(lib().vg_subm_conv3d_fwd_noalloc(_p(nbr_ws), _p(nbr), _p(mask), N, _dtype_code(feats), _p(feats),
                                            _p(weight), _p(bias), _p(out), Cin, Cout, flags, _s(stream)),
           "vg_subm_conv3d_fwd_noalloc")


def vg_subm_conv3d_fwd_noalloc_status(stream=None) -> int:
    """Device-side status of the last no-allocation forward on the current device (syncs `stream`)."""
    return lib().vg_subm_conv3d_fwd_noalloc_status(_s(stream))


def vg_subm_conv3d_bwd(nbr_ws, nbr, mask, grad_out, feats, weight, grad_feats, grad_weight, grad_bias,
                       conv_ws, flags=0, stream=None) -> None:
    N, Cout = grad_out.shape
    Cin = weight.shape[1]
    _check(lib().vg_subm_conv3d_bwd(_p(nbr_ws), _p(nbr), _p(mask), N, _dtype_code(grad_out), _p(grad_out),
                                    _p(feats), _p(weight), _p(grad_feats), _p(grad_weight), _p(grad_bias),
                                    Cin, Cout, flags, _p(conv_ws), conv_ws.numel() * conv_ws.element_size(),
                                    _s(stream)),
           "vg_subm_conv3d_bwd")


def vg_nbrmap_describe(N, B, X, Y, Z, flags=0, sm_count=0) -> dict:
    info = (ctypes.c_int * 4)()
    _check(lib().vg_nbrmap_describe(N, B, X, Y, Z, flags, sm_count, info), "vg_nbrmap_describe")
    return {"key64": 1 if info[0] == 1 else 0, "index": "columns" if info[0] == 2 else "hash",
            "sort_bits": info[1], "sort_passes": info[2], "launches": info[3]}


def vg_conv_describe(N, Cin, Cout, dtype, flags=0, sm_count=0) -> dict:
    code = dtype if isinstance(dtype, int) else _DT[dtype]
    info = (ctypes.c_int * 4)()
    _check(lib().vg_conv_describe(N, Cin, Cout, code, flags, sm_count, info), "vg_conv_describe")
    return {"tensor_core": info[0], "splits": info[1], "launches_fwd": info[2], "launches_bwd": info[3]}


def vg_sum_ordered(parts, out, stream=None) -> None:
    """out = parts[0] + parts[1] + ... (fp32 adds in index order, one rounding); parts [n, *out.shape]."""
    if parts.dtype != out.dtype or parts.shape[1:] != out.shape or not parts.is_contiguous() \
            or not out.is_contiguous():
        raise ValueError("vg_sum_ordered: parts must be [n, *out.shape], contiguous, of out's dtype")
    _check(lib().vg_sum_ordered(_p(parts), parts.shape[0], out.numel(), _dtype_code(out), _p(out), _s(stream)),
           "vg_sum_ordered")


def vg_encode_seq(coords, bits: int, mode: int, codes, stream=None) -> None:
    """codes[i] (int64 storage of uint64) = (b << 3*bits) | curve(x, y, z) of coords[i]."""
    _check(lib().vg_encode_seq(_p(coords), coords.shape[0], bits, mode, _p(codes), _s(stream)), "vg_encode_seq")


def vg_decode_seq(codes, bits: int, mode: int, coords, stream=None) -> None:
    """coords[i] = (b, x, y, z) of codes[i] (the inverse of vg_encode_seq)."""
    _check(lib().vg_decode_seq(_p(codes), codes.shape[0], bits, mode, _p(coords), _s(stream)), "vg_decode_seq")


def vg_conv_status(conv_ws, stream=None) -> int:
    return lib().vg_conv_status(_p(conv_ws), _s(stream))


# ---------------------------------------------------------------- buffer helpers
@dataclass
class NbrMap:
    """Caller-owned buffers of one neighbour map (allocated with torch)."""
    N: int
    grid: tuple
    flags: int
    ws: torch.Tensor     # uint8 workspace (the neighbour cache)
    nbr: torch.Tensor    # int32 [N,27] storage of uint32 entries
    mask: torch.Tensor   # int32 [N] storage of uint32 bitmasks

    @staticmethod
    def alloc(N, grid, flags=0, device="cuda") -> "NbrMap":
        B, X, Y, Z = grid
        nb = vg_nbrmap_workspace_bytes(N, B, X, Y, Z, flags)
        if nb == 0:
            raise VGError(VG_ERR_INVALID_ARG, "vg_nbrmap_workspace_bytes")
        ws = torch.empty(nb, dtype=torch.uint8, device=device)
        nbr = torch.empty(N, 27, dtype=torch.int32, device=device)
        mask = torch.empty(N, dtype=torch.int32, device=device)
        return NbrMap(N, tuple(grid), flags, ws, nbr, mask)

    def build(self, coords, stream=None) -> "NbrMap":
        vg_nbrmap_build(coords, *self.grid, self.flags, self.ws, self.nbr, self.mask, stream)
        return self

    def status(self, stream=None) -> int:
        return vg_nbrmap_status(self.ws, stream)

    def sorted_idx(self) -> torch.Tensor:
        return vg_nbrmap_sorted_idx(self.ws, self.N)

    def tile_mask(self) -> torch.Tensor:
        return vg_nbrmap_tile_mask(self.ws, self.N)

    def sorted_nbr(self) -> torch.Tensor:
        return vg_nbrmap_sorted_nbr(self.ws, self.N)


def conv_workspace(N, Cin, Cout, dtype, device="cuda", flags=0) -> torch.Tensor:
    nb = vg_conv_workspace_bytes(N, Cin, Cout, dtype, flags)
    if nb == 0:
        raise VGError(VG_ERR_UNSUPPORTED, "vg_conv_workspace_bytes")
    return torch.zeros(nb, dtype=torch.uint8, device=device)  # zero error record before any call


# ---------------------------------------------------------------- regular (strided / transposed) conv
class SparseMap:
    """A regular-convolution map (input sites -> strided output sites) in a torch-owned workspace."""

    def __init__(self, coords, grid, kernel: int, stride: int, flags: int = 0, stream=None):
        B, X, Y, Z = grid
        N = coords.shape[0]
        nb = int(lib().vg_sparse_map_workspace_bytes(N, B, X, Y, Z, kernel, stride, flags))
        if nb == 0:
            raise VGError(VG_ERR_INVALID_ARG, "vg_sparse_map_workspace_bytes")
        self.ws = torch.empty(nb, dtype=torch.uint8, device=coords.device)
        self.coords = coords
        self.m = SparseMapStruct()
        _check(lib().vg_sparse_map_build(_p(coords), N, B, X, Y, Z, kernel, stride, flags, _p(self.ws), nb,
                                         ctypes.byref(self.m), _s(stream)), "vg_sparse_map_build")

    @property
    def n_in(self) -> int:
        return self.m.n_in

    @property
    def n_out(self) -> int:
        return self.m.n_out

    @property
    def taps(self) -> int:
        return self.m.taps

    def _view(self, ptr, nbytes, dtype, shape):
        off = ptr - self.ws.data_ptr()
        return self.ws.view(torch.uint8)[off: off + nbytes].view(dtype).view(*shape)

    def coords_out(self) -> torch.Tensor:
        return self._view(self.m.coords_out, 16 * self.n_out, torch.int32, (self.n_out, 4))

    def down(self) -> torch.Tensor:
        return self._view(self.m.down, 4 * 27 * self.n_out, torch.int32, (self.n_out, 27))

    def up(self) -> torch.Tensor:
        return self._view(self.m.up, 4 * 27 * self.n_in, torch.int32, (self.n_in, 27))

    def workspace(self, transposed, Cin, Cout, dtype, flags=0) -> torch.Tensor:
        code = dtype if isinstance(dtype, int) else _DT[dtype]
        nb = int(lib().vg_sparse_conv_workspace_bytes(ctypes.byref(self.m), int(transposed), Cin, Cout, code, flags))
        if nb == 0:
            raise VGError(VG_ERR_UNSUPPORTED, "vg_sparse_conv_workspace_bytes")
        return torch.zeros(nb, dtype=torch.uint8, device=self.ws.device)

    def fwd(self, transposed, feats, weight, bias, out, conv_ws, flags=0, stream=None) -> None:
        Cin, Cout = weight.shape[1], weight.shape[2]
        _check(lib().vg_sparse_conv3d_fwd(ctypes.byref(self.m), int(transposed), _dtype_code(weight), _p(feats),
                                          _p(weight), _p(bias), _p(out), Cin, Cout, flags, _p(conv_ws),
                                          conv_ws.numel(), _s(stream)), "vg_sparse_conv3d_fwd")

    def bwd(self, transposed, grad_out, feats, weight, grad_feats, grad_weight, grad_bias, conv_ws, flags=0,
            stream=None) -> None:
        Cin, Cout = weight.shape[1], weight.shape[2]
        _check(lib().vg_sparse_conv3d_bwd(ctypes.byref(self.m), int(transposed), _dtype_code(weight), _p(grad_out),
                                          _p(feats), _p(weight), _p(grad_feats), _p(grad_weight), _p(grad_bias),
                                          Cin, Cout, flags, _p(conv_ws), conv_ws.numel(), _s(stream)),
               "vg_sparse_conv3d_bwd")


# ---------------------------------------------------------------- attention-block operators
_Int3 = ctypes.c_int * 3


def _on(device, what, *tensors):
    """Refuse tensors that are not on the GPU of index `device`: kernels take raw addresses and would follow them."""
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"{what}: every tensor must be on the GPU, and on one GPU; got one on {t.device}")


def _gpu(t, what):
    """Index of t's GPU."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{what}: every tensor must be on the GPU; got one on {t.device}")
    return device


def _heads(t, dtype, shape, device, what):
    """vg_heads of a [rows, heads, head_dim] tensor (any row and head strides), None for None."""
    if t is None:
        return None
    s = t.stride()
    if t.dtype != dtype or t.shape != shape or (s[2] != 1 and t.numel() > 0):
        raise ValueError(f"{what}: expected {dtype} {list(shape)} with contiguous elements, got {t.dtype} "
                         f"{list(t.shape)} of strides {s}")
    if t.get_device() != device:
        _on(device, what, t)
    return HeadsStruct(t.data_ptr(), s[0], s[1])


def rope_freqs(head_dim: int, axes: int = 3, theta: float = 10000.0, device="cuda"):
    """(freqs, axis_pairs): theta^(-i / pairs) for each of `axes` axes, head_dim // (2 axes) pairs apiece."""
    pairs = head_dim // (2 * axes)
    one = theta ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))
    return one.repeat(axes).to(device, torch.float32), tuple(pairs if a < axes else 0 for a in range(3))


def _rope_shapes(q, k, coords, freqs, axis_pairs, q_weight, k_weight, flags):
    """(N, heads_q, heads_k, head_dim, dtype, pairs, device) of a call, checked."""
    x = q if q is not None else k
    if x is None or x.dim() != 3:
        raise ValueError("q and k are [rows, heads, head_dim]; one of them may be None")
    n, d = x.shape[0], x.shape[2]
    hq, hk = (0 if t is None else t.shape[1] for t in (q, k))
    device = _gpu(x, "q and k")
    if (coords is None) != (freqs is None):
        raise ValueError("coords and freqs come together")
    pairs = None
    if coords is not None:
        if coords.dtype != torch.int32 or coords.shape != (n, 4) or not coords.is_contiguous():
            raise ValueError("coords must be contiguous int32 [rows, 4]")
        if freqs.dtype != torch.float32 or not freqs.is_contiguous() or freqs.numel() != sum(axis_pairs):
            raise ValueError("freqs must be contiguous float32 of sum(axis_pairs) elements")
        _on(device, "coords and freqs", coords, freqs)
        pairs = _Int3(*axis_pairs)
    for w, h, name in ((q_weight, hq, "q_weight"), (k_weight, hk, "k_weight")):
        if w is not None:
            want = (d,) if flags & VG_QK_SHARED_WEIGHT else (h, d)
            if w.dtype != x.dtype or w.shape != want or not w.is_contiguous():
                raise ValueError(f"{name} must be contiguous {x.dtype} {list(want)}")
            _on(device, name, w)
    return n, hq, hk, d, x.dtype, pairs, device


def _rope_flags(q_weight, k_weight, flags):
    """A one-dimensional weight is shared by the heads."""
    if (q_weight is not None and q_weight.dim() == 1) or (k_weight is not None and k_weight.dim() == 1):
        return flags | VG_QK_SHARED_WEIGHT
    return flags


def vg_qk_norm_rope_fwd(q, k, q_weight, k_weight, coords, freqs, axis_pairs, q_out, k_out, eps=1e-6, flags=0,
                        stream=None) -> None:
    """Norm of each head's queries and keys ([rows, heads, head_dim]; either may be None) and their rotation by
    coords [rows, 4]; weights [heads, head_dim], or [head_dim] for all heads, or None for ones."""
    flags = _rope_flags(q_weight, k_weight, flags)
    n, hq, hk, d, dt, pairs, dev = _rope_shapes(q, k, coords, freqs, axis_pairs, q_weight, k_weight, flags)
    sq, sk = (n, hq, d), (n, hk, d)
    _check(lib().vg_qk_norm_rope_fwd(n, hq, hk, d, _DT.get(dt, -1), _heads(q, dt, sq, dev, "q"),
                                     _heads(k, dt, sk, dev, "k"), _p(q_weight), _p(k_weight), _p(coords), _p(freqs),
                                     pairs, eps, flags, _heads(q_out, dt, sq, dev, "q_out"),
                                     _heads(k_out, dt, sk, dev, "k_out"), _s(stream)), "vg_qk_norm_rope_fwd")


def vg_qk_norm_rope_bwd(q, k, q_weight, k_weight, coords, freqs, axis_pairs, grad_q_out, grad_k_out, grad_q, grad_k,
                        grad_q_weight, grad_k_weight, ws, eps=1e-6, flags=0, stream=None) -> None:
    """Gradients of vg_qk_norm_rope_fwd's inputs and weights (weight gradients None: not wanted; ws then None too)."""
    flags = _rope_flags(q_weight if q_weight is not None else grad_q_weight,
                        k_weight if k_weight is not None else grad_k_weight, flags)
    n, hq, hk, d, dt, pairs, dev = _rope_shapes(q, k, coords, freqs, axis_pairs, q_weight, k_weight, flags)
    _rope_shapes(q, k, coords, freqs, axis_pairs, grad_q_weight, grad_k_weight, flags)
    _on(dev, "ws", ws)
    sq, sk = (n, hq, d), (n, hk, d)
    _check(lib().vg_qk_norm_rope_bwd(n, hq, hk, d, _DT.get(dt, -1), _heads(q, dt, sq, dev, "q"),
                                     _heads(k, dt, sk, dev, "k"), _p(q_weight), _p(k_weight), _p(coords), _p(freqs),
                                     pairs, eps, flags, _heads(grad_q_out, dt, sq, dev, "grad_q_out"),
                                     _heads(grad_k_out, dt, sk, dev, "grad_k_out"),
                                     _heads(grad_q, dt, sq, dev, "grad_q"), _heads(grad_k, dt, sk, dev, "grad_k"),
                                     _p(grad_q_weight), _p(grad_k_weight), _p(ws),
                                     0 if ws is None else ws.numel() * ws.element_size(), _s(stream)),
           "vg_qk_norm_rope_bwd")


def qk_norm_rope_workspace(n, heads_q, heads_k, head_dim, device="cuda") -> torch.Tensor:
    nb = int(lib().vg_qk_norm_rope_workspace_bytes(n, heads_q, heads_k, head_dim))
    if nb == 0:
        raise VGError(VG_ERR_INVALID_ARG, "vg_qk_norm_rope_workspace_bytes")
    return torch.empty(nb, dtype=torch.uint8, device=device)


def cross_attn_workspace(n_q, n_k, batch, heads_q, heads_k, head_dim, dtype, backward=False,
                         device="cuda") -> torch.Tensor:
    """Workspace of vg_cross_attn_fwd (and, with backward, of vg_cross_attn_bwd), its error record zero."""
    a = AttnStruct(n_q, n_k, batch, heads_q, heads_k, head_dim, _DT.get(dtype, -1), 1.0, None, None, None)
    nb = int(lib().vg_cross_attn_workspace_bytes(ctypes.byref(a), int(backward)))
    if nb == 0:
        raise VGError(VG_ERR_INVALID_ARG, "vg_cross_attn_workspace_bytes")
    ws = torch.empty(nb, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def _attn(q, k, q_offsets, k_offsets, k_lens, lse, ws, scale, what):
    """The call's vg_attn and its GPU's index, checked."""
    qs, ks = q.shape, k.shape
    if len(qs) != 3 or len(ks) != 3 or qs[2] != ks[2]:
        raise ValueError(f"{what}: q and k are [rows, heads, head_dim] of one head_dim")
    n_q, hq, d = qs
    device = _gpu(q, what)
    batch = q_offsets.numel() - 1
    for t, n, name in ((q_offsets, batch + 1, "q_offsets"), (k_offsets, batch + 1, "k_offsets"),
                       (k_lens, batch, "k_lens")):
        if t is not None and (t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous() or
                              t.get_device() != device):
            raise ValueError(f"{what}: {name} must be contiguous int32 [{n}] on q's GPU")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (hq, n_q) or not lse.is_contiguous()):
        raise ValueError(f"{what}: lse must be contiguous float32 [heads_q, n_q]")
    _on(device, what, lse, ws)
    return AttnStruct(n_q, ks[0], batch, hq, ks[1], d, _DT.get(q.dtype, -1),
                      d ** -0.5 if scale is None else scale, q_offsets.data_ptr(), k_offsets.data_ptr(),
                      None if k_lens is None else k_lens.data_ptr()), device


def vg_cross_attn_fwd(q, k, v, q_offsets, k_offsets, k_lens, out, lse, ws, scale=None, stream=None) -> None:
    """out = softmax(scale q k^T) v of each sample's queries over its first k_lens keys (None: all of them).

    q, out [n_q, heads_q, head_dim]; k, v [n_k, heads_k, head_dim] (any row and head strides); offsets int32
    [batch + 1]; lse float32 [heads_q, n_q] or None; scale head_dim ** -0.5 by default."""
    a, dev = _attn(q, k, q_offsets, k_offsets, k_lens, lse, ws, scale, "vg_cross_attn_fwd")
    sq, sk = (a.n_q, a.heads_q, a.head_dim), (a.n_k, a.heads_k, a.head_dim)
    _check(lib().vg_cross_attn_fwd(a, _heads(q, q.dtype, sq, dev, "q"), _heads(k, q.dtype, sk, dev, "k"),
                                   _heads(v, q.dtype, sk, dev, "v"), _heads(out, q.dtype, sq, dev, "out"), _p(lse),
                                   _p(ws), ws.numel() * ws.element_size(), _s(stream)), "vg_cross_attn_fwd")


def vg_cross_attn_bwd(q, k, v, q_offsets, k_offsets, k_lens, out, lse, grad_out, grad_q, grad_k, grad_v, ws,
                      scale=None, stream=None) -> None:
    """Gradients of vg_cross_attn_fwd's q, k and v, from its out and lse."""
    a, dev = _attn(q, k, q_offsets, k_offsets, k_lens, lse, ws, scale, "vg_cross_attn_bwd")
    dt, sq, sk = q.dtype, (a.n_q, a.heads_q, a.head_dim), (a.n_k, a.heads_k, a.head_dim)
    _check(lib().vg_cross_attn_bwd(a, _heads(q, dt, sq, dev, "q"), _heads(k, dt, sk, dev, "k"),
                                   _heads(v, dt, sk, dev, "v"), _heads(out, dt, sq, dev, "out"), _p(lse),
                                   _heads(grad_out, dt, sq, dev, "grad_out"), _heads(grad_q, dt, sq, dev, "grad_q"),
                                   _heads(grad_k, dt, sk, dev, "grad_k"), _heads(grad_v, dt, sk, dev, "grad_v"),
                                   _p(ws), ws.numel() * ws.element_size(), _s(stream)), "vg_cross_attn_bwd")


def vg_cross_attn_status(ws, stream=None) -> int:
    return lib().vg_cross_attn_status(_p(ws), _s(stream))


class AdamWState:
    """Moments of many parameters and the table that vg_adamw_step takes.

    params and grads are lists of contiguous tensors of one dtype each, written and read at every step where they lay
    when the state was made (it keeps that memory).  Where a parameter's own .grad was given, a step is refused once
    it has another one (zero_grad(set_to_none=False) keeps it) or its tensors have moved.  masters is a list of fp32
    tensors or None; weight_decay, a number or a list.  The moments lie in two arenas m and v, each tensor's at the
    next multiple of 256 elements (`offsets`), as fp32 or, with bits = 8, as uint8 codes beside m_scale and v_scale.
    Arenas that are not given start at zero."""

    def __init__(self, params, grads, masters=None, bits=32, weight_decay=0.0, m=None, v=None, m_scale=None,
                 v_scale=None):
        if len(params) != len(grads) or (masters is not None and len(masters) != len(params)):
            raise ValueError("AdamWState: params, grads and masters must be as many")
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * len(params)
        if len(decay) != len(params):
            raise ValueError("AdamWState: weight_decay must be a number or one per parameter")
        if bits not in (8, 32):
            raise VGError(VG_ERR_UNSUPPORTED, "AdamWState")
        self.bits, self.offsets, total = bits, [], 0
        device = params[0].device if params else torch.device("cuda", torch.cuda.current_device())
        for p, g in zip(params, grads):
            if p.device != device:
                raise ValueError("AdamWState: params must be on one GPU (its step is one launch): one state for each")
            if p.dtype not in _DT or g.dtype != p.dtype or g.shape != p.shape or not p.is_contiguous() \
                    or not g.is_contiguous() or not p.is_cuda or g.device != p.device:
                raise ValueError("AdamWState: params and grads must be contiguous CUDA tensors of one shape and dtype")
            self.offsets.append(total)
            total += -(-p.numel() // VG_ADAMW_BLOCK) * VG_ADAMW_BLOCK
        for p, x in zip(params, masters or []):
            if x.dtype != torch.float32 or x.shape != p.shape or not x.is_contiguous() or x.device != p.device:
                raise ValueError("AdamWState: masters must be contiguous float32 of their parameter's shape")
        code, blocks = torch.uint8 if bits == 8 else torch.float32, total // VG_ADAMW_BLOCK

        def arena(t, n, dtype):
            if t is None:
                return torch.zeros(n, dtype=dtype, device=device)
            if t.dtype != dtype or t.numel() < n or not t.is_contiguous() or t.device != device:
                raise ValueError(f"AdamWState: an arena must be contiguous {dtype} of {n} elements")
            return t
        self.m, self.v = arena(m, total, code), arena(v, total, code)
        self.m_scale = arena(m_scale, blocks, torch.float32) if bits == 8 else None
        self.v_scale = arena(v_scale, blocks, torch.float32) if bits == 8 else None
        self._keep = [t.detach() for t in (*params, *grads, *(masters or []))]  # the memory, whoever else lets go of it
        # parameters that autograd fills: what may be replaced behind the table's back, and where it lay (75 ns a
        # tensor to look at in each step; buffers of the caller's own cost nothing)
        self._autograd = [(p, g) for p, g in zip(params, grads) if p.is_leaf and p.grad is g]
        theirs = [t for p, g, x in zip(params, grads, masters or [None] * len(params)) if p.is_leaf and p.grad is g
                  for t in (p, g, x) if t is not None]
        self._moving, self._at = theirs, [t.data_ptr() for t in theirs]
        size = 1 if bits == 8 else 4

        def at(t, n):
            return None if t is None else t.data_ptr() + n
        self.table = (AdamWTensorStruct * len(params))()
        for i, (p, g, o) in enumerate(zip(params, grads, self.offsets)):
            s = o // VG_ADAMW_BLOCK * 4
            self.table[i] = AdamWTensorStruct(p.data_ptr(), g.data_ptr(),
                                              None if masters is None else masters[i].data_ptr(),
                                              at(self.m, size * o), at(self.v, size * o), at(self.m_scale, s),
                                              at(self.v_scale, s), p.numel(), decay[i], _DT[p.dtype])


    def check_in_place(self) -> None:
        """ValueError if autograd's parameters or gradients, or their masters, are not those of the table any more."""
        for p, g in self._autograd:
            if p.grad is not g:
                raise ValueError("AdamWState: a parameter has another .grad than the state was made with; make a new "
                                 "state, and keep the gradients (zero_grad(set_to_none=False))")
        if self._at != [t.data_ptr() for t in self._moving]:
            raise ValueError("AdamWState: a parameter, its gradient or master has moved; make a new state")


def vg_adamw_step(state: AdamWState, step: int, lr: float, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0,
                  stream=None) -> None:
    """One AdamW step (counted from 1) over all of the state's parameters, in place."""
    state.check_in_place()
    _check(lib().vg_adamw_step(state.table, len(state.table), state.bits, step, lr, beta1, beta2, eps, grad_scale,
                               _s(stream)), "vg_adamw_step")


def vg_adamw_decode(codes, scales, out, second: bool, stream=None) -> None:
    """out[i] = the value of 8-bit moment code i (second: of v, else of m); one scale per 256 codes."""
    n = codes.numel()
    if codes.dtype != torch.uint8 or scales.dtype != torch.float32 or out.dtype != torch.float32 \
            or out.numel() != n or scales.numel() < -(-n // VG_ADAMW_BLOCK) \
            or not (codes.is_contiguous() and scales.is_contiguous() and out.is_contiguous()):
        raise ValueError("vg_adamw_decode: codes uint8 [n], scales float32 [ceil(n / 256)], out float32 [n]")
    _on(_gpu(codes, "vg_adamw_decode"), "vg_adamw_decode", scales, out)
    _check(lib().vg_adamw_decode(_p(codes), _p(scales), n, int(second), _p(out), _s(stream)), "vg_adamw_decode")


# ---------------------------------------------------------------- recurrent-block operators
def _rows(t, dtype, shape, device, what):
    """vg_rows of a [rows, channels] tensor (any row stride), None for None."""
    if t is None:
        return None
    s = t.stride()
    if t.dtype != dtype or t.shape != shape or (s[1] != 1 and t.numel() > 0):
        raise ValueError(f"{what}: expected {dtype} {list(shape)} with contiguous elements, got {t.dtype} "
                         f"{list(t.shape)} of strides {s}")
    if t.get_device() != device:
        _on(device, what, t)
    return RowsStruct(t.data_ptr(), s[0])


def _flat(t, dtype, shape, device, what):
    """Address of a contiguous tensor, None for None."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: expected contiguous {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.get_device() != device:
        _on(device, what, t)
    return t.data_ptr()


def _current(device, stream, what):
    """Refuse tensors of another GPU than the call's: kernels are launched on the current one."""
    if torch.cuda.is_initialized() and device != torch._C._cuda_getDevice() or \
            stream is not None and device != stream.device_index:
        raise ValueError(f"{what}: the tensors are on GPU {device}, which is not the current GPU or not the stream's")


def _matrix(x, stream, what):
    """Shape, dtype and GPU of a [rows, channels] tensor."""
    if x.dim() != 2:
        raise ValueError(f"{what}: expected [rows, channels], got {list(x.shape)}")
    device = _gpu(x, what)
    _current(device, stream, what)
    return x.shape, x.dtype, device


def vg_layer_norm_fwd(x, weight, bias, y, stats, eps=1e-5, stream=None) -> None:
    """y = (x - mean) rstd weight + bias of each row of x [rows, channels] (any row stride); weight and bias
    [channels] or None; stats float32 [rows, 2] takes (mean, rstd) for the backward pass, or is None."""
    (n, c), dt, dev = _matrix(x, stream, "vg_layer_norm_fwd")
    _check(lib().vg_layer_norm_fwd(n, c, _DT.get(dt, -1), _rows(x, dt, (n, c), dev, "x"),
                                   _flat(weight, dt, (c,), dev, "weight"), _flat(bias, dt, (c,), dev, "bias"), eps,
                                   _rows(y, dt, (n, c), dev, "y"), _flat(stats, torch.float32, (n, 2), dev, "stats"),
                                   _s(stream)), "vg_layer_norm_fwd")


def vg_layer_norm_bwd(x, weight, stats, grad_y, grad_skip, grad_x, grad_weight, grad_bias, ws, stream=None) -> None:
    """Gradients of vg_layer_norm_fwd's x (plus grad_skip, unless None), weight and bias (None: not wanted; with both
    None, ws may be None too)."""
    (n, c), dt, dev = _matrix(x, stream, "vg_layer_norm_bwd")
    s = (n, c)
    _on(dev, "vg_layer_norm_bwd", ws)
    _check(lib().vg_layer_norm_bwd(n, c, _DT.get(dt, -1), _rows(x, dt, s, dev, "x"),
                                   _flat(weight, dt, (c,), dev, "weight"),
                                   _flat(stats, torch.float32, (n, 2), dev, "stats"),
                                   _rows(grad_y, dt, s, dev, "grad_y"), _rows(grad_skip, dt, s, dev, "grad_skip"),
                                   _rows(grad_x, dt, s, dev, "grad_x"),
                                   _flat(grad_weight, dt, (c,), dev, "grad_weight"),
                                   _flat(grad_bias, dt, (c,), dev, "grad_bias"), _p(ws),
                                   0 if ws is None else ws.numel() * ws.element_size(), _s(stream)),
           "vg_layer_norm_bwd")


def _word(number, what):
    """A whole number that C takes as one of 32 bits (ctypes would cut off the rest)."""
    if not 0 <= number < 1 << 32:
        raise ValueError(f"{what} must be a whole number of 32 bits, got {number}")
    return number


def layer_norm_workspace(n, channels, device="cuda") -> torch.Tensor:
    nb = int(lib().vg_layer_norm_workspace_bytes(n, channels))
    if nb == 0:
        raise VGError(VG_ERR_INVALID_ARG, "vg_layer_norm_workspace_bytes")
    return torch.empty(nb, dtype=torch.uint8, device=device)


def gated_scan_workspace(n, channels, batch, dtype, device="cuda") -> torch.Tensor:
    """Workspace of vg_gated_scan_fwd and _bwd, its error record zero; it serves calls of fewer rows too."""
    nb = int(lib().vg_gated_scan_workspace_bytes(ScanStruct(n, channels, batch, _DT.get(dtype, -1), 0, None, None)))
    if nb == 0:
        raise VGError(VG_ERR_INVALID_ARG, "vg_gated_scan_workspace_bytes")
    ws = torch.empty(nb, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def gated_scan_carries(n, channels, device="cuda") -> torch.Tensor:
    """The states that vg_gated_scan_fwd keeps for vg_gated_scan_bwd."""
    return torch.empty(int(lib().vg_gated_scan_carry_rows(n)), channels, dtype=torch.float32, device=device)


def _scan(gate, offsets, order, carries, flags, stream, what):
    """(vg_scan, shape, batch, dtype, device, carries' address) of a call, checked."""
    (n, c), dt, dev = _matrix(gate, stream, what)
    batch = offsets.numel() - 1
    f32 = torch.float32
    rows = -(-n // VG_SCAN_CARRY_ROWS)
    return (ScanStruct(n, c, batch, _DT.get(dt, -1), _word(flags, "flags"),
                       _flat(offsets, torch.int32, (batch + 1,), dev, "offsets"),
                       _flat(order, torch.int32, (n,), dev, "order")), (n, c), (batch, c), dt, dev,
            _flat(carries, f32, (rows, c), dev, "carries"))


def vg_gated_scan_fwd(gate, x, offsets, order, first, out, last, carries, ws, flags=0, stream=None) -> None:
    """out_t = h_t = a_t h_{t-1} + (1 - a_t) x_t with a = sigmoid(gate), along each sequence.

    gate, x, out [rows, channels] (any row stride); offsets int32 [batch + 1]; order int32 [rows], the row of each
    position, or None; first, last float32 [batch, channels], the states before and after, or None; carries
    (gated_scan_carries) for the backward pass, or None; flags VG_SCAN_REVERSE, VG_SCAN_FREE_INPUT."""
    a, s, b, dt, dev, kept = _scan(gate, offsets, order, carries, flags, stream, "vg_gated_scan_fwd")
    _on(dev, "vg_gated_scan_fwd", ws)
    _check(lib().vg_gated_scan_fwd(a, _rows(gate, dt, s, dev, "gate"), _rows(x, dt, s, dev, "x"),
                                   _flat(first, torch.float32, b, dev, "first"), _rows(out, dt, s, dev, "out"),
                                   _flat(last, torch.float32, b, dev, "last"), kept, _p(ws),
                                   0 if ws is None else ws.numel() * ws.element_size(), _s(stream)), "vg_gated_scan_fwd")


def vg_gated_scan_bwd(gate, x, offsets, order, first, carries, grad_out, grad_last, grad_gate, grad_x, grad_first, ws,
                      flags=0, stream=None) -> None:
    """Gradients of vg_gated_scan_fwd's gate, x and first (None: not wanted), from its carries; grad_last may be None."""
    a, s, b, dt, dev, kept = _scan(gate, offsets, order, carries, flags, stream, "vg_gated_scan_bwd")
    _on(dev, "vg_gated_scan_bwd", ws)
    _check(lib().vg_gated_scan_bwd(a, _rows(gate, dt, s, dev, "gate"), _rows(x, dt, s, dev, "x"),
                                   _flat(first, torch.float32, b, dev, "first"), kept,
                                   _rows(grad_out, dt, s, dev, "grad_out"),
                                   _flat(grad_last, torch.float32, b, dev, "grad_last"),
                                   _rows(grad_gate, dt, s, dev, "grad_gate"), _rows(grad_x, dt, s, dev, "grad_x"),
                                   _flat(grad_first, torch.float32, b, dev, "grad_first"), _p(ws),
                                   0 if ws is None else ws.numel() * ws.element_size(), _s(stream)), "vg_gated_scan_bwd")


def vg_gated_scan_step(gate, x, state, out, flags=0, stream=None) -> None:
    """One token of each of the rows' sequences: state float32 [rows, channels] goes from h_{t-1} to h_t, out = h_t."""
    s, dt, dev = _matrix(gate, stream, "vg_gated_scan_step")
    _check(lib().vg_gated_scan_step(s[0], s[1], _DT.get(dt, -1), _word(flags, "flags"), _rows(gate, dt, s, dev, "gate"),
                                    _rows(x, dt, s, dev, "x"), _flat(state, torch.float32, s, dev, "state"),
                                    _rows(out, dt, s, dev, "out"), _s(stream)), "vg_gated_scan_step")


def vg_gated_scan_status(ws, stream=None) -> int:
    return lib().vg_gated_scan_status(_p(ws), _s(stream))


def _dropout(name, x, residual, p, rng, call, out, stream):
    dt, dev = x.dtype, _gpu(x, name)
    _current(dev, stream, name)
    if rng.dtype not in (torch.int64, torch.uint64):
        raise ValueError(f"{name}: rng must be int64 [2] (seed, step)")
    args = [x.numel(), _dtype_code(x), _flat(x, dt, x.shape, dev, "input")]
    if name == "vg_dropout_add_fwd":
        args.append(_flat(residual, dt, x.shape, dev, "residual"))
    _check(getattr(lib(), name)(*args, p, _flat(rng, rng.dtype, (2,), dev, "rng"), _word(call, "call"),
                                _flat(out, dt, x.shape, dev, "output"), _s(stream)), name)


def vg_dropout_add_fwd(x, residual, p, rng, call, out, stream=None) -> None:
    """out = residual + dropout(x); residual may be None.  rng int64 [2] on the GPU: (seed, step); call, a number of
    32 bits that tells this call's mask from the others of the step."""
    _dropout("vg_dropout_add_fwd", x, residual, p, rng, call, out, stream)


def vg_dropout_add_bwd(grad_out, p, rng, call, grad_x, stream=None) -> None:
    """grad_x = the gradient of vg_dropout_add_fwd's x, with the mask of the same p, rng and call."""
    _dropout("vg_dropout_add_bwd", grad_out, None, p, rng, call, grad_x, stream)
