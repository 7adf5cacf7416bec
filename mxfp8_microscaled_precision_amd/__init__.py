"""MXFP8 microscaled-precision hot path for MI355X (gfx950).

Thin Python binding over the C ABI in ``include/mxfp8.h`` (``libmxfp8.so``,
built in-tree by ``python -m mxfp8_microscaled_precision_amd.build``).  The
functions named ``mx_*`` take raw device pointers and sizes exactly like the C
entry points; ``quant``, ``quant_batched``, ``quant_grouped_col``, ``gemm``,
``grouped_gemm``, ``grouped_gemm_wgrad``, ``process_quant_result`` and, around
the experts' products, ``route``, ``route_backward``, ``dispatch``,
``dispatch_quant``, ``combine``, ``combine_backward``, ``grad_norm`` and
``grad_clip`` and, for 4-bit weights and 8-bit checkpoints, ``quant4``,
``dequant``, ``gemm4``, ``grouped_gemm4``, ``swiglu_quant``,
``swiglu_backward``, ``swiglu_backward_quant``, ``requant_col`` and
``requant_grouped_col`` marshal torch CUDA tensors (device memory and the
current stream only) into those calls.  Every step of the computation runs in
the HIP kernels; there is no CPU fallback: without the built library, or on a
device other than gfx950, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Any, NamedTuple

__all__ = [
    "MXError", "lib", "mx_device_check", "mx_arch_supported", "mx_status_string",
    "mx_last_error", "mx_quant", "mx_gemm", "mx_grouped_gemm", "mx_grouped_gemm_workspace_size",
    "mx_quant_elem", "mx_gemm_elem",
    "mx_grouped_gemm_elem", "mx_quant_grouped_col_elem", "mx_grouped_gemm_wgrad_elem",
    "mx_gemm_quant", "gemm_quant",
    "mx_quant_batched", "mx_quant_batched_elem",
    "mx_grouped_col_capacity", "mx_quant_grouped_col", "mx_grouped_gemm_wgrad", "quant", "gemm",
    "grouped_gemm", "quant_batched", "quant_grouped_col", "grouped_gemm_wgrad",
    "grouped_col_capacity", "process_quant_result", "QUANT_MODES", "GEMM_LAYOUTS",
    "BSCALE_KINDS", "ELEM_TYPES",
    "mx_route", "mx_route_workspace_size", "mx_route_backward", "mx_dispatch", "mx_dispatch_quant",
    "mx_combine", "mx_combine_backward", "mx_grad_norm", "mx_grad_clip",
    "mx_grad_norm_workspace_size", "Routing", "route", "route_backward", "dispatch",
    "dispatch_quant", "combine", "combine_backward", "grad_norm", "grad_clip", "SCORES",
    "GROUP_VALUES",
    "mx_quant4", "mx_dequant", "mx_gemm4", "mx_gemm4_workspace_size", "mx_grouped_gemm4",
    "mx_swiglu_quant",
    "mx_swiglu_backward", "mx_swiglu_backward_quant", "mx_requant_col", "mx_requant_grouped_col",
    "quant4", "dequant", "gemm4", "grouped_gemm4", "swiglu_quant", "swiglu_backward",
    "swiglu_backward_quant", "requant_col", "requant_grouped_col", "OPERAND_ELEMS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxfp8.so")

MX_OK = 0
QUANT_MODES = {"row": 0, "col": 1, "dual": 2, "32x32": 3}
GEMM_LAYOUTS = {"fprop": 0, "dgrad": 1, "wgrad": 2}
BSCALE_KINDS = {"1x32": 0, "32x32": 1}
ELEM_TYPES = {"e4m3": 0, "e5m2": 1}
OPERAND_ELEMS = {**ELEM_TYPES, "e2m1": 4}  # element types that a product's or a restored operand has
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_VALUES = {"top2": 0, "max": 1}


class MXError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{mx_status_string(status)} (status {status}): {detail}")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmxfp8.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m mxfp8_microscaled_precision_amd.build` (hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, c_int, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.mx_device_check.restype = c_int
        L.mx_device_check.argtypes = [c_int]
        L.mx_arch_supported.restype = c_int
        L.mx_arch_supported.argtypes = [ctypes.c_char_p]
        L.mx_status_string.restype = ctypes.c_char_p
        L.mx_status_string.argtypes = [c_int]
        L.mx_last_error.restype = ctypes.c_char_p
        L.mx_last_error.argtypes = []
        L.mx_quant.restype = c_int
        L.mx_quant.argtypes = [c_int, vp, i64, i64, vp, vp, vp, vp, vp]
        L.mx_gemm.restype = c_int
        L.mx_gemm.argtypes = [c_int, c_int, i64, i64, i64, vp, vp, vp, vp, vp, vp]
        L.mx_grouped_gemm.restype = c_int
        L.mx_grouped_gemm.argtypes = [i64, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp]
        L.mx_grouped_gemm_workspace_size.restype = sz
        L.mx_grouped_gemm_workspace_size.argtypes = [i64, i64, i64]
        L.mx_quant_elem.restype = c_int
        L.mx_quant_elem.argtypes = [c_int, c_int, vp, i64, i64, vp, vp, vp, vp, vp]
        L.mx_gemm_elem.restype = c_int
        L.mx_gemm_elem.argtypes = [c_int, c_int, c_int, c_int, i64, i64, i64, vp, vp, vp, vp, vp, vp]
        L.mx_grouped_gemm_elem.restype = c_int
        L.mx_grouped_gemm_elem.argtypes = [c_int, c_int, i64, vp, i64, i64, i64, vp, vp, vp, vp, vp,
                                           vp, sz, vp]
        L.mx_gemm_quant.restype = c_int
        L.mx_gemm_quant.argtypes = [c_int, c_int, c_int, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp]
        L.mx_quant_batched.restype = c_int
        L.mx_quant_batched.argtypes = [c_int, vp, i64, i64, i64, vp, vp, vp, vp, vp]
        L.mx_quant_batched_elem.restype = c_int
        L.mx_quant_batched_elem.argtypes = [c_int, c_int, vp, i64, i64, i64, vp, vp, vp, vp, vp]
        L.mx_grouped_col_capacity.restype = i64
        L.mx_grouped_col_capacity.argtypes = [i64, i64]
        L.mx_quant_grouped_col.restype = c_int
        L.mx_quant_grouped_col.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp]
        L.mx_grouped_gemm_wgrad.restype = c_int
        L.mx_grouped_gemm_wgrad.argtypes = [i64, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp]
        L.mx_quant_grouped_col_elem.restype = c_int
        L.mx_quant_grouped_col_elem.argtypes = [c_int, vp, i64, i64, i64, vp, vp, vp, vp]
        L.mx_grouped_gemm_wgrad_elem.restype = c_int
        L.mx_grouped_gemm_wgrad_elem.argtypes = [c_int, c_int, i64, vp, i64, i64, i64, vp, vp, vp, vp,
                                                 vp, vp]
        f32 = ctypes.c_float
        L.mx_route.restype = c_int
        L.mx_route.argtypes = [c_int, c_int, vp, vp, i64, i64, i64, i64, i64, c_int, c_int, f32, vp,
                               vp, vp, vp, vp, sz, vp]
        L.mx_route_workspace_size.restype = sz
        L.mx_route_workspace_size.argtypes = [i64, i64]
        L.mx_route_backward.restype = c_int
        L.mx_route_backward.argtypes = [c_int, c_int, vp, vp, vp, i64, i64, i64, c_int, f32, vp, vp]
        L.mx_dispatch.restype = c_int
        L.mx_dispatch.argtypes = [vp, i64, i64, i64, i64, vp, vp, vp, vp]
        L.mx_dispatch_quant.restype = c_int
        L.mx_dispatch_quant.argtypes = [c_int, vp, i64, i64, i64, i64, vp, vp, vp, vp, vp]
        L.mx_combine.restype = c_int
        L.mx_combine.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp]
        L.mx_combine_backward.restype = c_int
        L.mx_combine_backward.argtypes = [vp, vp, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp]
        L.mx_grad_norm.restype = c_int
        L.mx_grad_norm.argtypes = [i64, vp, vp, vp, vp, vp, sz, vp]
        L.mx_grad_clip.restype = c_int
        L.mx_grad_clip.argtypes = [i64, vp, vp, vp, f32, vp, vp, sz, vp]
        L.mx_grad_norm_workspace_size.restype = sz
        L.mx_grad_norm_workspace_size.argtypes = [i64]
        L.mx_quant4.restype = c_int
        L.mx_quant4.argtypes = [c_int, vp, i64, i64, i64, vp, vp, vp, vp, vp]
        L.mx_dequant.restype = c_int
        L.mx_dequant.argtypes = [c_int, vp, vp, i64, i64, vp, vp]
        L.mx_gemm4.restype = c_int
        L.mx_gemm4.argtypes = [c_int, i64, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp]
        L.mx_gemm4_workspace_size.restype = sz
        L.mx_gemm4_workspace_size.argtypes = [c_int, i64, i64, i64]
        L.mx_grouped_gemm4.restype = c_int
        L.mx_grouped_gemm4.argtypes = [c_int, i64, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp]
        L.mx_swiglu_quant.restype = c_int
        L.mx_swiglu_quant.argtypes = [c_int, c_int, vp, i64, i64, vp, vp, vp, vp, vp]
        L.mx_swiglu_backward.restype = c_int
        L.mx_swiglu_backward.argtypes = [c_int, vp, vp, vp, i64, i64, vp, vp]
        L.mx_swiglu_backward_quant.restype = c_int
        L.mx_swiglu_backward_quant.argtypes = [c_int, c_int, vp, vp, vp, i64, i64, vp, vp, vp]
        L.mx_requant_col.restype = c_int
        L.mx_requant_col.argtypes = [c_int, c_int, vp, vp, i64, i64, vp, vp, vp]
        L.mx_requant_grouped_col.restype = c_int
        L.mx_requant_grouped_col.argtypes = [c_int, c_int, vp, vp, i64, i64, i64, vp, vp, vp, vp]
        _lib = L
    return _lib


# ---------------------------------------------------------------------------
# The C entry points, same names and arguments (raw pointers as ints)
# ---------------------------------------------------------------------------

def mx_device_check(device: int) -> int:
    return lib().mx_device_check(device)


def mx_arch_supported(name: str) -> int:
    return lib().mx_arch_supported(name.encode() if name is not None else None)


def mx_status_string(status: int) -> str:
    return lib().mx_status_string(status).decode()


def mx_last_error() -> str:
    return lib().mx_last_error().decode()


def mx_quant(mode, x, rows, cols, q, s, q_t, s_t, stream) -> int:
    return lib().mx_quant(mode, x, rows, cols, q, s, q_t, s_t, stream)


def mx_gemm(layout, bkind, M, N, K, a, sa, b, sb, c, stream) -> int:
    return lib().mx_gemm(layout, bkind, M, N, K, a, sa, b, sb, c, stream)


def mx_grouped_gemm(G, offsets, T, N, K, a, sa, b, sb, c, workspace, workspace_bytes, stream) -> int:
    return lib().mx_grouped_gemm(G, offsets, T, N, K, a, sa, b, sb, c, workspace, workspace_bytes,
                                 stream)


def mx_grouped_gemm_workspace_size(G, T, N) -> int:
    return lib().mx_grouped_gemm_workspace_size(G, T, N)


def mx_grouped_gemm_elem(a_elem, b_elem, G, offsets, T, N, K, a, sa, b, sb, c, workspace,
                         workspace_bytes, stream) -> int:
    return lib().mx_grouped_gemm_elem(a_elem, b_elem, G, offsets, T, N, K, a, sa, b, sb, c,
                                      workspace, workspace_bytes, stream)


def mx_quant_elem(mode, elem, x, rows, cols, q, s, q_t, s_t, stream) -> int:
    return lib().mx_quant_elem(mode, elem, x, rows, cols, q, s, q_t, s_t, stream)


def mx_gemm_elem(layout, bkind, a_elem, b_elem, M, N, K, a, sa, b, sb, c, stream) -> int:
    return lib().mx_gemm_elem(layout, bkind, a_elem, b_elem, M, N, K, a, sa, b, sb, c, stream)


def mx_gemm_quant(layout, bkind, out_elem, M, N, K, a, sa, b, sb, q, s, stream) -> int:
    return lib().mx_gemm_quant(layout, bkind, out_elem, M, N, K, a, sa, b, sb, q, s, stream)


def mx_quant_batched(mode, x, batch, rows, cols, q, s, q_t, s_t, stream) -> int:
    return lib().mx_quant_batched(mode, x, batch, rows, cols, q, s, q_t, s_t, stream)


def mx_quant_batched_elem(mode, elem, x, batch, rows, cols, q, s, q_t, s_t, stream) -> int:
    return lib().mx_quant_batched_elem(mode, elem, x, batch, rows, cols, q, s, q_t, s_t, stream)


def mx_grouped_col_capacity(T, G) -> int:
    return lib().mx_grouped_col_capacity(T, G)


def mx_quant_grouped_col(x, T, C, G, offsets, q_t, s_t, stream) -> int:
    return lib().mx_quant_grouped_col(x, T, C, G, offsets, q_t, s_t, stream)


def mx_grouped_gemm_wgrad(G, offsets, T, M, N, a, sa, b, sb, c, stream) -> int:
    return lib().mx_grouped_gemm_wgrad(G, offsets, T, M, N, a, sa, b, sb, c, stream)


def mx_quant_grouped_col_elem(elem, x, T, C, G, offsets, q_t, s_t, stream) -> int:
    return lib().mx_quant_grouped_col_elem(elem, x, T, C, G, offsets, q_t, s_t, stream)


def mx_grouped_gemm_wgrad_elem(a_elem, b_elem, G, offsets, T, M, N, a, sa, b, sb, c, stream) -> int:
    return lib().mx_grouped_gemm_wgrad_elem(a_elem, b_elem, G, offsets, T, M, N, a, sa, b, sb, c,
                                            stream)


def mx_route(score, dtype, logits, bias, T, E, top_k, n_groups, top_groups, group_value, renormalize,
             scale, weights, experts, offsets, slots, workspace, workspace_bytes, stream) -> int:
    return lib().mx_route(score, dtype, logits, bias, T, E, top_k, n_groups, top_groups, group_value,
                          renormalize, scale, weights, experts, offsets, slots, workspace,
                          workspace_bytes, stream)


def mx_route_workspace_size(T, E) -> int:
    return lib().mx_route_workspace_size(T, E)


def mx_route_backward(score, dtype, dweights, logits, experts, T, E, top_k, renormalize, scale,
                      dlogits, stream) -> int:
    return lib().mx_route_backward(score, dtype, dweights, logits, experts, T, E, top_k, renormalize,
                                   scale, dlogits, stream)


def mx_dispatch(x, T, H, top_k, E, offsets, slots, y, stream) -> int:
    return lib().mx_dispatch(x, T, H, top_k, E, offsets, slots, y, stream)


def mx_dispatch_quant(elem, x, T, H, top_k, E, offsets, slots, q, s, stream) -> int:
    return lib().mx_dispatch_quant(elem, x, T, H, top_k, E, offsets, slots, q, s, stream)


def mx_combine(y, T, H, top_k, slots, weights, residual, out, stream) -> int:
    return lib().mx_combine(y, T, H, top_k, slots, weights, residual, out, stream)


def mx_combine_backward(dout, y, T, H, top_k, E, offsets, slots, weights, dy, dweights,
                        stream) -> int:
    return lib().mx_combine_backward(dout, y, T, H, top_k, E, offsets, slots, weights, dy, dweights,
                                     stream)


def mx_grad_norm(n, tensors, numels, dtypes, norm, workspace, workspace_bytes, stream) -> int:
    return lib().mx_grad_norm(n, tensors, numels, dtypes, norm, workspace, workspace_bytes, stream)


def mx_grad_clip(n, tensors, numels, dtypes, max_norm, norm, workspace, workspace_bytes,
                 stream) -> int:
    return lib().mx_grad_clip(n, tensors, numels, dtypes, max_norm, norm, workspace, workspace_bytes,
                              stream)


def mx_grad_norm_workspace_size(n) -> int:
    return lib().mx_grad_norm_workspace_size(n)


def mx_quant4(mode, x, batch, rows, cols, q, s, q_t, s_t, stream) -> int:
    return lib().mx_quant4(mode, x, batch, rows, cols, q, s, q_t, s_t, stream)


def mx_dequant(elem, q, s, rows, cols, y, stream) -> int:
    return lib().mx_dequant(elem, q, s, rows, cols, y, stream)


def mx_gemm4(a_elem, M, N, K, a, sa, b, sb, c, workspace, workspace_bytes, stream) -> int:
    return lib().mx_gemm4(a_elem, M, N, K, a, sa, b, sb, c, workspace, workspace_bytes, stream)


def mx_gemm4_workspace_size(a_elem, M, N, K) -> int:
    return lib().mx_gemm4_workspace_size(a_elem, M, N, K)


def mx_grouped_gemm4(a_elem, G, offsets, T, N, K, a, sa, b, sb, c, stream) -> int:
    return lib().mx_grouped_gemm4(a_elem, G, offsets, T, N, K, a, sa, b, sb, c, stream)


def mx_swiglu_quant(elem, ckpt_elem, x, T, F, q, s, ckpt_q, ckpt_s, stream) -> int:
    return lib().mx_swiglu_quant(elem, ckpt_elem, x, T, F, q, s, ckpt_q, ckpt_s, stream)


def mx_swiglu_backward(ckpt_elem, dh, ckpt_q, ckpt_s, T, F, dx, stream) -> int:
    return lib().mx_swiglu_backward(ckpt_elem, dh, ckpt_q, ckpt_s, T, F, dx, stream)


def mx_swiglu_backward_quant(ckpt_elem, elem, dh, ckpt_q, ckpt_s, T, F, q, s, stream) -> int:
    return lib().mx_swiglu_backward_quant(ckpt_elem, elem, dh, ckpt_q, ckpt_s, T, F, q, s, stream)


def mx_requant_col(elem, out_elem, q, s, rows, cols, q_t, s_t, stream) -> int:
    return lib().mx_requant_col(elem, out_elem, q, s, rows, cols, q_t, s_t, stream)


def mx_requant_grouped_col(elem, out_elem, q, s, T, C, G, offsets, q_t, s_t, stream) -> int:
    return lib().mx_requant_grouped_col(elem, out_elem, q, s, T, C, G, offsets, q_t, s_t, stream)


def _check(status: int):
    if status != MX_OK:
        raise MXError(status, mx_last_error())


# ---------------------------------------------------------------------------
# torch marshalling
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    # the raw handle alone: building a torch.cuda.Stream object takes 2 us of
    # host time, as long as a launch
    torch = _torch()
    index = torch.cuda.current_device() if device.index is None else device.index
    return torch._C._cuda_getCurrentRawStream(index)


def _written(tensors):
    """Counts a write into a caller's tensors, so that a backward pass that
    has saved one raises instead of using the new values."""
    _torch().autograd.graph.increment_version(tensors)


def _need(t, dtype, name, ndim=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    # the library launches on the current device
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{t.get_device()}, not on the current device "
                         f"cuda:{torch.cuda.current_device()}")


def _shape(t, shape, name):
    """The library reads exactly the bytes the sizes describe, so every
    operand must have them (a short tensor would be read past its end)."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _gemm_operands(a, sa, b, sb, layout, bscale):
    """(M, N, K) of a dense GEMM call, after checking every operand's shape
    against them (K % 32 and N % 32 for 32x32 tiles are left to the library,
    which reports them as unsupported shapes)."""
    M, K = a.shape
    tiles = bscale == "32x32"
    N = b.shape[1] if (tiles and layout == "dgrad") else b.shape[0]
    if K % 32 == 0:
        _shape(sa, (M, K // 32), "sa")
        if not tiles:
            _shape(b, (N, K), "b")
            _shape(sb, (N, K // 32), "sb")
        elif N % 32 == 0:
            if layout == "dgrad":      # the shared weight [K, N], tiles along both
                _shape(b, (K, N), "b")
                _shape(sb, (K // 32, N // 32), "sb")
            else:
                _shape(b, (N, K), "b")
                _shape(sb, (N // 32, K // 32), "sb")
    return M, N, K


def quant(x, mode: str = "row", elem: str = "e4m3"):
    """Dynamic MX quantisation of a BF16 [rows, cols] tensor.

    mode "row"   -> (q [rows,cols], s [rows,cols/32])
         "col"   -> (q_t [cols,rows], s_t [cols,rows/32])
         "dual"  -> (q, s, q_t, s_t)
         "32x32" -> (q [rows,cols], s [rows/32,cols/32])
    Payloads are uint8 E4M3 (or, with elem="e5m2", E5M2) bytes, scales
    uint8 E8M0 bytes.
    """
    torch = _torch()
    if mode not in QUANT_MODES:
        raise ValueError(f"unknown quantisation mode {mode!r}; expected one of {list(QUANT_MODES)}")
    if elem not in ELEM_TYPES:
        raise ValueError(f"unknown element type {elem!r}; expected one of {list(ELEM_TYPES)}")
    _need(x, torch.bfloat16, "x", 2)
    R, C = x.shape
    dev, u8 = x.device, torch.uint8
    q = s = qt = st = None
    if mode in ("row", "dual", "32x32"):
        q = torch.empty((R, C), dtype=u8, device=dev)
        s = torch.empty((R // 32, C // 32) if mode == "32x32" else (R, C // 32), dtype=u8, device=dev)
    if mode in ("col", "dual"):
        qt = torch.empty((C, R), dtype=u8, device=dev)
        st = torch.empty((C, R // 32), dtype=u8, device=dev)
    _check(mx_quant_elem(QUANT_MODES[mode], ELEM_TYPES[elem], _ptr(x), R, C, _ptr(q), _ptr(s),
                         _ptr(qt), _ptr(st), _stream(dev)))
    if mode == "row" or mode == "32x32":
        return q, s
    if mode == "col":
        return qt, st
    return q, s, qt, st


def gemm(a, sa, b, sb, layout: str = "fprop", bscale: str = "1x32", out=None,
         a_elem: str = "e4m3", b_elem: str = "e4m3"):
    """MXFP8 GEMM C = A * B^T (FP32 accumulation, BF16 result).

    a [M,K] u8 + sa [M,K/32]; b [N,K] u8 + sb [N,K/32] for 1x32 scales;
    with bscale "32x32": fprop b [N,K] + tiles [N/32,K/32], dgrad b [K,N]
    (the shared weight, contracted over rows) + tiles [K/32,N/32].
    a_elem / b_elem: payload element types ("e4m3" or "e5m2").
    """
    torch = _torch()
    if layout not in GEMM_LAYOUTS or bscale not in BSCALE_KINDS:
        raise ValueError(f"unknown layout {layout!r} or B scale kind {bscale!r}")
    if a_elem not in ELEM_TYPES or b_elem not in ELEM_TYPES:
        raise ValueError(f"unknown element types {a_elem!r}, {b_elem!r}")
    for t, n in ((a, "a"), (sa, "sa"), (b, "b"), (sb, "sb")):
        _need(t, torch.uint8, n, 2)
    M, N, K = _gemm_operands(a, sa, b, sb, layout, bscale)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _need(out, torch.bfloat16, "out", 2)
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must be [{M}, {N}]")
    _check(mx_gemm_elem(GEMM_LAYOUTS[layout], BSCALE_KINDS[bscale], ELEM_TYPES[a_elem],
                        ELEM_TYPES[b_elem], M, N, K, _ptr(a), _ptr(sa), _ptr(b), _ptr(sb),
                        _ptr(out), _stream(a.device)))
    return out


def gemm_quant(a, sa, b, sb, layout: str = "fprop", bscale: str = "1x32", out_elem: str = "e4m3"):
    """Fused producer: the GEMM's BF16 result quantised in 1x32 blocks along N
    in the epilogue -> (q [M,N] u8, s [M,N/32] u8), equal to
    quant(gemm(...), "row", out_elem)."""
    torch = _torch()
    if layout not in GEMM_LAYOUTS or bscale not in BSCALE_KINDS or out_elem not in ELEM_TYPES:
        raise ValueError(f"unknown layout {layout!r}, B scale kind {bscale!r} or element {out_elem!r}")
    for t, n in ((a, "a"), (sa, "sa"), (b, "b"), (sb, "sb")):
        _need(t, torch.uint8, n, 2)
    M, N, K = _gemm_operands(a, sa, b, sb, layout, bscale)
    q = torch.empty((M, N), dtype=torch.uint8, device=a.device)
    s = torch.empty((M, N // 32), dtype=torch.uint8, device=a.device)
    _check(mx_gemm_quant(GEMM_LAYOUTS[layout], BSCALE_KINDS[bscale], ELEM_TYPES[out_elem], M, N, K,
                         _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(q), _ptr(s), _stream(a.device)))
    return q, s


def grouped_gemm(offsets, a, sa, b, sb, out=None, a_elem: str = "e4m3", b_elem: str = "e4m3"):
    """MoE grouped MXFP8 GEMM: rows offsets[g]:offsets[g+1] of a times b[g]^T.

    offsets int64 [G+1] on the device; a [T,K] u8 + sa [T,K/32];
    b [G,N,K] u8 + sb [G,N,K/32]; returns BF16 [T,N].  a_elem / b_elem:
    payload element types ("e4m3" or "e5m2").
    """
    torch = _torch()
    if a_elem not in ELEM_TYPES or b_elem not in ELEM_TYPES:
        raise ValueError(f"unknown element types {a_elem!r}, {b_elem!r}")
    _need(offsets, torch.int64, "offsets", 1)
    for t, n in ((a, "a"), (sa, "sa")):
        _need(t, torch.uint8, n, 2)
    for t, n in ((b, "b"), (sb, "sb")):
        _need(t, torch.uint8, n, 3)
    G = offsets.numel() - 1
    T, K = a.shape
    N = b.shape[1]
    if G < 1:
        raise ValueError("offsets must hold at least two entries (one group)")
    if K % 32 == 0:
        _shape(sa, (T, K // 32), "sa")
        _shape(b, (G, N, K), "b")
        _shape(sb, (G, N, K // 32), "sb")
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=a.device)
    _need(out, torch.bfloat16, "out", 2)
    _shape(out, (T, N), "out")
    nws = mx_grouped_gemm_workspace_size(G, T, N)
    ws = torch.empty(nws, dtype=torch.uint8, device=a.device) if nws else None
    _check(mx_grouped_gemm_elem(ELEM_TYPES[a_elem], ELEM_TYPES[b_elem], G, _ptr(offsets), T, N, K,
                                _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(out), _ptr(ws), nws,
                                _stream(a.device)))
    return out


def quant_batched(x, mode: str = "row", elem: str = "e4m3"):
    """mx_quant on every matrix of a BF16 stack x [B, rows, cols] (e.g. the
    per-expert weights of an MoE layer); outputs are the stacked per-matrix
    outputs of ``quant`` in the same mode and element type."""
    torch = _torch()
    if mode not in QUANT_MODES:
        raise ValueError(f"unknown quantisation mode {mode!r}; expected one of {list(QUANT_MODES)}")
    if elem not in ELEM_TYPES:
        raise ValueError(f"unknown element type {elem!r}; expected one of {list(ELEM_TYPES)}")
    _need(x, torch.bfloat16, "x", 3)
    B, R, C = x.shape
    dev, u8 = x.device, torch.uint8
    q = s = qt = st = None
    if mode in ("row", "dual", "32x32"):
        q = torch.empty((B, R, C), dtype=u8, device=dev)
        s = torch.empty((B, R // 32, C // 32) if mode == "32x32" else (B, R, C // 32), dtype=u8,
                        device=dev)
    if mode in ("col", "dual"):
        qt = torch.empty((B, C, R), dtype=u8, device=dev)
        st = torch.empty((B, C, R // 32), dtype=u8, device=dev)
    _check(mx_quant_batched_elem(QUANT_MODES[mode], ELEM_TYPES[elem], _ptr(x), B, R, C, _ptr(q),
                                 _ptr(s), _ptr(qt), _ptr(st), _stream(dev)))
    if mode == "row" or mode == "32x32":
        return q, s
    if mode == "col":
        return qt, st
    return q, s, qt, st


def grouped_col_capacity(T: int, G: int) -> int:
    """Columns of the per-group column-quantised token matrix."""
    cap = mx_grouped_col_capacity(int(T), int(G))
    if cap < 0:
        raise ValueError(f"no capacity for T={T}, G={G}")
    return cap


def quant_grouped_col(x, offsets, elem: str = "e4m3"):
    """Per-expert column quantisation along the token axis (MoE backward):
    x BF16 [T, C], offsets int64 [G+1] on the device ->
    (q_t [C, cap] u8, s_t [C, cap/32] u8), cap = grouped_col_capacity(T, G);
    group g's tokens at columns 128 (offsets[g] // 128 + g) on.  elem: the
    payload element type ("e4m3" or "e5m2")."""
    torch = _torch()
    if elem not in ELEM_TYPES:
        raise ValueError(f"unknown element type {elem!r}")
    _need(x, torch.bfloat16, "x", 2)
    _need(offsets, torch.int64, "offsets", 1)
    T, C = x.shape
    G = offsets.numel() - 1
    cap = grouped_col_capacity(T, G)
    qt = torch.empty((C, cap), dtype=torch.uint8, device=x.device)
    st = torch.empty((C, cap // 32), dtype=torch.uint8, device=x.device)
    _check(mx_quant_grouped_col_elem(ELEM_TYPES[elem], _ptr(x), T, C, G, _ptr(offsets), _ptr(qt),
                                     _ptr(st), _stream(x.device)))
    return qt, st


def grouped_gemm_wgrad(offsets, T: int, a, sa, b, sb, out=None, a_elem: str = "e4m3",
                       b_elem: str = "e4m3"):
    """Per-expert weight gradient: out[g] = A_g * B_g^T over group g's token
    columns of a [M, cap] and b [N, cap] (both from ``quant_grouped_col`` with
    the same offsets); returns BF16 [G, M, N].  a_elem / b_elem: the payload
    element types of a and b."""
    torch = _torch()
    if a_elem not in ELEM_TYPES or b_elem not in ELEM_TYPES:
        raise ValueError(f"unknown element types {a_elem!r}, {b_elem!r}")
    _need(offsets, torch.int64, "offsets", 1)
    for t, n in ((a, "a"), (sa, "sa"), (b, "b"), (sb, "sb")):
        _need(t, torch.uint8, n, 2)
    G = offsets.numel() - 1
    M, N = a.shape[0], b.shape[0]
    cap = grouped_col_capacity(T, G)
    if a.shape[1] != cap or b.shape[1] != cap or sa.shape != (M, cap // 32) or sb.shape != (N, cap // 32):
        raise ValueError(f"operands must be [rows, {cap}] with scales [rows, {cap // 32}]")
    if out is None:
        out = torch.empty((G, M, N), dtype=torch.bfloat16, device=a.device)
    _need(out, torch.bfloat16, "out", 3)
    if tuple(out.shape) != (G, M, N):
        raise ValueError(f"out must be [{G}, {M}, {N}]")
    _check(mx_grouped_gemm_wgrad_elem(ELEM_TYPES[a_elem], ELEM_TYPES[b_elem], G, _ptr(offsets), T, M,
                                      N, _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(out),
                                      _stream(a.device)))
    return out


def _dst_type_name(dst_type) -> str:
    """'e4m3' / 'e5m2' from a name or a torch FP8 dtype (the RFC passes the
    target dtype itself)."""
    if isinstance(dst_type, str):
        name = dst_type.lower()
    else:
        name = {"torch.float8_e4m3fn": "e4m3", "torch.float8_e5m2": "e5m2"}.get(str(dst_type), "")
    if name not in ELEM_TYPES:
        raise ValueError(f"unsupported dst_type {dst_type!r}: expected 'e4m3' (torch.float8_e4m3fn) "
                         f"or 'e5m2' (torch.float8_e5m2)")
    return name


def process_quant_result(weight, recipe: str = "mxfp8", dst_type="e4m3"):
    """Quantise a weight for both passes, in the RFC's tuple order
    (weight_fwd, scale_fwd, weight_bwd, scale_bwd).

    recipe   "mxfp8"       -> dual-axis 1x32: two FP8 copies, row and column
                              scales.
             "mxfp8-32x32" -> 32x32 tiles: weight_bwd IS weight_fwd and the
                              one tile scale array serves both passes (forward
                              blocks K along the columns, backward along the
                              rows).
    dst_type the FP8 payload type: "e4m3" / torch.float8_e4m3fn or "e5m2" /
             torch.float8_e5m2 (the scale rule follows the type's largest
             finite value).
    (MindSpeed RFC "add MXFP8-32x32 quantisation support to FSDP", sections
    3.3.3 and 3.5.2.3: process_quant_result_fn(weight, dst_type, config); an
    unsupported recipe or dst_type raises ValueError.)
    """
    if recipe not in ("mxfp8", "mxfp8-32x32"):
        raise ValueError(f"unsupported recipe {recipe!r}: expected 'mxfp8' or 'mxfp8-32x32'")
    elem = _dst_type_name(dst_type)
    if recipe == "mxfp8":
        q, s, qt, st = quant(weight, "dual", elem)
        return q, s, qt, st
    q, s = quant(weight, "32x32", elem)
    return q, s, q, s


# ---------------------------------------------------------------------------
# Around the experts' products: routing, token movement, gradient norm
# ---------------------------------------------------------------------------

class Routing(NamedTuple):
    """Which experts T tokens go to, and the expert order of their rows.

    weights [T, k] FP32, experts [T, k] INT32 (-1: no expert left), offsets
    [E + 1] INT64 (``grouped_gemm``'s), slots [T, k] INT32: the row of each
    choice in the expert order, -1 where there is none; the choices' rows are
    0 .. offsets[E] - 1, each taken once.
    """
    weights: Any
    experts: Any
    offsets: Any
    slots: Any


def _dtype_code(t, name):
    torch = _torch()
    if t.dtype == torch.float32:
        return 1
    if t.dtype == torch.bfloat16:
        return 0
    raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")


def _logits(logits):
    torch = _torch()
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a CUDA (HIP) tensor")
    code = _dtype_code(logits, "logits")
    _need(logits, logits.dtype, "logits", 2)
    return code


def route(logits, top_k: int, score: str = "softmax", bias=None, n_groups: int = 1,
          top_groups: int = 1, group_value: str = "top2", renormalize: bool = True,
          scale: float = 1.0) -> Routing:
    """Route T tokens to top_k of E experts (logits [T, E] BF16 or FP32).

    score       "softmax" over all experts or "sigmoid" of each.
    bias        FP32 [E], added to the scores for the choice only (balance).
    n_groups, top_groups, group_value
                with n_groups > 1 only the experts of the top_groups best
                groups of consecutive experts can be chosen; a group's value
                is the sum of its best two ("top2") or its best ("max").
    renormalize weights are divided by their sum; scale multiplies them.

    Experts with a logit of -inf are masked; a token with fewer than top_k
    unmasked experts has -1 and weight 0 in the places left over.  Equal
    values go to the lowest index.
    """
    torch = _torch()
    if score not in SCORES:
        raise ValueError(f"unknown score {score!r}; expected one of {list(SCORES)}")
    if group_value not in GROUP_VALUES:
        raise ValueError(f"unknown group value {group_value!r}; expected one of {list(GROUP_VALUES)}")
    code = _logits(logits)
    T, E = logits.shape
    if bias is not None:
        _need(bias, torch.float32, "bias", 1)
        _shape(bias, (E,), "bias")
    top_k = int(top_k)
    if not 1 <= top_k <= E:
        raise ValueError(f"top_k {top_k} not in [1, {E}]")
    dev, i32 = logits.device, torch.int32
    weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    experts = torch.empty((T, top_k), dtype=i32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int64, device=dev)
    slots = torch.empty((T, top_k), dtype=i32, device=dev)
    nws = mx_route_workspace_size(T, E)
    ws = torch.empty(nws, dtype=torch.uint8, device=dev) if nws else None
    _check(mx_route(SCORES[score], code, _ptr(logits), _ptr(bias), T, E, top_k, n_groups, top_groups,
                    GROUP_VALUES[group_value], int(bool(renormalize)), scale, _ptr(weights),
                    _ptr(experts), _ptr(offsets), _ptr(slots), _ptr(ws), nws, _stream(dev)))
    return Routing(weights, experts, offsets, slots)


def route_backward(dweights, logits, experts, score: str = "softmax", renormalize: bool = True,
                   scale: float = 1.0):
    """Gradient of ``route``'s weights with respect to the logits, for the
    choice it made: dweights FP32 [T, k], experts INT32 [T, k] -> dlogits
    [T, E] in the logits' type."""
    torch = _torch()
    if score not in SCORES:
        raise ValueError(f"unknown score {score!r}; expected one of {list(SCORES)}")
    code = _logits(logits)
    _need(dweights, torch.float32, "dweights", 2)
    _need(experts, torch.int32, "experts", 2)
    T, E = logits.shape
    k = experts.shape[1]
    _shape(experts, (T, k), "experts")
    _shape(dweights, (T, k), "dweights")
    out = torch.empty_like(logits)
    _check(mx_route_backward(SCORES[score], code, _ptr(dweights), _ptr(logits), _ptr(experts), T, E, k,
                             int(bool(renormalize)), scale, _ptr(out), _stream(logits.device)))
    return out


def _routed(routing, weights: bool = False):
    """(T, k, E) of a routing, after checking the tensors a call reads."""
    torch = _torch()
    offsets, slots = routing.offsets, routing.slots
    _need(slots, torch.int32, "routing.slots", 2)
    _need(offsets, torch.int64, "routing.offsets", 1)
    T, k = slots.shape
    if weights:
        _need(routing.weights, torch.float32, "routing.weights", 2)
        _shape(routing.weights, (T, k), "routing.weights")
    if offsets.numel() < 2:
        raise ValueError("routing.offsets must hold at least two entries (one expert)")
    return T, k, offsets.numel() - 1


def dispatch(x, routing):
    """Token rows in the expert order: x BF16 [T, H] -> BF16 [T k, H] with
    row slots[t, j] = x[t], rows offsets[E] and on zero.  Its gradient is
    ``combine(dy, routing, weighted=False)``.

    The rows below offsets[E] are the choices', as ``route`` lays them out.  A
    choice taken out of slots alone (-1) leaves its row there unwritten, with
    what the memory held: the experts' products and weight gradients would
    read it.  To drop choices, number the ones left anew, in offsets and
    slots."""
    torch = _torch()
    T, k, E = _routed(routing)
    _need(x, torch.bfloat16, "x", 2)
    H = x.shape[1]
    _shape(x, (T, H), "x")
    y = torch.empty((T * k, H), dtype=torch.bfloat16, device=x.device)
    _check(mx_dispatch(_ptr(x), T, H, k, E, _ptr(routing.offsets), _ptr(routing.slots), _ptr(y),
                       _stream(x.device)))
    return y


def dispatch_quant(x, routing, elem: str = "e4m3"):
    """``quant(dispatch(x, routing), "row", elem)`` in one pass: (q [T k, H]
    u8, s [T k, H/32] u8), ``grouped_gemm``'s a and sa.  offsets and slots as
    for ``dispatch``."""
    torch = _torch()
    if elem not in ELEM_TYPES:
        raise ValueError(f"unknown element type {elem!r}; expected one of {list(ELEM_TYPES)}")
    T, k, E = _routed(routing)
    _need(x, torch.bfloat16, "x", 2)
    H = x.shape[1]
    _shape(x, (T, H), "x")
    q = torch.empty((T * k, H), dtype=torch.uint8, device=x.device)
    s = torch.empty((T * k, H // 32), dtype=torch.uint8, device=x.device)
    _check(mx_dispatch_quant(ELEM_TYPES[elem], _ptr(x), T, H, k, E, _ptr(routing.offsets),
                             _ptr(routing.slots), _ptr(q), _ptr(s), _stream(x.device)))
    return q, s


def combine(y, routing, residual=None, weighted: bool = True, out=None):
    """Expert rows back to the tokens: y BF16 [T k, H] -> BF16 [T, H],
    out[t] = residual[t] + sum_j weights[t, j] y[slots[t, j]] (weights of one
    with weighted=False).  out may be residual itself; other memory of the
    inputs it may not share."""
    torch = _torch()
    T, k, _ = _routed(routing, weighted)
    _need(y, torch.bfloat16, "y", 2)
    H = y.shape[1]
    _shape(y, (T * k, H), "y")
    if residual is not None:
        _need(residual, torch.bfloat16, "residual", 2)
        _shape(residual, (T, H), "residual")
    given = out is not None
    if given:
        _need(out, torch.bfloat16, "out", 2)
        _shape(out, (T, H), "out")
    else:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    _check(mx_combine(_ptr(y), T, H, k, _ptr(routing.slots),
                      _ptr(routing.weights) if weighted else None, _ptr(residual), _ptr(out),
                      _stream(y.device)))
    if given:
        _written(out)
    return out


def combine_backward(dout, y, routing):
    """Gradient of ``combine``: (dy BF16 [T k, H], dweights FP32 [T, k]) from
    dout BF16 [T, H] and the y that was combined.  The residual's gradient is
    dout.  offsets and slots as for ``dispatch``, whose zero rows dy has."""
    torch = _torch()
    T, k, E = _routed(routing, True)
    _need(dout, torch.bfloat16, "dout", 2)
    _need(y, torch.bfloat16, "y", 2)
    H = dout.shape[1]
    _shape(dout, (T, H), "dout")
    _shape(y, (T * k, H), "y")
    dy = torch.empty((T * k, H), dtype=torch.bfloat16, device=y.device)
    dw = torch.empty((T, k), dtype=torch.float32, device=y.device)
    _check(mx_combine_backward(_ptr(dout), _ptr(y), T, H, k, E, _ptr(routing.offsets),
                               _ptr(routing.slots), _ptr(routing.weights), _ptr(dy), _ptr(dw),
                               _stream(y.device)))
    return dy, dw


def _tensor_list(tensors):
    """(count, pointers, element counts, element types) of gradients.  A list
    holds hundreds of tensors, so each property is checked in one sweep and
    the tensor at fault is looked for only once there is one."""
    torch = _torch()
    n = len(tensors)
    known = {torch.bfloat16: 0, torch.float32: 1}
    try:
        codes = [known[t.dtype] for t in tensors]
        good = ({t.get_device() for t in tensors} <= {torch.cuda.current_device()}
                and False not in {t.is_contiguous() for t in tensors})
    except (AttributeError, KeyError, RuntimeError, AssertionError):
        good = False
    if not good:
        for i, t in enumerate(tensors):
            _need(t, getattr(t, "dtype", None), f"tensors[{i}]")
            _dtype_code(t, f"tensors[{i}]")
        codes = [known[t.dtype] for t in tensors]
    return (n, (ctypes.c_void_p * n)(*[t.data_ptr() for t in tensors]),
            (ctypes.c_int64 * n)(*[t.numel() for t in tensors]), (ctypes.c_int * n)(*codes))


def _norm_buffers(n, device):
    torch = _torch()
    nws = mx_grad_norm_workspace_size(n)
    norm = torch.empty((), dtype=torch.float32, device=device)
    ws = torch.empty(nws, dtype=torch.uint8, device=device) if nws else None
    return norm, ws, nws


def grad_norm(tensors):
    """L2 norm of all elements of a list of BF16 and FP32 tensors, as a 0-d
    FP32 tensor on the device."""
    tensors = list(tensors)
    n, ptrs, sizes, codes = _tensor_list(tensors)
    device = tensors[0].device if tensors else _torch().device("cuda")
    norm, ws, nws = _norm_buffers(n, device)
    _check(mx_grad_norm(n, ptrs, sizes, codes, _ptr(norm), _ptr(ws), nws, _stream(device)))
    return norm


def grad_clip(tensors, max_norm: float):
    """Scale a list of BF16 and FP32 tensors in place by min(1, max_norm /
    (norm + 1e-6)), norm their global L2 norm; returns the norm before, as a
    0-d FP32 tensor on the device.  Tensors of the list must not overlap."""
    tensors = list(tensors)
    n, ptrs, sizes, codes = _tensor_list(tensors)
    device = tensors[0].device if tensors else _torch().device("cuda")
    norm, ws, nws = _norm_buffers(n, device)
    _check(mx_grad_clip(n, ptrs, sizes, codes, max_norm, _ptr(norm), _ptr(ws), nws, _stream(device)))
    _written(tensors)
    return norm


# ---------------------------------------------------------------------------
# 4-bit weights and 8-bit activation checkpoints
# ---------------------------------------------------------------------------

def _elem(name, known):
    if name not in known:
        raise ValueError(f"unknown element type {name!r}; expected one of {list(known)}")
    return known[name]


def _needs(dtype, ndim, *named):
    """``_need`` of several (tensor, name) pairs of one type and rank: the
    properties are swept first, and the one at fault is looked for only once
    there is one (a call of a few microseconds has no time for more)."""
    try:
        here = _torch().cuda.current_device()
        for t, _ in named:
            if not (t.dtype is dtype and t.dim() == ndim and t.get_device() == here
                    and t.is_contiguous()):
                break
        else:
            return
    except (AttributeError, RuntimeError, AssertionError):
        pass
    for t, name in named:
        _need(t, dtype, name, ndim)


def _out(out, shape, device):
    """(result tensor, whether the caller gave it) of a BF16 product."""
    torch = _torch()
    if out is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=device), False
    _need(out, torch.bfloat16, "out", len(shape))
    _shape(out, shape, "out")
    return out, True


def quant4(x, mode: str = "row"):
    """Dynamic MX quantisation of a BF16 [rows, cols] tensor, or of a stack
    [B, rows, cols], to 4 bits (E2M1, two codes to a byte, element 2i in the
    low half of byte i).

    mode "row"  -> (q [rows, cols/2], s [rows, cols/32])
         "col"  -> (q_t [cols, rows/2], s_t [cols, rows/32])
         "dual" -> (q, s, q_t, s_t)
    each with a leading B for a stack.
    """
    torch = _torch()
    if mode not in QUANT_MODES or mode == "32x32":
        raise ValueError(f"unknown 4-bit quantisation mode {mode!r}; expected 'row', 'col' or 'dual'")
    _need(x, torch.bfloat16, "x")
    if x.dim() not in (2, 3):
        raise ValueError(f"x must have 2 or 3 dims, got {x.dim()}")
    R, C = x.shape[-2:]
    lead = tuple(x.shape[:-2])
    q = s = qt = st = None
    if mode != "col":
        q = torch.empty(lead + (R, C // 2), dtype=torch.uint8, device=x.device)
        s = torch.empty(lead + (R, C // 32), dtype=torch.uint8, device=x.device)
    if mode != "row":
        qt = torch.empty(lead + (C, R // 2), dtype=torch.uint8, device=x.device)
        st = torch.empty(lead + (C, R // 32), dtype=torch.uint8, device=x.device)
    _check(mx_quant4(QUANT_MODES[mode], _ptr(x), lead[0] if lead else 1, R, C, _ptr(q), _ptr(s),
                     _ptr(qt), _ptr(st), _stream(x.device)))
    if mode == "row":
        return q, s
    return (qt, st) if mode == "col" else (q, s, qt, st)


def dequant(q, s, elem: str = "e4m3"):
    """An MX tensor in row blocks back to BF16 [..., cols]: q u8 [..., cols]
    ("e4m3", "e5m2") or [..., cols/2] ("e2m1"), s u8 [..., cols/32]."""
    torch = _torch()
    code = _elem(elem, OPERAND_ELEMS)
    _need(q, torch.uint8, "q")
    _need(s, torch.uint8, "s")
    if q.dim() < 1:
        raise ValueError("q must have at least one dim")
    lead = tuple(q.shape[:-1])
    C = q.shape[-1] * (2 if elem == "e2m1" else 1)
    if C % 32 == 0:
        _shape(s, lead + (C // 32,), "s")
    y = torch.empty(lead + (C,), dtype=torch.bfloat16, device=q.device)
    rows = 1
    for d in lead:
        rows *= d
    _check(mx_dequant(code, _ptr(q), _ptr(s), rows, C, _ptr(y), _stream(q.device)))
    return y


def gemm4(a, sa, b, sb, a_elem: str = "e4m3", out=None):
    """Product with a 4-bit weight, C = A * B^T (FP32 accumulation, BF16
    result): a u8 [M, K] ("e4m3", "e5m2") or [M, K/2] ("e2m1") with sa [M,
    K/32], b u8 [N, K/2] with sb [N, K/32], both as ``quant4`` lays them out.
    For the forward pass b is the weight's row blocks, for the input's
    gradient its column blocks.  out may share no memory with the operands."""
    torch = _torch()
    code = _elem(a_elem, OPERAND_ELEMS)
    _needs(torch.uint8, 2, (a, "a"), (sa, "sa"), (b, "b"), (sb, "sb"))
    M, K = a.shape
    N = b.shape[0]
    if a_elem == "e2m1":
        K *= 2
    if K % 32 == 0:
        _shape(sa, (M, K // 32), "sa")
        _shape(b, (N, K // 2), "b")
        _shape(sb, (N, K // 32), "sb")
    out, given = _out(out, (M, N), a.device)
    nws = mx_gemm4_workspace_size(code, M, N, K)
    ws = torch.empty(nws, dtype=torch.uint8, device=a.device) if nws else None
    _check(mx_gemm4(code, M, N, K, _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(out), _ptr(ws), nws,
                    _stream(a.device)))
    if given:
        _written(out)
    return out


def grouped_gemm4(offsets, a, sa, b, sb, a_elem: str = "e4m3", out=None):
    """``gemm4`` over per-expert token groups: rows offsets[g]:offsets[g+1] of
    a times b[g]^T, b u8 [G, N, K/2] with sb [G, N, K/32]; offsets int64 [G+1]
    on the device.  Returns BF16 [T, N]; rows from offsets[G] on are not
    written."""
    torch = _torch()
    code = _elem(a_elem, OPERAND_ELEMS)
    _need(offsets, torch.int64, "offsets", 1)
    _needs(torch.uint8, 2, (a, "a"), (sa, "sa"))
    _needs(torch.uint8, 3, (b, "b"), (sb, "sb"))
    G, T, N = offsets.numel() - 1, a.shape[0], b.shape[1]
    K = a.shape[1] * (2 if a_elem == "e2m1" else 1)
    if G < 1:
        raise ValueError("offsets must hold at least two entries (one group)")
    if K % 32 == 0:
        _shape(sa, (T, K // 32), "sa")
        _shape(b, (G, N, K // 2), "b")
        _shape(sb, (G, N, K // 32), "sb")
    out, given = _out(out, (T, N), a.device)
    _check(mx_grouped_gemm4(code, G, _ptr(offsets), T, N, K, _ptr(a), _ptr(sa), _ptr(b), _ptr(sb),
                            _ptr(out), _stream(a.device)))
    if given:
        _written(out)
    return out


def swiglu_quant(gate_up, elem: str = "e4m3", checkpoint: bool = True, checkpoint_elem: str = "e4m3"):
    """SwiGLU between an MLP's two products: gate_up BF16 [T, 2F] (gates
    first) -> (q u8 [T, F], s u8 [T, F/32], ckpt), h = silu(gate) * up in row
    blocks, the bytes of ``quant(h, "row", elem)`` for h rounded to BF16.
    ckpt is gate_up itself in 8 bits, (u8 [T, 2F], u8 [T, 2F/32]), for
    ``swiglu_backward``; None with checkpoint=False."""
    torch = _torch()
    code, ckpt_code = _elem(elem, ELEM_TYPES), _elem(checkpoint_elem, ELEM_TYPES)
    _needs(torch.bfloat16, 2, (gate_up, "gate_up"))
    T, F2 = gate_up.shape
    if F2 % 2:
        raise ValueError(f"gate_up must have an even number of columns, got {F2}")
    u8, dev = torch.uint8, gate_up.device
    q = torch.empty((T, F2 // 2), dtype=u8, device=dev)
    s = torch.empty((T, F2 // 64), dtype=u8, device=dev)
    cq = torch.empty((T, F2), dtype=u8, device=dev) if checkpoint else None
    cs = torch.empty((T, F2 // 32), dtype=u8, device=dev) if checkpoint else None
    _check(mx_swiglu_quant(code, ckpt_code, _ptr(gate_up), T, F2 // 2, _ptr(q), _ptr(s),
                           _ptr(cq) if checkpoint and T else None,
                           _ptr(cs) if checkpoint and T else None, _stream(dev)))
    return q, s, ((cq, cs) if checkpoint else None)


def _swiglu_operands(dh, ckpt_q, ckpt_s):
    torch = _torch()
    _needs(torch.bfloat16, 2, (dh, "dh"))
    _needs(torch.uint8, 2, (ckpt_q, "ckpt_q"), (ckpt_s, "ckpt_s"))
    T, F = dh.shape
    _shape(ckpt_q, (T, 2 * F), "ckpt_q")
    if F % 32 == 0:
        _shape(ckpt_s, (T, F // 16), "ckpt_s")
    return T, F


def swiglu_backward(dh, ckpt_q, ckpt_s, checkpoint_elem: str = "e4m3"):
    """Gradient of the SwiGLU at the gate_up that the 8-bit checkpoint holds:
    dh BF16 [T, F] -> d gate_up BF16 [T, 2F]."""
    torch = _torch()
    code = _elem(checkpoint_elem, ELEM_TYPES)
    T, F = _swiglu_operands(dh, ckpt_q, ckpt_s)
    dx = torch.empty((T, 2 * F), dtype=torch.bfloat16, device=dh.device)
    _check(mx_swiglu_backward(code, _ptr(dh), _ptr(ckpt_q), _ptr(ckpt_s), T, F, _ptr(dx),
                              _stream(dh.device)))
    return dx


def swiglu_backward_quant(dh, ckpt_q, ckpt_s, elem: str = "e4m3", checkpoint_elem: str = "e4m3"):
    """``quant(swiglu_backward(...), "row", elem)`` in one pass: (q u8 [T, 2F],
    s u8 [T, 2F/32]), the operand of the input's gradient, and of
    ``requant_grouped_col`` for the weight's."""
    torch = _torch()
    code, ckpt_code = _elem(elem, ELEM_TYPES), _elem(checkpoint_elem, ELEM_TYPES)
    T, F = _swiglu_operands(dh, ckpt_q, ckpt_s)
    q = torch.empty((T, 2 * F), dtype=torch.uint8, device=dh.device)
    s = torch.empty((T, F // 16), dtype=torch.uint8, device=dh.device)
    _check(mx_swiglu_backward_quant(ckpt_code, code, _ptr(dh), _ptr(ckpt_q), _ptr(ckpt_s), T, F,
                                    _ptr(q), _ptr(s), _stream(dh.device)))
    return q, s


def requant_col(q, s, elem: str = "e4m3", out_elem: str = "e4m3"):
    """``quant(dequant(q, s, elem), "col", out_elem)`` in one pass over the
    8-bit data: a forward product's operand (row blocks), kept as the
    checkpoint, as the weight gradient's (q_t u8 [cols, rows], s_t u8 [cols,
    rows/32])."""
    torch = _torch()
    code, out_code = _elem(elem, ELEM_TYPES), _elem(out_elem, ELEM_TYPES)
    _needs(torch.uint8, 2, (q, "q"), (s, "s"))
    R, C = q.shape
    if C % 32 == 0:
        _shape(s, (R, C // 32), "s")
    qt = torch.empty((C, R), dtype=torch.uint8, device=q.device)
    st = torch.empty((C, R // 32), dtype=torch.uint8, device=q.device)
    _check(mx_requant_col(code, out_code, _ptr(q), _ptr(s), R, C, _ptr(qt), _ptr(st),
                          _stream(q.device)))
    return qt, st


def requant_grouped_col(q, s, offsets, elem: str = "e4m3", out_elem: str = "e4m3"):
    """``quant_grouped_col(dequant(q, s, elem), offsets, out_elem)`` in one
    pass over the 8-bit data: q u8 [T, C], s u8 [T, C/32], offsets int64 [G+1]
    on the device -> (q_t u8 [C, cap], s_t u8 [C, cap/32])."""
    torch = _torch()
    code, out_code = _elem(elem, ELEM_TYPES), _elem(out_elem, ELEM_TYPES)
    _needs(torch.uint8, 2, (q, "q"), (s, "s"))
    _need(offsets, torch.int64, "offsets", 1)
    T, C = q.shape
    if C % 32 == 0:
        _shape(s, (T, C // 32), "s")
    G = offsets.numel() - 1
    cap = grouped_col_capacity(T, G)
    qt = torch.empty((C, cap), dtype=torch.uint8, device=q.device)
    st = torch.empty((C, cap // 32), dtype=torch.uint8, device=q.device)
    _check(mx_requant_grouped_col(code, out_code, _ptr(q), _ptr(s), T, C, G, _ptr(offsets), _ptr(qt),
                                  _ptr(st), _stream(q.device)))
    return qt, st
