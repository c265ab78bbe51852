"""ctypes binding of libmxq.so, the sm_103a MX quantized-training library.

Argument marshalling only: every operation runs in the CUDA library.  torch
is used to allocate device memory and to name the current stream.  If the
library has not been built, every call raises -- there is no CPU fallback.

Low-level functions keep the C names (``mxq_quantize`` ...) and take raw
pointers; the tensor-level helpers follow the names of the method's
statement: ``mx_quantize``, ``hadamard_mx_quantize``, ``mx_quantize_dual``,
``mx_quantize_ablation``, ``mx_dequantize``, ``mx_gemm``, ``mx_gemm_quantize``.
The FP8 recipe with one fp32 scale per block of 128 has ``fp8_quantize``,
``fp8_quantize_dual``, ``fp8_quantize_tiles`` and ``fp8_gemm``; the norms in
front of it ``layer_norm``, ``rms_norm``, their ``_quantize`` and
``_backward`` forms.  Layers of experts have ``expert_order``, ``expert_gather``,
``expert_combine``, ``expert_combine_backward``, ``mx_gemm_experts`` and
``mx_gemm_experts_wgrad``; the optimizer's update ``adamw_state``, ``adamw_plan``
and ``adamw_step``.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import struct
import threading
from bisect import bisect_left, bisect_right
from itertools import repeat

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# MXQ_BOUNDS_CHECKED=1 selects the bounds-checked build of the same library
# (every kernel checks the global indices it computes and reports
# MXQ_ERR_BOUNDS through mxq_check instead of accessing out of range)
BOUNDS_CHECKED = os.environ.get("MXQ_BOUNDS_CHECKED", "0") == "1"
LIB_PATH = os.path.join(_HERE, "_lib", "libmxq_debug.so" if BOUNDS_CHECKED else "libmxq.so")

E4M3, E2M1, E5M2 = 0, 1, 2
ROWWISE, COLWISE_T = 0, 1
SCALES_ROWMAJOR, SCALES_TC = 0, 1
SCALE_LAYOUTS = {"rowmajor": SCALES_ROWMAJOR, "tc": SCALES_TC,
                 SCALES_ROWMAJOR: SCALES_ROWMAJOR, SCALES_TC: SCALES_TC}
OUT_F32, OUT_BF16 = 0, 1
FP8_LINES, FP8_TILES = 0, 1
B_SCALES = {"line": FP8_LINES, "tile": FP8_TILES, FP8_LINES: FP8_LINES, FP8_TILES: FP8_TILES}
FP8_FMTS = {"e4m3": E4M3, "e5m2": E5M2, E4M3: E4M3, E5M2: E5M2}
NORM_LAYER, NORM_RMS = 0, 1
FMTS = {"e4m3": E4M3, "e2m1": E2M1, "e5m2": E5M2, E4M3: E4M3, E2M1: E2M1, E5M2: E5M2}
AXES = {"row": ROWWISE, "col": COLWISE_T, ROWWISE: ROWWISE, COLWISE_T: COLWISE_T}

STATUS = {0: "MXQ_OK", 1: "MXQ_ERR_ARG", 2: "MXQ_ERR_ALIGN", 3: "MXQ_ERR_UNSUPPORTED",
          4: "MXQ_ERR_CUDA", 5: "MXQ_ERR_TIMEOUT", 6: "MXQ_ERR_WORKSPACE",
          7: "MXQ_ERR_BOUNDS"}

# C signatures: (name, restype, argtypes)
_I64, _P, _I, _SZ, _U64 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64
SIGNATURES = [
    ("mxq_version", ctypes.c_int, []),
    ("mxq_status_str", ctypes.c_char_p, [_I]),
    ("mxq_quantize", _I, [_P, _I64, _I64, _I, _I, _P, _P, _P]),
    ("mxq_hadamard_quantize", _I, [_P, _I64, _I64, _I, _I, _P, _P, _P]),
    ("mxq_quantize_dual", _I, [_P, _I64, _I64, _I, _I, _P, _P, _I, _I, _P, _P, _P]),
    ("mxq_quantize_ex", _I, [_P, _I64, _I64, _I, _I, _I, _P, _P, _I, _P]),
    ("mxq_quantize_dual_ex", _I, [_P, _I64, _I64, _I, _I, _P, _P, _I, _I, _P, _P, _I, _P]),
    ("mxq_scales_tc_bytes", _SZ, [_I64, _I64]),
    ("mxq_gemm_ex", _I, [_P, _P, _P, _P, _I, _I64, _I64, _I64, _P, _I, _I, _P, _SZ, _P]),
    ("mxq_quantize_ablation", _I, [_P, _I64, _I64, _I, _I, _I, ctypes.c_uint32, _I, _U64, _P, _P, _P]),
    ("mxq_dequantize", _I, [_P, _P, _I64, _I64, _I, _I, _P, _I, _P]),
    ("mxq_gemm", _I, [_P, _P, _P, _P, _I, _I64, _I64, _I64, _P, _I, _P, _SZ, _P]),
    ("mxq_gemm_quantize", _I, [_P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _P, _P, _P, _SZ, _P]),
    ("mxq_gemm_quantize_ex", _I, [_P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _I, _P, _P, _I, _P, _SZ,
                                  _P]),
    ("mxq_gemm_workspace_size", _SZ, [_I64, _I64, _I64, _I]),
    ("mxq_gemm_noalloc", _I, [_P, _P, _P, _P, _I, _I64, _I64, _I64, _P, _I, _P]),
    ("mxq_gemm_grouped", _I, [_P, _I, _I, _P]),
    ("mxq_fp8_pitch", _SZ, [_I64]),
    ("mxq_fp8_scale_count", _SZ, [_I64, _I64, _I]),
    ("mxq_fp8_quantize", _I, [_P, _I64, _I64, _I, _I, _P, _P, _P]),
    ("mxq_fp8_quantize_dual", _I, [_P, _I64, _I64, _I, _P, _P, _I, _P, _P, _P]),
    ("mxq_fp8_quantize_tiles", _I, [_P, _I64, _I64, _I, _P, _P, _P, _P, _P]),
    ("mxq_fp8_gemm", _I, [_P, _P, _I, _P, _P, _I, _I, _I64, _I64, _I64, _P, _I, _P]),
    ("mxq_norm_forward", _I, [_P, _P]),
    ("mxq_norm_backward", _I, [_P, _P]),
    ("mxq_norm_backward_workspace_size", _SZ, [_I64, _I64]),
    ("mxq_expert_order", _I, [_P, _I, _I64, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    ("mxq_expert_order_workspace_size", _SZ, [_I64, _I]),
    ("mxq_expert_gather", _I, [_P, _P]),
    ("mxq_expert_combine", _I, [_P, _P]),
    ("mxq_expert_combine_backward", _I, [_P, _P]),
    ("mxq_gemm_experts", _I, [_P, _P]),
    ("mxq_gemm_experts_wgrad", _I, [_P, _P]),
    ("mxq_gemm_experts_workspace_size", _SZ, [_I64, _I64, _I64, _I, _I, _I]),
    ("mxq_gemm_experts_wgrad_workspace_size", _SZ, [_I64, _I64, _I64, _I, _I]),
    ("mxq_adamw", _I, [_P, _P, _I, _P, _P]),
    ("mxq_check", _I, [_P]),
    ("mxq_set_wait_timeout_ns", None, [_U64]),
    ("mxq_debug_expire_wait", _I, [_U64, _P]),
    ("mxq_debug_fp8_gemm", _I, [_P, _P, _I, _P, _P, _I, _I, _I64, _I64, _I64, _P, _I, _I, _P]),
]

class GemmProblem(ctypes.Structure):
    """mxq_gemm_problem of the C header (field order and types as declared)."""
    _fields_ = [("A", ctypes.c_void_p), ("sA", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("sB", ctypes.c_void_p), ("C", ctypes.c_void_p), ("M", ctypes.c_int64),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("out_dtype", ctypes.c_int)]


class NormArgs(ctypes.Structure):
    """mxq_norm_args of the C header (field order and types as declared)."""
    _fields_ = [("x", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("eps", ctypes.c_float), ("kind", ctypes.c_int),
                ("x_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int), ("fmt", ctypes.c_int)]


class NormGradArgs(ctypes.Structure):
    """mxq_norm_grad_args of the C header (field order and types as declared)."""
    _fields_ = [("dy", ctypes.c_void_p), ("x", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p), ("dx", ctypes.c_void_p),
                ("dweight", ctypes.c_void_p), ("dbias", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("kind", ctypes.c_int),
                ("x_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int)]


class ExpertRowsArgs(ctypes.Structure):
    """mxq_expert_rows_args of the C header (field order and types as declared)."""
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("row_of", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("counts", ctypes.c_void_p), ("weights", ctypes.c_void_p),
                ("dweights", ctypes.c_void_p), ("tokens", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("topk", ctypes.c_int),
                ("experts", ctypes.c_int), ("dtype", ctypes.c_int)]


class ExpertsArgs(ctypes.Structure):
    """mxq_experts_args of the C header (field order and types as declared)."""
    _fields_ = [("A", ctypes.c_void_p), ("sA", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("sB", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("C", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("rows", ctypes.c_int64), ("M", ctypes.c_int64), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("experts", ctypes.c_int), ("fmt", ctypes.c_int),
                ("out_dtype", ctypes.c_int), ("b_scale_layout", ctypes.c_int)]


class AdamWTensor(ctypes.Structure):
    """mxq_adamw_tensor of the C header (field order and types as declared)."""
    _fields_ = [("param", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("r_scale", ctypes.c_void_p),
                ("copy", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("weight_decay", ctypes.c_float)]


class AdamWArgs(ctypes.Structure):
    """mxq_adamw_args of the C header (field order and types as declared)."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("lr_at", ctypes.c_void_p),
                ("step_at", ctypes.c_void_p), ("grad_scale_at", ctypes.c_void_p),
                ("grad_dtype", ctypes.c_int), ("state_bits", ctypes.c_int)]


# The same structures as native-layout formats: packing one takes a third of the
# time of filling the ctypes mirror, which small calls notice.
_NORM_ARGS = struct.Struct("@8P2qf4i0q")
_NORM_GRAD_ARGS = struct.Struct("@9PN2q3i0q")
_EXPERT_ROWS_ARGS = struct.Struct("@8P3q3i0q")
_EXPERTS_ARGS = struct.Struct("@7PN4q4i0q")
_ADAMW_TENSOR = struct.Struct("@6Pqf0q")
_ADAMW_ARGS = struct.Struct("@4dq3P2i0q")

_lib = None
_lock = threading.Lock()


class MXQError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it was never built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"libmxq.so is not built ({LIB_PATH} missing); run "
                        "precision_mx_quantize_gb300.build.build() first")
                handle = ctypes.CDLL(LIB_PATH)
                for name, res, args in SIGNATURES:
                    fn = getattr(handle, name)
                    fn.restype = res
                    fn.argtypes = args
                _lib = handle
    return _lib


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(device=None) -> int:
    """The raw handle of the current CUDA stream of `device`, which must be the
    current device (the default): handle 0 is the default stream of whichever
    device is current, and a launch there would take another device's memory.
    Uses torch's raw-handle accessors when it has them, which skip building a
    Stream object and torch's own set-up on every call."""
    if device is None:
        idx = torch.cuda.current_device()
    else:
        idx = device if isinstance(device, int) else torch.device(device).index
        if idx is None:
            idx = torch.cuda.current_device()
        elif idx != _current_device():
            raise ValueError(f"the tensors are on CUDA device {idx}, the current device is "
                             f"{_current_device()}: make the call inside torch.cuda.device({idx})")
    if _raw_stream is not None:
        return _raw_stream(idx)
    return torch.cuda.current_stream(idx).cuda_stream


def _ok(status: int, where: str):
    if status != 0:
        raise MXQError(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


# ---- raw C-ABI calls (pointers and sizes) ------------------------------------

def mxq_quantize(x, rows, cols, layout, fmt, codes, scales, stream):
    return lib().mxq_quantize(x, rows, cols, layout, fmt, codes, scales, stream)


def mxq_hadamard_quantize(x, rows, cols, layout, fmt, codes, scales, stream):
    return lib().mxq_hadamard_quantize(x, rows, cols, layout, fmt, codes, scales, stream)


def mxq_quantize_dual(x, rows, cols, fmt_r, had_r, codes_r, scales_r, fmt_c, had_c, codes_c,
                      scales_c, stream):
    return lib().mxq_quantize_dual(x, rows, cols, fmt_r, had_r, codes_r, scales_r, fmt_c, had_c,
                                   codes_c, scales_c, stream)


def mxq_quantize_ex(x, rows, cols, layout, fmt, hadamard, codes, scales, scale_layout, stream):
    return lib().mxq_quantize_ex(x, rows, cols, layout, fmt, hadamard, codes, scales, scale_layout,
                                 stream)


def mxq_quantize_dual_ex(x, rows, cols, fmt_r, had_r, codes_r, scales_r, fmt_c, had_c, codes_c,
                         scales_c, scale_layout, stream):
    return lib().mxq_quantize_dual_ex(x, rows, cols, fmt_r, had_r, codes_r, scales_r, fmt_c,
                                      had_c, codes_c, scales_c, scale_layout, stream)


def mxq_scales_tc_bytes(lines, blocked):
    return lib().mxq_scales_tc_bytes(lines, blocked)


def mxq_gemm_ex(A, sA, B, sB, fmt, M, N, K, C, out_dtype, scale_layout, workspace, ws_bytes,
                stream):
    return lib().mxq_gemm_ex(A, sA, B, sB, fmt, M, N, K, C, out_dtype, scale_layout, workspace,
                             ws_bytes, stream)


def mxq_quantize_ablation(x, rows, cols, layout, fmt, hadamard, sign_mask, stochastic, seed, codes,
                          scales, stream):
    return lib().mxq_quantize_ablation(x, rows, cols, layout, fmt, hadamard, sign_mask, stochastic,
                                       seed, codes, scales, stream)


def mxq_dequantize(codes, scales, rows, cols, layout, fmt, out, out_dtype, stream):
    return lib().mxq_dequantize(codes, scales, rows, cols, layout, fmt, out, out_dtype, stream)


def mxq_gemm(A, sA, B, sB, fmt, M, N, K, C, out_dtype, workspace, ws_bytes, stream):
    return lib().mxq_gemm(A, sA, B, sB, fmt, M, N, K, C, out_dtype, workspace, ws_bytes, stream)


def mxq_gemm_quantize(A, sA, B, sB, fmt, M, N, K, out_fmt, codes, scales, workspace, ws_bytes,
                      stream):
    return lib().mxq_gemm_quantize(A, sA, B, sB, fmt, M, N, K, out_fmt, codes, scales, workspace,
                                   ws_bytes, stream)


def mxq_gemm_quantize_ex(A, sA, B, sB, fmt, M, N, K, scale_layout, out_fmt, codes, scales,
                         out_scale_layout, workspace, ws_bytes, stream):
    return lib().mxq_gemm_quantize_ex(A, sA, B, sB, fmt, M, N, K, scale_layout, out_fmt, codes,
                                      scales, out_scale_layout, workspace, ws_bytes, stream)


def mxq_gemm_noalloc(A, sA, B, sB, fmt, M, N, K, C, out_dtype, stream):
    """mxq_gemm with the library's fixed internal scratch (for callers that cannot allocate)."""
    return lib().mxq_gemm_noalloc(A, sA, B, sB, fmt, M, N, K, C, out_dtype, stream)


def mxq_gemm_grouped(problems, count, fmt, stream):
    """problems: address of `count` GemmProblem structures in host memory."""
    return lib().mxq_gemm_grouped(problems, count, fmt, stream)


def mxq_gemm_workspace_size(M, N, K, fmt):
    return lib().mxq_gemm_workspace_size(M, N, K, fmt)


def mxq_fp8_quantize(x, rows, cols, layout, fmt, codes, scales, stream):
    return lib().mxq_fp8_quantize(x, rows, cols, layout, fmt, codes, scales, stream)


def mxq_fp8_quantize_dual(x, rows, cols, fmt_r, codes_r, scales_r, fmt_c, codes_c, scales_c,
                          stream):
    return lib().mxq_fp8_quantize_dual(x, rows, cols, fmt_r, codes_r, scales_r, fmt_c, codes_c,
                                       scales_c, stream)


def mxq_fp8_quantize_tiles(x, rows, cols, fmt, codes, scales, codes_t, scales_t, stream):
    return lib().mxq_fp8_quantize_tiles(x, rows, cols, fmt, codes, scales, codes_t, scales_t,
                                        stream)


def mxq_fp8_gemm(A, sA, fmt_a, B, sB, fmt_b, b_scales, M, N, K, C, out_dtype, stream):
    return lib().mxq_fp8_gemm(A, sA, fmt_a, B, sB, fmt_b, b_scales, M, N, K, C, out_dtype, stream)


def mxq_norm_forward(args, stream):
    """args: address of a NormArgs structure in host memory, or its bytes."""
    return lib().mxq_norm_forward(args, stream)


def mxq_norm_backward(args, stream):
    """args: address of a NormGradArgs structure in host memory, or its bytes."""
    return lib().mxq_norm_backward(args, stream)


def mxq_norm_backward_workspace_size(rows, cols):
    return lib().mxq_norm_backward_workspace_size(rows, cols)


def mxq_expert_order(ids, id_bytes, n, experts, align, row_of, offsets, counts, workspace,
                     ws_bytes, stream):
    return lib().mxq_expert_order(ids, id_bytes, n, experts, align, row_of, offsets, counts,
                                  workspace, ws_bytes, stream)


def mxq_expert_order_workspace_size(n, experts):
    return lib().mxq_expert_order_workspace_size(n, experts)


def mxq_expert_gather(args, stream):
    """args: address of an ExpertRowsArgs structure in host memory, or its bytes."""
    return lib().mxq_expert_gather(args, stream)


def mxq_expert_combine(args, stream):
    """args: as mxq_expert_gather."""
    return lib().mxq_expert_combine(args, stream)


def mxq_expert_combine_backward(args, stream):
    """args: as mxq_expert_gather."""
    return lib().mxq_expert_combine_backward(args, stream)


def mxq_gemm_experts(args, stream):
    """args: address of an ExpertsArgs structure in host memory, or its bytes."""
    return lib().mxq_gemm_experts(args, stream)


def mxq_gemm_experts_wgrad(args, stream):
    """args: as mxq_gemm_experts."""
    return lib().mxq_gemm_experts_wgrad(args, stream)


def mxq_gemm_experts_workspace_size(rows, N, K, experts, fmt, b_scale_layout):
    return lib().mxq_gemm_experts_workspace_size(rows, N, K, experts, fmt, b_scale_layout)


def mxq_gemm_experts_wgrad_workspace_size(rows, M, N, experts, fmt):
    return lib().mxq_gemm_experts_wgrad_workspace_size(rows, M, N, experts, fmt)


def mxq_adamw(tensors, grads, count, args, stream):
    """tensors: address of `count` AdamWTensor structures in host memory, or their
    bytes; grads: of as many device pointers; args: of an AdamWArgs structure."""
    return lib().mxq_adamw(tensors, grads, count, args, stream)


def mxq_check(stream=None):
    return lib().mxq_check(stream)


def check(device=None):
    """Synchronize the current stream and raise on any error recorded on the device (the
    current one, which `device` must be where it is given)."""
    _ok(mxq_check(_stream(device)), "mxq_check")


def set_wait_timeout_ns(ns: int):
    lib().mxq_set_wait_timeout_ns(int(ns))


# ---- tensor-level helpers -----------------------------------------------------

def code_shape(rows: int, cols: int, axis, fmt):
    """(codes shape, scales shape) for a [rows, cols] tensor."""
    ax, f = AXES[axis], FMTS[fmt]
    r, c = (rows, cols) if ax == ROWWISE else (cols, rows)
    return (r, c // 2 if f == E2M1 else c), (r, c // 32)


# The kernels get raw pointers and sizes: a host tensor, or a buffer shorter
# than the sizes imply, would be read or written past its end on the GPU.
# These checks run before every launch (explicit raises, not asserts, so
# that they survive python -O).

def _on_gpu(t):
    return t.is_cuda


def _need(t, name, dtype, numel, dev=None):
    """Raise unless t is a contiguous CUDA tensor of `dtype` (None: any) with
    at least `numel` elements, on device index `dev` when given.  Cheap on
    the success path (the binding runs it on every call): one combined test,
    and the detailed checks only to word the error."""
    try:
        if ((dtype is None or t.dtype is dtype) and t.numel() >= numel and t.is_contiguous()
                and _on_gpu(t) and (dev is None or t.get_device() == dev)):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements; {numel} are needed")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not _on_gpu(t):
        raise ValueError(f"{name} must be on a CUDA device (the library has no CPU path)")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on device {t.get_device()}, the inputs on {dev}")


def _need_rows(t, name, dtype, shape, dev=None):
    """The same for a tensor of the shape [rows, length], or a flat buffer of as many
    elements, or one with more rows.  Rows of another length are refused: the
    library would read them with the wrong pitch."""
    try:
        if (t.shape == shape and t.dtype is dtype and t.is_contiguous() and _on_gpu(t)
                and (dev is None or t.get_device() == dev)):
            return
    except AttributeError:
        pass
    _need(t, name, dtype, shape[0] * shape[1], dev)
    if t.dim() > 1 and t.size(-1) != shape[1]:
        raise ValueError(f"{name} has rows of {t.size(-1)} elements; they must hold {shape[1]}")


def _need_input(x):
    """x: a contiguous 2-D bf16 CUDA tensor."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D torch.Tensor [rows, cols]")
    _need(x, "x", torch.bfloat16, 0)


@functools.lru_cache(maxsize=4096)
def _buffer_sizes(rows, cols, axis, fmt, scale_layout):
    """(code bytes, scale bytes) of a [rows, cols] tensor quantized along
    `axis`, with its scales in `scale_layout`."""
    cs, _ = code_shape(rows, cols, axis, fmt)
    lines, blocked = (rows, cols) if AXES[axis] == ROWWISE else (cols, rows)
    if SCALE_LAYOUTS[scale_layout] == SCALES_TC:
        n = int(mxq_scales_tc_bytes(lines, blocked))
        if n == 0:
            raise ValueError(f"no tensor-core scale layout for {lines} lines x {blocked}")
    else:
        n = lines * (blocked // 32)
    return cs[0] * cs[1], n


def _need_codes(codes, scales, rows, cols, axis, fmt, scale_layout, dev, tag=""):
    """The code and scale buffers of a [rows, cols] tensor quantized along `axis`."""
    nc, ns = _buffer_sizes(int(rows), int(cols), axis, fmt, scale_layout)
    _need(codes, "codes" + tag, torch.uint8, nc, dev)
    _need(scales, "scales" + tag, torch.uint8, ns, dev)


def _out_code(out_dtype):
    if out_dtype is torch.float32:
        return OUT_F32
    if out_dtype is torch.bfloat16:
        return OUT_BF16
    raise ValueError(f"out_dtype must be torch.float32 or torch.bfloat16, got {out_dtype}")


def _need_operands(A, sA, B, sB, fmt, M, N, K, scale_layout):
    """GEMM operands: K-major codes of A [M, K] and B [N, K] and their scales.
    Returns the device index of A."""
    _need(A, "A", torch.uint8, 0)
    dev = A.get_device()
    _need_codes(A, sA, M, K, "row", fmt, scale_layout, dev, "_A")
    _need_codes(B, sB, N, K, "row", fmt, scale_layout, dev, "_B")
    return dev


def _alloc_codes(x, axis, fmt, scale_layout="rowmajor"):
    cs, ss = code_shape(x.shape[0], x.shape[1], axis, fmt)
    if SCALE_LAYOUTS[scale_layout] == SCALES_TC:
        lines, blocked = (x.shape[0], x.shape[1]) if AXES[axis] == ROWWISE else (x.shape[1], x.shape[0])
        n = mxq_scales_tc_bytes(lines, blocked)
        if n == 0:
            raise ValueError(f"no tensor-core scale layout for {lines} lines x {blocked}")
        ss = (n,)
    return (torch.empty(cs, dtype=torch.uint8, device=x.device),
            torch.empty(ss, dtype=torch.uint8, device=x.device))


def mx_quantize(x: torch.Tensor, axis="row", fmt="e4m3", out=None, scale_layout="rowmajor"):
    """MX-quantize a contiguous bf16 CUDA tensor [rows, cols]; returns (codes, scales).

    scale_layout "tc": scales in the tensor cores' chunk layout (a flat byte
    tensor), which mx_gemm(..., scale_layout="tc") reads in place."""
    _need_input(x)
    codes, scales = out if out is not None else _alloc_codes(x, axis, fmt, scale_layout)
    R, C = x.shape
    dev = x.get_device()
    _need_codes(codes, scales, R, C, axis, fmt, scale_layout, dev)
    if SCALE_LAYOUTS[scale_layout] == SCALES_ROWMAJOR:
        _ok(mxq_quantize(x.data_ptr(), R, C, AXES[axis], FMTS[fmt], codes.data_ptr(),
                         scales.data_ptr(), _stream(dev)), "mxq_quantize")
    else:
        _ok(mxq_quantize_ex(x.data_ptr(), R, C, AXES[axis], FMTS[fmt], 0, codes.data_ptr(),
                            scales.data_ptr(), SCALES_TC, _stream(dev)), "mxq_quantize_ex")
    return codes, scales


def hadamard_mx_quantize(x: torch.Tensor, axis="col", fmt="e2m1", out=None,
                         scale_layout="rowmajor"):
    """Fixed 32-point Hadamard rotation of each block, then MX quantization."""
    _need_input(x)
    codes, scales = out if out is not None else _alloc_codes(x, axis, fmt, scale_layout)
    R, C = x.shape
    dev = x.get_device()
    _need_codes(codes, scales, R, C, axis, fmt, scale_layout, dev)
    if SCALE_LAYOUTS[scale_layout] == SCALES_ROWMAJOR:
        _ok(mxq_hadamard_quantize(x.data_ptr(), R, C, AXES[axis], FMTS[fmt], codes.data_ptr(),
                                  scales.data_ptr(), _stream(dev)), "mxq_hadamard_quantize")
    else:
        _ok(mxq_quantize_ex(x.data_ptr(), R, C, AXES[axis], FMTS[fmt], 1, codes.data_ptr(),
                            scales.data_ptr(), SCALES_TC, _stream(dev)), "mxq_quantize_ex")
    return codes, scales


def mx_quantize_dual(x: torch.Tensor, fmt_r="e4m3", had_r=False, fmt_c="e2m1", had_c=True,
                     out=None, scale_layout="rowmajor"):
    """One pass producing the row-wise and the column-wise (transposed) outputs."""
    _need_input(x)
    if out is None:
        cr, sr = _alloc_codes(x, "row", fmt_r, scale_layout)
        cc, sc = _alloc_codes(x, "col", fmt_c, scale_layout)
    else:
        cr, sr, cc, sc = out
    _need_codes(cr, sr, x.shape[0], x.shape[1], "row", fmt_r, scale_layout, x.get_device(), "_r")
    _need_codes(cc, sc, x.shape[0], x.shape[1], "col", fmt_c, scale_layout, x.get_device(), "_c")
    if SCALE_LAYOUTS[scale_layout] == SCALES_ROWMAJOR:
        _ok(mxq_quantize_dual(x.data_ptr(), x.shape[0], x.shape[1], FMTS[fmt_r], int(had_r),
                              cr.data_ptr(), sr.data_ptr(), FMTS[fmt_c], int(had_c), cc.data_ptr(),
                              sc.data_ptr(), _stream(x.get_device())), "mxq_quantize_dual")
    else:
        _ok(mxq_quantize_dual_ex(x.data_ptr(), x.shape[0], x.shape[1], FMTS[fmt_r], int(had_r),
                                 cr.data_ptr(), sr.data_ptr(), FMTS[fmt_c], int(had_c),
                                 cc.data_ptr(), sc.data_ptr(), SCALES_TC, _stream(x.get_device())),
            "mxq_quantize_dual_ex")
    return cr, sr, cc, sc


def mx_quantize_ablation(x: torch.Tensor, axis="col", fmt="e2m1", hadamard=True, sign_mask=0,
                         stochastic=False, seed=0, out=None):
    """MX quantization with a random-sign Hadamard rotation (sign_mask) and/or
    stochastic rounding (Philox bits keyed by seed); the ablation of the
    deterministic path."""
    _need_input(x)
    codes, scales = out if out is not None else _alloc_codes(x, axis, fmt)
    _need_codes(codes, scales, x.shape[0], x.shape[1], axis, fmt, "rowmajor", x.get_device())
    _ok(mxq_quantize_ablation(x.data_ptr(), x.shape[0], x.shape[1], AXES[axis], FMTS[fmt],
                              int(hadamard), int(sign_mask) & 0xFFFFFFFF, int(stochastic),
                              int(seed) & 0xFFFFFFFFFFFFFFFF, codes.data_ptr(), scales.data_ptr(),
                              _stream(x.get_device())), "mxq_quantize_ablation")
    return codes, scales


def mx_dequantize(codes, scales, rows, cols, axis="row", fmt="e4m3", out_dtype=torch.float32,
                  out=None):
    """Dequantize codes written by mx_quantize back to a [rows, cols] tensor."""
    od = _out_code(out_dtype)
    _need(codes, "codes", torch.uint8, 0)
    dev = codes.get_device()
    _need_codes(codes, scales, rows, cols, axis, fmt, "rowmajor", dev)
    if out is None:
        out = torch.empty((rows, cols), dtype=out_dtype, device=codes.device)
    _need(out, "out", out_dtype, rows * cols, dev)
    _ok(mxq_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, AXES[axis], FMTS[fmt],
                       out.data_ptr(), od, _stream(dev)), "mxq_dequantize")
    return out


def gemm_workspace(M, N, K, fmt, device):
    n = mxq_gemm_workspace_size(M, N, K, FMTS[fmt])
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device=device)


def mx_gemm(A, sA, B, sB, fmt, M, N, K, out_dtype=torch.float32, out=None, workspace=None,
            scale_layout="rowmajor"):
    """C[M, N] = dec(A) @ dec(B)^T on the tensor cores (A, B K-major MX codes).

    scale_layout "tc": sA, sB in the tensor cores' chunk layout (no workspace)."""
    od = _out_code(out_dtype)
    dev = _need_operands(A, sA, B, sB, fmt, M, N, K, scale_layout)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A.device)
    _need(out, "out", out_dtype, M * N, dev)
    if SCALE_LAYOUTS[scale_layout] == SCALES_TC:
        _ok(mxq_gemm_ex(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(), FMTS[fmt], M, N,
                        K, out.data_ptr(), od, SCALES_TC, None, 0, _stream(A.get_device())),
            "mxq_gemm_ex")
        return out
    if workspace is None:
        workspace = gemm_workspace(M, N, K, fmt, A.device)
    _need(workspace, "workspace", torch.uint8, 0, dev)   # its size is checked by the library
    _ok(mxq_gemm(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(), FMTS[fmt], M, N, K,
                 out.data_ptr(), od, workspace.data_ptr(), workspace.numel(),
                 _stream(A.get_device())), "mxq_gemm")
    return out


def mx_gemm_grouped(problems, fmt, out_dtype=torch.float32):
    """Independent GEMMs of one format in one launch (see mxq_gemm_grouped).

    problems: list of (A, sA, B, sB, M, N, K) or (A, sA, B, sB, M, N, K, out),
    with the scales in the tensor cores' chunk layout (as returned by the
    quantizers with scale_layout="tc").  Returns the list of outputs C, each
    bitwise what mx_gemm(..., scale_layout="tc") would return."""
    if not 1 <= len(problems) <= 8:
        raise ValueError("mx_gemm_grouped takes 1 to 8 problems")
    od = _out_code(out_dtype)
    arr = (GemmProblem * len(problems))()
    outs = []
    dev = None
    for i, pr in enumerate(problems):
        A, sA, B, sB, M, N, K = pr[:7]
        d = _need_operands(A, sA, B, sB, fmt, M, N, K, "tc")
        if dev is None:
            dev = d
        elif d != dev:
            raise ValueError(f"problem {i} is on device {d}, problem 0 on {dev}")
        out = pr[7] if len(pr) > 7 else torch.empty((M, N), dtype=out_dtype, device=A.device)
        _need(out, f"out[{i}]", out_dtype, M * N, dev)
        arr[i] = GemmProblem(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(),
                             out.data_ptr(), M, N, K, od)
        outs.append(out)
    _ok(mxq_gemm_grouped(ctypes.addressof(arr), len(problems), FMTS[fmt], _stream(dev)),
        "mxq_gemm_grouped")
    return outs


def mx_gemm_quantize(A, sA, B, sB, fmt, M, N, K, out_fmt="e4m3", out=None, workspace=None,
                     scale_layout="rowmajor", out_scale_layout="rowmajor"):
    """dec(A) @ dec(B)^T with the epilogue writing row-wise MX codes of the
    fp32 product (blocks of 32 along N); returns (codes, scales)."""
    in_tc = SCALE_LAYOUTS[scale_layout] == SCALES_TC
    out_tc = SCALE_LAYOUTS[out_scale_layout] == SCALES_TC
    dev = _need_operands(A, sA, B, sB, fmt, M, N, K, scale_layout)
    if out is None:
        cs, ss = code_shape(M, N, "row", out_fmt)
        if out_tc:
            ss = (mxq_scales_tc_bytes(M, N),)
        out = (torch.empty(cs, dtype=torch.uint8, device=A.device),
               torch.empty(ss, dtype=torch.uint8, device=A.device))
    codes, scales = out
    _need_codes(codes, scales, M, N, "row", out_fmt, out_scale_layout, dev, "_out")
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, 0, dev)
    if not in_tc and not out_tc:
        if workspace is None:
            workspace = gemm_workspace(M, N, K, fmt, A.device)
        _ok(mxq_gemm_quantize(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(), FMTS[fmt], M,
                              N, K, FMTS[out_fmt], codes.data_ptr(), scales.data_ptr(),
                              workspace.data_ptr(), workspace.numel(), _stream(A.get_device())),
            "mxq_gemm_quantize")
        return codes, scales
    if not in_tc and workspace is None:
        workspace = gemm_workspace(M, N, K, fmt, A.device)
    ws_ptr, ws_n = (None, 0) if in_tc else (workspace.data_ptr(), workspace.numel())
    _ok(mxq_gemm_quantize_ex(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(), FMTS[fmt], M,
                             N, K, SCALE_LAYOUTS[scale_layout], FMTS[out_fmt], codes.data_ptr(),
                             scales.data_ptr(), SCALE_LAYOUTS[out_scale_layout], ws_ptr, ws_n,
                             _stream(A.get_device())), "mxq_gemm_quantize_ex")
    return codes, scales


# ---- FP8 with one fp32 scale per block of 128 ---------------------------------------

@functools.lru_cache(maxsize=4096)
def fp8_shapes(lines: int, blocked: int, scales="line"):
    """(codes shape, scales shape) of `lines` code lines of `blocked` elements:
    a line's pitch is `blocked` rounded up to 16; line scales are [ceil(blocked
    / 128)][lines rounded up to 4], tile scales [ceil(lines / 128)][ceil(blocked
    / 128)]."""
    kb = (blocked + 127) // 128
    ss = (kb, (lines + 3) // 4 * 4) if B_SCALES[scales] == FP8_LINES else ((lines + 127) // 128, kb)
    return (lines, (blocked + 15) // 16 * 16), ss


def _fp8_buffers(lines, blocked, scales, device):
    cs, ss = fp8_shapes(lines, blocked, scales)
    return (torch.empty(cs, dtype=torch.uint8, device=device),
            torch.empty(ss, dtype=torch.float32, device=device))


def _need_fp8(codes, scales, lines, blocked, kind, dev, tag=""):
    """The code and scale buffers of `lines` lines of `blocked` elements: shaped as
    fp8_shapes says (more lines of codes may follow), or flat."""
    cs, ss = fp8_shapes(lines, blocked, kind)
    _need_rows(codes, "codes" + tag, torch.uint8, cs, dev)
    _need_rows(scales, "scales" + tag, torch.float32, ss, dev)


def fp8_quantize(x: torch.Tensor, axis="row", fmt="e4m3", out=None):
    """FP8 codes of a contiguous bf16 CUDA tensor [rows, cols] with one fp32
    scale per 1x128 block along `axis` ("col": stored transposed); returns
    (codes, scales), shaped as fp8_shapes says."""
    _need_input(x)
    R, C = x.shape
    ax, f = AXES[axis], FP8_FMTS[fmt]
    lines, blocked = (R, C) if ax == ROWWISE else (C, R)
    dev = x.get_device()
    if out is None:
        codes, scales = _fp8_buffers(lines, blocked, "line", x.device)
    else:
        codes, scales = out
        _need_fp8(codes, scales, lines, blocked, "line", dev)
    _ok(mxq_fp8_quantize(x.data_ptr(), R, C, ax, f, codes.data_ptr(), scales.data_ptr(),
                         _stream(dev)), "mxq_fp8_quantize")
    return codes, scales


def fp8_quantize_dual(x: torch.Tensor, fmt_r="e4m3", fmt_c="e4m3", out=None):
    """Both layouts of fp8_quantize from one read of x; returns (codes_r,
    scales_r, codes_c, scales_c)."""
    _need_input(x)
    R, C = x.shape
    fr, fc = FP8_FMTS[fmt_r], FP8_FMTS[fmt_c]
    dev = x.get_device()
    if out is None:
        cr, sr = _fp8_buffers(R, C, "line", x.device)
        cc, sc = _fp8_buffers(C, R, "line", x.device)
    else:
        cr, sr, cc, sc = out
        _need_fp8(cr, sr, R, C, "line", dev, "_r")
        _need_fp8(cc, sc, C, R, "line", dev, "_c")
    _ok(mxq_fp8_quantize_dual(x.data_ptr(), R, C, fr, cr.data_ptr(), sr.data_ptr(), fc,
                              cc.data_ptr(), sc.data_ptr(), _stream(dev)), "mxq_fp8_quantize_dual")
    return cr, sr, cc, sc


def fp8_quantize_tiles(w: torch.Tensor, fmt="e4m3", out=None):
    """FP8 codes of a bf16 weight [rows, cols] with one fp32 scale per 128x128
    tile, and the transposed codes and scales; returns (codes, scales, codes_t,
    scales_t).  In `out`, codes_t and scales_t may be None: not written."""
    _need_input(w)
    R, C = w.shape
    f = FP8_FMTS[fmt]
    dev = w.get_device()
    if out is None:
        codes, scales = _fp8_buffers(R, C, "tile", w.device)
        codes_t, scales_t = _fp8_buffers(C, R, "tile", w.device)
    else:
        codes, scales, codes_t, scales_t = out
        _need_fp8(codes, scales, R, C, "tile", dev)
        if codes_t is not None or scales_t is not None:
            _need_fp8(codes_t, scales_t, C, R, "tile", dev, "_t")
    _ok(mxq_fp8_quantize_tiles(w.data_ptr(), R, C, f, codes.data_ptr(), scales.data_ptr(),
                               _ptr(codes_t), _ptr(scales_t), _stream(dev)),
        "mxq_fp8_quantize_tiles")
    return codes, scales, codes_t, scales_t


def fp8_gemm(A, sA, B, sB, M, N, K, fmt_a="e4m3", fmt_b="e4m3", b_scales="tile",
             out_dtype=torch.bfloat16, out=None):
    """C[M, N] = dec(A) @ dec(B)^T of block-128 FP8 codes (K-major lines).

    A: M lines with line scales.  B: N lines with tile scales (b_scales "tile",
    a weight) or line scales ("line", the weight gradient)."""
    od = _out_code(out_dtype)
    fa, fb, bs = FP8_FMTS[fmt_a], FP8_FMTS[fmt_b], B_SCALES[b_scales]
    M, N, K = int(M), int(N), int(K)
    ca, ra = fp8_shapes(M, K)
    cb, rb = fp8_shapes(N, K, bs)
    _need_rows(A, "codes_A", torch.uint8, ca)
    dev = A.get_device()
    _need_rows(sA, "scales_A", torch.float32, ra, dev)
    _need_rows(B, "codes_B", torch.uint8, cb, dev)
    _need_rows(sB, "scales_B", torch.float32, rb, dev)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A.device)
    else:
        _need_rows(out, "out", out_dtype, (M, N), dev)
    _ok(mxq_fp8_gemm(A.data_ptr(), sA.data_ptr(), fa, B.data_ptr(), sB.data_ptr(), fb, bs, M, N, K,
                     out.data_ptr(), od, _stream(dev)), "mxq_fp8_gemm")
    return out


# ---- layer norm and RMS norm ---------------------------------------------------------

_FLOAT_CODES = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}


def _need_norm(x, weight, bias):
    """x [rows, cols] and the vectors of its norm; returns (device index, code of
    x's dtype, code of weight's dtype)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D torch.Tensor [rows, cols]")
    _need(x, "x", None, 0)
    dev = x.get_device()
    _need(weight, "weight", None, x.shape[1], dev)
    if bias is not None:
        _need(bias, "bias", weight.dtype, x.shape[1], dev)
    xd, wd = _FLOAT_CODES.get(x.dtype), _FLOAT_CODES.get(weight.dtype)
    if xd is None or wd is None:
        raise ValueError(f"x and weight must be torch.float32 or torch.bfloat16, got {x.dtype} "
                         f"and {weight.dtype}")
    return dev, xd, wd


def _norm_forward(x, weight, bias, eps, kind, fmt, with_y, out):
    """(y or None, codes or None, scales or None, mean or None, rstd)."""
    dev, xd, wd = _need_norm(x, weight, bias)
    R, C = x.shape
    y = codes = scales = None
    f = 0
    if with_y:
        if out is None:
            y = torch.empty_like(x)
        else:
            y = out
            _need_rows(y, "out", x.dtype, (R, C), dev)
    else:
        f = FP8_FMTS[fmt]
        if out is None:
            codes, scales = _fp8_buffers(R, C, "line", x.device)
        else:
            codes, scales = out
            _need_fp8(codes, scales, R, C, "line", dev)
    rstd = torch.empty(R, dtype=torch.float32, device=x.device)
    mean = torch.empty_like(rstd) if kind == NORM_LAYER else None
    if C == 0:   # the library writes nothing: the mean of no elements, 0 / 0
        for stat in (rstd,) if mean is None else (mean, rstd):
            stat.fill_(float("nan"))
    a = _NORM_ARGS.pack(x.data_ptr(), weight.data_ptr(), 0 if bias is None else bias.data_ptr(),
                        y.data_ptr() if with_y else 0, 0 if mean is None else mean.data_ptr(),
                        rstd.data_ptr(), 0 if with_y else codes.data_ptr(),
                        0 if with_y else scales.data_ptr(), R, C, eps, kind, xd, wd, f)
    _ok(mxq_norm_forward(a, _stream(dev)), "mxq_norm_forward")
    return y, codes, scales, mean, rstd


def layer_norm(x: torch.Tensor, weight, bias=None, eps=1e-5, out=None):
    """Layer norm of the rows of a contiguous bf16 or fp32 CUDA tensor; weight
    and bias bf16 or fp32.  Returns (y, mean, rstd), the statistics in fp32."""
    y, _, _, mean, rstd = _norm_forward(x, weight, bias, eps, NORM_LAYER, None, True, out)
    return y, mean, rstd


def rms_norm(x: torch.Tensor, weight, eps=1e-5, out=None):
    """RMS norm of the rows of a contiguous bf16 or fp32 CUDA tensor; returns
    (y, rstd)."""
    y, _, _, _, rstd = _norm_forward(x, weight, None, eps, NORM_RMS, None, True, out)
    return y, rstd


def layer_norm_quantize(x: torch.Tensor, weight, bias=None, eps=1e-5, fmt="e4m3", out=None):
    """Layer norm straight to row-wise block-128 FP8 codes of the fp32 values;
    returns (codes, scales, mean, rstd)."""
    _, codes, scales, mean, rstd = _norm_forward(x, weight, bias, eps, NORM_LAYER, fmt, False, out)
    return codes, scales, mean, rstd


def rms_norm_quantize(x: torch.Tensor, weight, eps=1e-5, fmt="e4m3", out=None):
    """RMS norm straight to row-wise block-128 FP8 codes of the fp32 values;
    returns (codes, scales, rstd)."""
    _, codes, scales, _, rstd = _norm_forward(x, weight, None, eps, NORM_RMS, fmt, False, out)
    return codes, scales, rstd


@functools.lru_cache(maxsize=4096)
def _norm_backward_workspace(rows, cols, index):
    """Bytes on the device of that index (None: no GPU in play): they depend on its
    number of SMs, and the library asks the current device."""
    with contextlib.nullcontext() if index is None else torch.cuda.device(index):
        return int(mxq_norm_backward_workspace_size(rows, cols))


def norm_backward_workspace(rows, cols, device):
    """A workspace of layer_norm_backward and rms_norm_backward on a CUDA device."""
    device = torch.device(device)
    index = device.index
    if index is None and device.type == "cuda":
        index = torch.cuda.current_device()
    return torch.empty(max(_norm_backward_workspace(rows, cols, index), 256), dtype=torch.uint8,
                       device=device)


def _norm_backward(dy, x, weight, mean, rstd, kind, out, workspace):
    dev, xd, wd = _need_norm(x, weight, None)
    R, C = x.shape
    _need_rows(dy, "dy", x.dtype, (R, C), dev)
    _need(rstd, "rstd", torch.float32, R, dev)
    if kind == NORM_LAYER:
        _need(mean, "mean", torch.float32, R, dev)
    if out is None:
        dx = torch.empty_like(x)
    else:
        dx = out
        _need_rows(dx, "out", x.dtype, (R, C), dev)
    if workspace is None:
        workspace = norm_backward_workspace(R, C, x.device)
    else:
        _need(workspace, "workspace", torch.uint8, 0, dev)   # its size is checked by the library
    dw = torch.empty(C, dtype=torch.float32, device=x.device)
    db = torch.empty_like(dw) if kind == NORM_LAYER else None
    a = _NORM_GRAD_ARGS.pack(dy.data_ptr(), x.data_ptr(), weight.data_ptr(),
                             0 if mean is None else mean.data_ptr(), rstd.data_ptr(),
                             dx.data_ptr(), dw.data_ptr(), 0 if db is None else db.data_ptr(),
                             workspace.data_ptr(), workspace.numel(), R, C, kind, xd, wd)
    _ok(mxq_norm_backward(a, _stream(dev)), "mxq_norm_backward")
    return dx, dw, db


def layer_norm_backward(dy, x, weight, mean, rstd, out=None, workspace=None):
    """Gradients of layer_norm from its statistics; returns (dx, dweight, dbias),
    dx in x's dtype and the others in fp32.  workspace: as
    norm_backward_workspace returns it, for callers that keep one."""
    return _norm_backward(dy, x, weight, mean, rstd, NORM_LAYER, out, workspace)


def rms_norm_backward(dy, x, weight, rstd, out=None, workspace=None):
    """Gradients of rms_norm from its statistics; returns (dx, dweight)."""
    return _norm_backward(dy, x, weight, None, rstd, NORM_RMS, out, workspace)[:2]


# ---- layers of experts -----------------------------------------------------------------

def expert_rows(choices: int, experts: int, align: int = 1) -> int:
    """Rows of a buffer that holds any routing of `choices` choices, every expert's rows
    padded to a multiple of `align`."""
    n = choices + min(experts, choices) * (align - 1)
    return (n + align - 1) // align * align


@functools.lru_cache(maxsize=4096)
def _order_workspace(n, experts):
    return int(mxq_expert_order_workspace_size(n, experts))


def expert_order(ids: torch.Tensor, experts: int, align: int = 1):
    """Rows of the choices ids [tokens, topk] (int32 or int64, contiguous, on the GPU) in
    a buffer sorted by expert; an id outside [0, experts) goes to no expert.  Returns
    (row_of [tokens, topk], offsets [experts + 1], counts [experts]), all int32: expert
    e holds rows offsets[e] to offsets[e + 1], its counts[e] choices in their order and
    padding up to a multiple of `align`.  Nothing waits for the device."""
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a 2-D torch.Tensor [tokens, topk]")
    if ids.dtype is not torch.int32 and ids.dtype is not torch.int64:
        raise ValueError(f"ids must be torch.int32 or torch.int64, got {ids.dtype}")
    _need(ids, "ids", None, 0)
    experts, align = int(experts), int(align)
    if not 1 <= experts <= 1024:
        raise ValueError(f"experts must be 1 to 1024, got {experts}")
    tokens, topk = ids.shape
    n, dev = tokens * topk, ids.get_device()
    where = ids.device
    row_of = torch.empty((tokens, topk), dtype=torch.int32, device=where)
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=where)
    counts = torch.empty(experts, dtype=torch.int32, device=where)
    ws_bytes = _order_workspace(n, experts)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=where) if ws_bytes else None
    _ok(mxq_expert_order(ids.data_ptr(), ids.element_size(), n, experts, align, row_of.data_ptr(),
                         offsets.data_ptr(), counts.data_ptr(), _ptr(ws), ws_bytes,
                         _stream(dev)), "mxq_expert_order")
    return row_of, offsets, counts


def _need_tokens(t, name):
    """t: a contiguous 2-D bf16 or fp32 CUDA tensor; returns (device index, code of its
    dtype)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D torch.Tensor")
    _need(t, name, None, 0)
    code = _FLOAT_CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    return t.get_device(), code


def _need_choices(row_of, weights, dev, tokens=None):
    """row_of [tokens, topk] and the weights beside it; returns its shape."""
    _need(row_of, "row_of", torch.int32, 0, dev)
    if row_of.dim() != 2 or (tokens is not None and row_of.shape[0] != tokens):
        raise ValueError(f"row_of must be [tokens, topk], got {tuple(row_of.shape)}")
    if weights is not None:
        _need(weights, "weights", torch.float32, 0, dev)
        if weights.shape != row_of.shape:
            raise ValueError(f"weights must be {tuple(row_of.shape)}, got {tuple(weights.shape)}")
    return row_of.shape


def _need_apart(out, t, name):
    """out and t share no memory: a call reads rows of t after it has written rows of out."""
    a, b = out.data_ptr(), t.data_ptr()
    if a < b + t.numel() * t.element_size() and b < a + out.numel() * out.element_size():
        raise ValueError(f"out and {name} share memory")


def _need_offsets(offsets, counts, dev):
    """Returns the number of experts."""
    _need(counts, "counts", torch.int32, 1, dev)
    experts = counts.numel()
    _need(offsets, "offsets", torch.int32, experts + 1, dev)
    if offsets.numel() != experts + 1:
        raise ValueError(f"offsets holds {offsets.numel()} elements, counts {experts}")
    return experts


def expert_gather(x: torch.Tensor, row_of, offsets, counts, rows, weights=None, out=None):
    """The tokens x [tokens, cols] (bf16 or fp32) at their choices' rows of a buffer
    [rows, cols], times weights [tokens, topk] (fp32) where given; zeros in the experts'
    padding.  row_of, offsets, counts: as expert_order returns them; rows: as
    expert_rows says, or fewer where the program knows the routing.  Rows from
    offsets[-1] on are not written.  Its gradient is expert_combine's sum (with the same
    weights)."""
    dev, code = _need_tokens(x, "x")
    tokens, topk = _need_choices(row_of, weights, dev, x.shape[0])
    experts = _need_offsets(offsets, counts, dev)
    rows, cols = int(rows), x.shape[1]
    if out is None:
        out = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
    else:
        _need_rows(out, "out", x.dtype, (rows, cols), dev)
        _need_apart(out, x, "x")
    a = _EXPERT_ROWS_ARGS.pack(x.data_ptr(), 0, out.data_ptr(), row_of.data_ptr(),
                               offsets.data_ptr(), counts.data_ptr(),
                               0 if weights is None else weights.data_ptr(), 0, tokens, rows, cols,
                               topk, experts, code)
    _ok(mxq_expert_gather(a, _stream(dev)), "mxq_expert_gather")
    return out


def expert_combine(y: torch.Tensor, row_of, weights=None, out=None):
    """Sums of the rows y [rows, cols] (bf16 or fp32) back into the tokens: token t gets
    sum_j weights[t, j] * y[row_of[t, j]] in fp32, rounded once (weights None: ones)."""
    dev, code = _need_tokens(y, "y")
    tokens, topk = _need_choices(row_of, weights, dev)
    rows, cols = y.shape
    if out is None:
        out = torch.empty((tokens, cols), dtype=y.dtype, device=y.device)
    else:
        _need_rows(out, "out", y.dtype, (tokens, cols), dev)
        _need_apart(out, y, "y")
    a = _EXPERT_ROWS_ARGS.pack(0, y.data_ptr(), out.data_ptr(), row_of.data_ptr(), 0, 0,
                               0 if weights is None else weights.data_ptr(), 0, tokens, rows, cols,
                               topk, 0, code)
    _ok(mxq_expert_combine(a, _stream(dev)), "mxq_expert_combine")
    return out


def expert_combine_backward(dout: torch.Tensor, y, row_of, offsets, counts, weights=None,
                            out=None):
    """Gradients of expert_combine: (dy [rows, cols] in y's dtype, dweights [tokens, topk]
    in fp32).  The experts' padding of dy is zeros; rows from offsets[-1] on are not
    written.  out: dy's buffer, which may be y."""
    dev, code = _need_tokens(dout, "dout")
    tokens, topk = _need_choices(row_of, weights, dev, dout.shape[0])
    experts = _need_offsets(offsets, counts, dev)
    cols = dout.shape[1]
    if not isinstance(y, torch.Tensor) or y.dim() != 2 or y.shape[1] != cols:
        raise ValueError(f"y must be a 2-D torch.Tensor with rows of {cols} elements")
    rows = y.shape[0]
    _need(y, "y", dout.dtype, 0, dev)
    if out is None:
        out = torch.empty_like(y)
    else:
        _need_rows(out, "out", y.dtype, (rows, cols), dev)
        _need_apart(out, dout, "dout")
        if out.data_ptr() != y.data_ptr():
            _need_apart(out, y, "y")
    dweights = torch.empty((tokens, topk), dtype=torch.float32, device=y.device)
    a = _EXPERT_ROWS_ARGS.pack(dout.data_ptr(), y.data_ptr(), out.data_ptr(), row_of.data_ptr(),
                               offsets.data_ptr(), counts.data_ptr(),
                               0 if weights is None else weights.data_ptr(), dweights.data_ptr(),
                               tokens, rows, cols, topk, experts, code)
    _ok(mxq_expert_combine_backward(a, _stream(dev)), "mxq_expert_combine_backward")
    return out, dweights


@functools.lru_cache(maxsize=4096)
def _experts_workspace(rows, N, K, experts, fmt, b_scale_layout):
    return int(mxq_gemm_experts_workspace_size(rows, N, K, experts, fmt, b_scale_layout))


@functools.lru_cache(maxsize=4096)
def _experts_wgrad_workspace(rows, M, N, experts, fmt):
    return int(mxq_gemm_experts_wgrad_workspace_size(rows, M, N, experts, fmt))


def gemm_experts_workspace(rows, N, K, experts, fmt, device, b_scale_layout="rowmajor"):
    """A workspace of mx_gemm_experts."""
    n = _experts_workspace(int(rows), int(N), int(K), int(experts), FMTS[fmt],
                           SCALE_LAYOUTS[b_scale_layout])
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def gemm_experts_wgrad_workspace(rows, M, N, experts, fmt, device):
    """A workspace of mx_gemm_experts_wgrad."""
    n = _experts_wgrad_workspace(int(rows), int(M), int(N), int(experts), FMTS[fmt])
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _count_experts(offsets):
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1:
        raise ValueError("offsets must be a 1-D torch.Tensor [experts + 1]")
    return offsets.numel() - 1


@functools.lru_cache(maxsize=4096)
def _experts_sizes(rows, N, K, experts, fmt, b_scale_layout):
    """Bytes of mx_gemm_experts' A, sA, B, sB and workspace, and the library's codes of
    the format and the layout."""
    f, layout = FMTS[fmt], SCALE_LAYOUTS[b_scale_layout]
    kb = K // 2 if f == E2M1 else K
    sb = N * (K // 32)
    if layout == SCALES_TC:
        sb = int(mxq_scales_tc_bytes(N, K))
        if sb == 0 or (f == E2M1 and K % 256 != 0):
            raise ValueError(f"no tensor-core scale layout for {N} lines x {K}")
    return (rows * kb, rows * (K // 32), experts * N * kb, experts * sb,
            max(_experts_workspace(rows, N, K, experts, f, layout), 256), f, layout)


@functools.lru_cache(maxsize=4096)
def _experts_wgrad_sizes(rows, M, N, experts, fmt):
    """The same of mx_gemm_experts_wgrad."""
    f = FMTS[fmt]
    rb = rows // 2 if f == E2M1 else rows
    return (M * rb, M * (rows // 32), N * rb, N * (rows // 32),
            max(_experts_wgrad_workspace(rows, M, N, experts, f), 256), f)


def _need_product(A, sA, B, sB, offsets, sizes, dev):
    """The operands of a product grouped by expert."""
    _need(A, "codes_A", torch.uint8, sizes[0], dev)
    _need(sA, "scales_A", torch.uint8, sizes[1], dev)
    _need(B, "codes_B", torch.uint8, sizes[2], dev)
    _need(sB, "scales_B", torch.uint8, sizes[3], dev)
    _need(offsets, "offsets", torch.int32, 2, dev)


def mx_gemm_experts(A, sA, B, sB, offsets, fmt, rows, N, K, out_dtype=torch.float32, out=None,
                    workspace=None, b_scale_layout="rowmajor"):
    """C[r] = dec(A[r]) @ dec(B[e])^T for the rows r of every expert e, offsets[e] <= r <
    offsets[e + 1], on the tensor cores; returns C [rows, N].

    A: MX codes of the rows [rows, K] and their row-major scales; B: codes of the experts'
    weights [experts, N, K] and their scales, row-major, or ("tc") in the tensor cores'
    chunk layout, one buffer of mx_quantize(..., scale_layout="tc") per expert, one after
    another.  offsets: int32 [experts + 1] on the device (expert_order).  Rows that no
    expert holds are not written.  workspace: as gemm_experts_workspace returns it, for
    callers that keep one; two calls that may run at the same time need one each."""
    od = _out_code(out_dtype)
    experts = _count_experts(offsets)
    rows, N, K = int(rows), int(N), int(K)
    sizes = _experts_sizes(rows, N, K, experts, fmt, b_scale_layout)
    _need(A, "codes_A", torch.uint8, 0)
    dev = A.get_device()
    _need_product(A, sA, B, sB, offsets, sizes, dev)
    if out is None:
        out = torch.empty((rows, N), dtype=out_dtype, device=A.device)
    else:
        _need_rows(out, "out", out_dtype, (rows, N), dev)
    if workspace is None:
        workspace = torch.empty(sizes[4], dtype=torch.uint8, device=A.device)
    else:
        _need(workspace, "workspace", torch.uint8, 0, dev)   # its size is checked by the library
    a = _EXPERTS_ARGS.pack(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(),
                           offsets.data_ptr(), out.data_ptr(), workspace.data_ptr(),
                           workspace.numel(), rows, 0, N, K, experts, sizes[5], od, sizes[6])
    _ok(mxq_gemm_experts(a, _stream(dev)), "mxq_gemm_experts")
    return out


def mx_gemm_experts_wgrad(A, sA, B, sB, offsets, fmt, M, N, rows, out_dtype=torch.float32,
                          out=None, workspace=None):
    """C[e] = dec(A[:, r]) @ dec(B[:, r])^T over the rows r of every expert e; returns C
    [experts, M, N], zeros for an expert without rows.

    A: codes [M, rows] and row-major scales, B: [N, rows], both as
    mx_quantize(..., "col") writes them.  offsets: multiples of 32 (E2M1: 64), as
    expert_order(..., align=32) gives them.  workspace: as
    gemm_experts_wgrad_workspace returns it, for callers that keep one; two calls that
    may run at the same time need one each."""
    od = _out_code(out_dtype)
    experts = _count_experts(offsets)
    rows, M, N = int(rows), int(M), int(N)
    sizes = _experts_wgrad_sizes(rows, M, N, experts, fmt)
    _need(A, "codes_A", torch.uint8, 0)
    dev = A.get_device()
    _need_product(A, sA, B, sB, offsets, sizes, dev)
    if out is None:
        out = torch.empty((experts, M, N), dtype=out_dtype, device=A.device)
    else:
        _need(out, "out", out_dtype, experts * M * N, dev)
        if out.dim() > 1 and out.size(-1) != N:
            raise ValueError(f"out has rows of {out.size(-1)} elements; they must hold {N}")
    if workspace is None:
        workspace = torch.empty(sizes[4], dtype=torch.uint8, device=A.device)
    else:
        _need(workspace, "workspace", torch.uint8, 0, dev)   # its size is checked by the library
    a = _EXPERTS_ARGS.pack(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(),
                           offsets.data_ptr(), out.data_ptr(), workspace.data_ptr(),
                           workspace.numel(), rows, M, N, 0, experts, sizes[5], od,
                           SCALES_ROWMAJOR)
    _ok(mxq_gemm_experts_wgrad(a, _stream(dev)), "mxq_gemm_experts_wgrad")
    return out


# ---- AdamW ---------------------------------------------------------------------------------

def adamw_state(param: torch.Tensor, bits: int = 32):
    """The moments of an AdamW step on `param`, at zero: (m, v) in fp32, or, bits 8,
    ((codes, scales), (codes, scales)) of m and sqrt(v), E4M3 with one fp32 scale per
    128 elements."""
    if bits == 32:
        return tuple(torch.zeros(param.shape, dtype=torch.float32, device=param.device)
                     for _ in range(2))
    if bits != 8:
        raise ValueError(f"bits must be 32 or 8, got {bits}")
    blocks = (param.numel() + 127) // 128
    return tuple((torch.zeros(param.shape, dtype=torch.uint8, device=param.device),
                  torch.full((blocks,), 2.0 ** -126, device=param.device)) for _ in range(2))


def _spans(places, tensors):
    """[(first byte, end, index)] of the tensors' memory, in order."""
    sizes = [n * z for n, z in zip(map(torch.Tensor.numel, tensors),
                                   map(torch.Tensor.element_size, tensors))]
    return sorted([(a, a + n, i) for i, (a, n) in enumerate(zip(places, sizes)) if n])


def _overlap(names, spans):
    """The names of two of the spans' tensors that share memory, or None."""
    end, last = 0, None
    for a, b, i in spans:
        if a < end:
            return names(last), names(i)
        end, last = b, i
    return None


def _plain_tensors(tensors, dtype, numels, dev):
    """Whether all are contiguous CUDA tensors of dtype on device dev (host tensors have no
    device index of a GPU), each with at least as many elements as its number in numels."""
    try:
        return (all([t.dtype is dtype for t in tensors]) and all(map(_on_gpu, tensors[:1]))
                and all(map(torch.Tensor.is_contiguous, tensors))
                and all([n >= m for n, m in zip(map(torch.Tensor.numel, tensors), numels)])
                and set(map(torch.Tensor.get_device, tensors)) <= {dev})
    except (AttributeError, TypeError):
        return False


class AdamWPlan:
    """The tensors that adamw_step updates, checked once.  It keeps them; where one of
    them, a moment too, has moved since (its .data replaced, its storage resized), or a
    parameter or weight has another size or order at the same place, all are checked
    and looked up anew at the next step.  A captured step goes on with the memory that
    they had when it was captured."""

    def __init__(self, params, states, weights=None, weight_decay=0.0):
        self.params = list(params)
        self.states = [(m, v) if isinstance(m, torch.Tensor) else (tuple(m), tuple(v))
                       for m, v in states]
        self.weights = [None] * len(self.params) if weights is None else list(weights)
        try:
            self.weight_decay = [float(weight_decay)] * len(self.params)
        except TypeError:
            self.weight_decay = [float(w) for w in weight_decay]
        if not (len(self.params) == len(self.states) == len(self.weights)
                == len(self.weight_decay)):
            raise ValueError(f"{len(self.params)} params, {len(self.states)} states, "
                             f"{len(self.weights)} weights and {len(self.weight_decay)} "
                             "weight decays")
        self._check()

    def _groups(self):
        """[(name, dtype, tensors, elements that each must hold)] of everything written."""
        numels = [p.numel() for p in self.params]
        kinds = {isinstance(m, torch.Tensor) for m, _ in self.states}
        if len(kinds) > 1:
            raise ValueError("the states of a plan are all in 32 or all in 8 bits")
        groups = [("params[%d]", torch.float32, self.params, [0] * len(numels))]
        if True in kinds:
            for k, name in enumerate(("m", "v")):
                groups.append((f"states[%d].{name}", torch.float32, [s[k] for s in self.states],
                               numels))
        else:
            blocks = [(n + 127) // 128 for n in numels]
            for k, name in enumerate(("m", "v")):
                groups.append((f"states[%d].{name}[0]", torch.uint8,
                               [s[k][0] for s in self.states], numels))
            for k, name in enumerate(("m", "v")):
                groups.append((f"states[%d].{name}[1]", torch.float32,
                               [s[k][1] for s in self.states], blocks))
        self.bits = 32 if True in kinds else 8
        return numels, groups

    def _check(self, moved=False):
        for i, p in enumerate(self.params):
            if not isinstance(p, torch.Tensor):
                _need(p, f"params[{i}]", torch.float32, 0)
        dev = self.params[0].get_device() if self.params else None
        numels, groups = self._groups()
        have = [i for i, w in enumerate(self.weights) if w is not None]
        weights = [self.weights[i] for i in have]
        for name, dtype, tensors, least in groups:
            if not _plain_tensors(tensors, dtype, least, dev):
                for i, t in enumerate(tensors):   # word the error
                    _need(t, name % i, dtype, least[i], dev)
        if not _plain_tensors(weights, torch.bfloat16, [numels[i] for i in have], dev):
            for i in have:
                _need(self.weights[i], f"weights[{i}]", torch.bfloat16, numels[i], dev)
        columns = [list(map(torch.Tensor.data_ptr, g[2])) for g in groups]
        copies = [0] * len(numels)
        for i, a in zip(have, map(torch.Tensor.data_ptr, weights)):
            copies[i] = a
        every = [t for g in groups for t in g[2]] + weights
        places = [a for c in columns for a in c] + [copies[i] for i in have]

        def name(i):
            k, n = divmod(i, max(len(numels), 1))
            return groups[k][0] % n if i < len(numels) * len(groups) \
                else f"weights[{have[i - len(numels) * len(groups)]}]"

        if moved or 0 in places:   # a resized storage may hold less than its tensor
            for i, t in enumerate(every):
                if t.untyped_storage().nbytes() < (t.storage_offset() + t.numel()) * t.element_size() \
                        and t.numel():
                    raise ValueError(f"the storage of {name(i)} holds less than the tensor")
        spans = _spans(places, every)
        twice = _overlap(name, spans)
        if twice:
            raise ValueError(f"{twice[0]} and {twice[1]} share memory")
        none = [0] * len(numels)
        rows = zip(*columns, *([none] * (5 - len(columns))), copies, numels, self.weight_decay)
        self.device, self.numels = dev, numels
        self._written, self._places = every, places
        # moments are their memory: elements at the parameter's places, whatever the view
        self._viewed, self._sizes = self.params + weights, numels + [t.numel() for t in weights]
        self._table = b"".join([_ADAMW_TENSOR.pack(*row) for row in rows])
        # first and last byte of every written piece of memory, in order, and the gradients
        # that were found apart from them
        self._bounds = [at for span in spans for at in span[:2]]
        self._apart = None
        self._grads = struct.Struct(f"@{len(numels)}P")

    def table(self):
        """The tensors' part of a launch; taken anew where one has moved."""
        if (list(map(torch.Tensor.data_ptr, self._written)) != self._places
                or list(map(torch.Tensor.numel, self._viewed)) != self._sizes
                or not all(map(torch.Tensor.is_contiguous, self._viewed))):
            self._check(moved=True)
        return self._table

    def grads(self, grads):
        """(the gradients' part of a launch, the code of their dtype)."""
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} grads for {len(self.params)} params")
        try:
            dtypes = {g.dtype for g in grads}
            ok = (len(dtypes) == 1 and list(map(torch.Tensor.numel, grads)) == self.numels
                  and all(map(torch.Tensor.is_contiguous, grads))
                  and set(map(torch.Tensor.get_device, grads)) == {self.device})
        except (AttributeError, TypeError):
            ok = False
        dtype = grads[0].dtype if isinstance(grads[0], torch.Tensor) else None
        code = _FLOAT_CODES.get(dtype)
        if code is None:
            raise ValueError(f"grads must be torch.float32 or torch.bfloat16, got {dtype}")
        if not ok:   # word the error
            for i, (g, n) in enumerate(zip(grads, self.numels)):
                _need(g, f"grads[{i}]", dtype, n, self.device)
                if g.numel() != n:
                    raise ValueError(f"grads[{i}] holds {g.numel()} elements, its parameter {n}")
        places = list(map(torch.Tensor.data_ptr, grads))
        packed = self._grads.pack(*places)
        if self._apart != (packed, code):   # the same places of as many bytes: known
            size = grads[0].element_size()
            first = list(map(bisect_right, repeat(self._bounds), places))
            last = list(map(bisect_left, repeat(self._bounds),
                            [a + n * size for a, n in zip(places, self.numels)]))
            if first != last or any([k & 1 for k in first]):
                for i, g in enumerate(grads):
                    self.need_apart(g, places[i], f"grads[{i}]")
            self._apart = packed, code
        return packed, code

    def need_apart(self, t, at, name):
        """t, at address `at`, shares no memory with what a step writes."""
        end = at + t.numel() * t.element_size()
        k = bisect_right(self._bounds, at)
        if at < end and (k & 1 or k != bisect_left(self._bounds, end)):
            raise ValueError(f"{name} shares memory with a parameter, its weight or its state")


def adamw_plan(params, states, weights=None, weight_decay=0.0):
    """A plan of adamw_step: contiguous fp32 CUDA tensors `params`, for each what
    adamw_state returned, and for each a bf16 tensor of its size that receives the
    rounded parameter (the quantizers' input), or None.  weight_decay: one number, or one
    per tensor.  No two of them may share memory.  A step finds tensors that have moved
    since, a captured one does not (AdamWPlan)."""
    return AdamWPlan(params, states, weights, weight_decay)


def _scalar(value, name, dtype, plan):
    """(number, device address or 0) of a number or a 1-element CUDA tensor."""
    if not isinstance(value, torch.Tensor):
        return value, 0
    _need(value, name, dtype, 1, plan.device)
    at = value.data_ptr()
    plan.need_apart(value, at, name)
    return 1, at


def adamw_step(plan: AdamWPlan, grads, step, lr, betas=(0.9, 0.999), eps=1e-8, grad_scale=None):
    """One AdamW step of the plan's tensors, in place.  grads: one contiguous tensor per
    parameter, all fp32 or all bf16; step: 1 at the first step.  step (int64), lr (fp32)
    and grad_scale (fp32; a factor of the gradients, NaN or infinity to leave everything
    as it is) may be 1-element CUDA tensors, which a captured launch reads anew.  None of
    what it reads may overlap what it writes."""
    if not plan.params:
        return
    table, dev = plan.table(), plan.device
    places, code = plan.grads(grads)
    t, t_at = _scalar(step, "step", torch.int64, plan)
    rate, rate_at = _scalar(lr, "lr", torch.float32, plan)
    scale_at = 0
    if grad_scale is not None:
        _need(grad_scale, "grad_scale", torch.float32, 1, dev)
        _, scale_at = _scalar(grad_scale, "grad_scale", torch.float32, plan)
    a = _ADAMW_ARGS.pack(rate, betas[0], betas[1], eps, t, rate_at, t_at, scale_at, code, plan.bits)
    _ok(mxq_adamw(table, places, len(plan.params), a, _stream(dev)), "mxq_adamw")
