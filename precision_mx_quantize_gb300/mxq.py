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
``_backward`` forms.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import struct
import threading

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


# The same two structures as native-layout formats: packing one takes a third
# of the time of filling the ctypes mirror, which small calls notice.
_NORM_ARGS = struct.Struct("@8P2qf4i0q")
_NORM_GRAD_ARGS = struct.Struct("@9PN2q3i0q")

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


def _stream(device=None) -> int:
    """The raw handle of the current CUDA stream of `device` (default: the
    current device).  Uses torch's raw-handle accessor when it has one, which
    skips building a Stream object on every call."""
    if _raw_stream is not None:
        if device is None:
            idx = torch.cuda.current_device()
        elif isinstance(device, int):
            idx = device
        else:
            idx = device.index if device.index is not None else torch.cuda.current_device()
        return _raw_stream(idx)
    return torch.cuda.current_stream(device).cuda_stream


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


def mxq_check(stream=None):
    return lib().mxq_check(stream)


def check(device=None):
    """Synchronize the current stream and raise on any recorded device error."""
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
                              sc.data_ptr(), _stream(x.device)), "mxq_quantize_dual")
    else:
        _ok(mxq_quantize_dual_ex(x.data_ptr(), x.shape[0], x.shape[1], FMTS[fmt_r], int(had_r),
                                 cr.data_ptr(), sr.data_ptr(), FMTS[fmt_c], int(had_c),
                                 cc.data_ptr(), sc.data_ptr(), SCALES_TC, _stream(x.device)),
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
                              _stream(x.device)), "mxq_quantize_ablation")
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
                        K, out.data_ptr(), od, SCALES_TC, None, 0, _stream(A.device)),
            "mxq_gemm_ex")
        return out
    if workspace is None:
        workspace = gemm_workspace(M, N, K, fmt, A.device)
    _need(workspace, "workspace", torch.uint8, 0, dev)   # its size is checked by the library
    _ok(mxq_gemm(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(), FMTS[fmt], M, N, K,
                 out.data_ptr(), od, workspace.data_ptr(), workspace.numel(),
                 _stream(A.device)), "mxq_gemm")
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
                              workspace.data_ptr(), workspace.numel(), _stream(A.device)),
            "mxq_gemm_quantize")
        return codes, scales
    if not in_tc and workspace is None:
        workspace = gemm_workspace(M, N, K, fmt, A.device)
    ws_ptr, ws_n = (None, 0) if in_tc else (workspace.data_ptr(), workspace.numel())
    _ok(mxq_gemm_quantize_ex(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(), FMTS[fmt], M,
                             N, K, SCALE_LAYOUTS[scale_layout], FMTS[out_fmt], codes.data_ptr(),
                             scales.data_ptr(), SCALE_LAYOUTS[out_scale_layout], ws_ptr, ws_n,
                             _stream(A.device)), "mxq_gemm_quantize_ex")
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
