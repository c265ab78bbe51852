"""Plain CPU definitions of the block-128 FP8 format, its product and the norms.

Written from the definitions in include/mxq.h, in float64, independent of the
CUDA code.  The quantizer's three fp32 roundings (scale, reciprocal, product)
are part of its definition; each is one float64 operation on fp32 values
rounded to fp32, which is the correctly rounded fp32 result (float64 carries
more than twice the bits).
"""

from __future__ import annotations

import numpy as np

from oracle import mx_oracle as O

BLOCK = 128
TINY = np.float32(2.0 ** -126)


def up(n: int, m: int) -> int:
    return (n + m - 1) // m * m


def _scale(amax: np.ndarray, bad: np.ndarray, fmt: str):
    """fp32 (scale, multiplier) per block; NaN scale for a bad block."""
    fmax = O.fmt_params(fmt)["maxval"]
    s = np.maximum((amax.astype(np.float64) / fmax).astype(np.float32), TINY)
    mul = (1.0 / s.astype(np.float64)).astype(np.float32)
    return np.where(bad, np.float32(np.nan), s), mul


def _codes(v: np.ndarray, mul: np.ndarray, bad: np.ndarray, fmt: str) -> np.ndarray:
    with np.errstate(invalid="ignore", over="ignore"):
        q = (np.where(bad, 0.0, v.astype(np.float64)) * mul.astype(np.float64)).astype(np.float32)
    c = O.encode_element(O.round_to_element(q.astype(np.float64), fmt), fmt)
    return np.where(bad, np.uint8(0), c)


def quantize_lines(x: np.ndarray, fmt: str):
    """x [lines][K] fp32 -> codes [lines][K up to 16] uint8, scales [K blocks]
    [lines up to 4] fp32."""
    lines, k = x.shape
    kb, lp = up(k, BLOCK) // BLOCK, up(lines, 4)
    v = np.zeros((lp, kb, BLOCK), np.float32)
    v.reshape(lp, -1)[:lines, :k] = x
    bad = ~np.isfinite(v).all(-1)
    amax = np.abs(np.where(np.isfinite(v), v, 0)).max(-1)
    s, mul = _scale(amax, bad, fmt)
    c = _codes(v, mul[..., None], bad[..., None], fmt).reshape(lp, -1)
    return np.ascontiguousarray(c[:lines, :up(k, 16)]), np.ascontiguousarray(s.T)


def quantize_tiles(x: np.ndarray, fmt: str):
    """x [rows][cols] -> codes, scales, transposed codes, transposed scales."""
    r, c = x.shape
    rb, cb = up(r, BLOCK) // BLOCK, up(c, BLOCK) // BLOCK
    v = np.zeros((rb * BLOCK, cb * BLOCK), np.float32)
    v[:r, :c] = x
    t = v.reshape(rb, BLOCK, cb, BLOCK)
    bad = ~np.isfinite(t).all((1, 3))
    amax = np.abs(np.where(np.isfinite(t), t, 0)).max((1, 3))
    s, mul = _scale(amax, bad, fmt)
    q = _codes(t, mul[:, None, :, None], bad[:, None, :, None], fmt).reshape(v.shape)
    return (np.ascontiguousarray(q[:r, :up(c, 16)]), s,
            np.ascontiguousarray(q.T[:c, :up(r, 16)]), np.ascontiguousarray(s.T))


def values(codes: np.ndarray, scales: np.ndarray, k: int, fmt: str, kind: str) -> np.ndarray:
    """The float64 values that `codes` of lines of k elements stand for."""
    v = O.decode_table(fmt)[codes[:, :k]]
    at = np.arange(k) // BLOCK
    if kind == "tile":
        return v * scales.astype(np.float64)[np.arange(v.shape[0]) // BLOCK][:, at]
    return v * scales.astype(np.float64)[:, :v.shape[0]].T[:, at]


def gemm(a: np.ndarray, b: np.ndarray):
    """(C, S): the product of the values and sum_k |a b| per element."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def norm(x, w, b, eps, kind):
    """(y, mean or None, rstd) of the rows of x in float64."""
    x = x.astype(np.float64)
    mean = x.mean(1) if kind == "layer" else None
    d = x - mean[:, None] if kind == "layer" else x
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None] * w.astype(np.float64)
    return (y if b is None else y + b.astype(np.float64)), mean, rstd


def norm_backward(dy, x, w, mean, rstd, kind):
    """(dx, dweight, dbias) in float64 from the given statistics."""
    x, dy, w = (t.astype(np.float64) for t in (x, dy, w))
    h = (x - mean.astype(np.float64)[:, None] if kind == "layer" else x) \
        * rstd.astype(np.float64)[:, None]
    g = dy * w
    dx = g - h * (g * h).mean(1, keepdims=True)
    if kind == "layer":
        dx = dx - g.mean(1, keepdims=True)
    return dx * rstd.astype(np.float64)[:, None], (dy * h).sum(0), dy.sum(0)
