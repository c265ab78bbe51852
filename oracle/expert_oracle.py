"""Plain CPU definitions of a layer of experts and of the AdamW step, in float64.

Written from the definitions in include/mxq.h, independent of the CUDA code.
"""

from __future__ import annotations

import numpy as np

from oracle import fp8_oracle as F
from oracle import mx_oracle as O


def order(ids: np.ndarray, experts: int, align: int):
    """(row_of, offsets, counts) of the choices ids [tokens, topk]."""
    flat = ids.reshape(-1).astype(np.int64)
    counts = np.array([(flat == e).sum() for e in range(experts)], np.int64)
    offsets = np.concatenate([[0], np.cumsum((counts + align - 1) // align * align)])
    row_of, seen = np.full(flat.size, -1, np.int64), np.zeros(experts, np.int64)
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            row_of[i] = offsets[e] + seen[e]
            seen[e] += 1
    return row_of.reshape(ids.shape), offsets, counts


def gather(x, row_of, offsets, counts, out, weights=None):
    """`out` with x's rows at their choices' rows and zeros in the experts' padding."""
    out = out.astype(np.float64).copy()
    for e, c in enumerate(counts):
        out[offsets[e] + c:offsets[e + 1]] = 0.0
    for (t, j), r in np.ndenumerate(row_of):
        if r >= 0:
            out[r] = x[t] * (1.0 if weights is None else float(weights[t, j]))
    return out


def combine(y, row_of, weights=None):
    """(sums, sums of magnitudes)."""
    out = np.zeros((row_of.shape[0], y.shape[1]))
    size = np.zeros_like(out)
    for (t, j), r in np.ndenumerate(row_of):
        if r >= 0:
            v = y[r].astype(np.float64) * (1.0 if weights is None else float(weights[t, j]))
            out[t] += v
            size[t] += np.abs(v)
    return out, size


def combine_dweights(dout, y, row_of):
    """(gradients of the weights, sums of magnitudes)."""
    dw, size = np.zeros(row_of.shape), np.zeros(row_of.shape)
    for (t, j), r in np.ndenumerate(row_of):
        if r >= 0:
            v = dout[t].astype(np.float64) * y[r].astype(np.float64)
            dw[t, j], size[t, j] = v.sum(), np.abs(v).sum()
    return dw, size


def experts_product(A, sA, B, sB, offsets, fmt, out):
    """(C, S) of the rows form; rows that no expert holds keep `out` (S 0)."""
    c, s = out.astype(np.float64).copy(), np.zeros(out.shape)
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            c[lo:hi], s[lo:hi] = O.mx_gemm_f64(A[lo:hi], sA[lo:hi], B[e], sB[e], fmt)
    return c, s


def experts_wgrad(A, sA, B, sB, offsets, fmt):
    """(C, S) of the weight gradients [experts][M][N]."""
    a, b = O.dequantize_f64(A, sA, fmt), O.dequantize_f64(B, sB, fmt)
    parts = [(a[:, lo:hi] @ b[:, lo:hi].T, np.abs(a[:, lo:hi]) @ np.abs(b[:, lo:hi]).T)
             for lo, hi in zip(offsets, offsets[1:])]
    return np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])


def moment(codes, scales):
    """Values of an 8-bit moment: E4M3 codes, one scale per 128 of them."""
    return O.decode_table("e4m3")[codes] * np.repeat(scales.astype(np.float64), F.BLOCK)[:codes.size]


def adamw(p, g, m, v, step, lr, b1, b2, eps, decay):
    """(p, m, v, update) after one step: float64 values of flat tensors; `update` is the
    magnitude that m's two terms give the step of p."""
    b1, b2 = float(b1), float(b2)
    new_m, new_v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    denom = np.sqrt(new_v / (1 - b2 ** step)) + eps
    rate = lr / (1 - b1 ** step)
    with np.errstate(invalid="ignore", divide="ignore"):
        new_p = p - lr * decay * p - rate * new_m / denom
        update = rate * (np.abs(b1 * m) + np.abs((1 - b1) * g)) / denom
    return new_p, new_m, new_v, update
