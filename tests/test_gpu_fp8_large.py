"""Block-128 FP8 operators and norms on tensors of more than 2^31 elements.

The last rows and lines lie past every 32-bit offset.  Quantizers and the
backward pass's rows do not depend on the other rows: they equal a call on the
last rows alone, bit for bit.  Norm outputs and products are held to the bounds
of the small cases.
"""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from precision_mx_quantize_gb300 import mxq
from tests.libutil import ensure_built, to_np
from tests.test_gpu_norm import EPS, U, _bounds, _f

pytestmark = pytest.mark.gpu
COLS = 4096
LAST = 384                          # a multiple of 128: whole blocks of the columns
ROWS = 2 ** 31 // COLS + LAST


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()
    yield
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def x():
    torch.manual_seed(5)
    return torch.randn(ROWS, COLS, device="cuda", dtype=torch.bfloat16)


def test_quantizers(x):
    first = ROWS - LAST
    tail = x[first:].clone()
    c, s = mxq.fp8_quantize(x)
    tc, ts = mxq.fp8_quantize(tail)
    assert torch.equal(c[first:], tc) and torch.equal(s[:, first:], ts)
    del c, s
    cr, sr, cc, sc = mxq.fp8_quantize_dual(x)
    ec, es = mxq.fp8_quantize(tail, "col")
    assert torch.equal(cr[first:], tc) and torch.equal(sr[:, first:], ts)
    assert torch.equal(cc[:, first:], ec) and torch.equal(sc[first // 128:], es)
    del cr, sr, cc, sc
    got, want = mxq.fp8_quantize_tiles(x), mxq.fp8_quantize_tiles(tail)
    b = first // 128
    mxq.check()
    for g, w in zip((got[0][first:], got[1][b:], got[2][:, first:], got[3][:, b:]), want):
        assert torch.equal(g, w)


def test_norm(x):
    first = ROWS - LAST
    w = torch.linspace(0.5, 1.5, COLS, device="cuda")
    b = torch.linspace(-0.1, 0.1, COLS, device="cuda")
    tail = x[first:].clone()
    y, mean, rstd = mxq.layer_norm(x, w, b, EPS)
    ey, _, er, ty, dm, dr = _bounds(tail, w, b, "layer")
    ty = ty + 2.0 ** -8 * (np.abs(ey) + ty)
    assert (np.abs(_f(y[first:]) - ey) <= ty).all()
    assert (np.abs(_f(rstd[first:]) - er) <= dr * er).all()
    c, s, rms = mxq.rms_norm_quantize(x, w, EPS)
    tc, ts, trms = mxq.rms_norm_quantize(tail, w, EPS)
    # other kernels for fewer rows: their statistics may differ by 2 dr, a code by a step
    _, _, _, _, _, dr = _bounds(tail, w, None, "rms")
    assert (np.abs(_f(rms[first:]) - _f(trms)) <= 2 * dr * _f(trms)).all()
    near = (c[first:].int() - tc.int()).abs() <= 1
    assert near.all() and (s[:, first:] / ts - 1).abs().max() <= 2 * dr.max() + 16 * U
    del c, s
    dy = y                          # any gradient does
    dx, dw, db = mxq.layer_norm_backward(dy, x, w, mean, rstd)
    tdx, _, _ = mxq.layer_norm_backward(dy[first:].clone(), tail, w, mean[first:].clone(),
                                        rstd[first:].clone())
    mxq.check()
    assert torch.equal(dx[first:], tdx)
    del dx
    sums = torch.zeros(4, COLS, device="cuda", dtype=torch.float64)
    for r in range(0, ROWS, 16384):
        g = dy[r:r + 16384].double()
        gh = (x[r:r + 16384].double() - mean[r:r + 16384, None]) * rstd[r:r + 16384, None] * g
        sums += torch.stack([gh.sum(0), gh.abs().sum(0), g.sum(0), g.abs().sum(0)])
    # chains of at most a CTA's rows, the join's sets and a few more: far below ROWS
    chain = ROWS / 152 + 1024
    assert ((dw - sums[0]).abs() <= chain * U * sums[1]).all()
    assert ((db - sums[2]).abs() <= chain * U * sums[3]).all()


# 2^31 elements of C (tile stores, element copies), 2^31 codes of B (a token, many)
@pytest.mark.parametrize("m, n, k, kind", [(65664, 32776, 256, "tile"), (65664, 32777, 256, "line"),
                                           (1, 131200, 16384, "line"), (512, 131200, 16384, "line")],
                         ids=str)
def test_product(m, n, k, kind):
    torch.manual_seed(6)
    A, sA = mxq.fp8_quantize(torch.randn(m, k, device="cuda", dtype=torch.bfloat16))
    w = torch.randn(n, k, device="cuda", dtype=torch.bfloat16)
    B, sB = mxq.fp8_quantize(w) if kind == "line" else mxq.fp8_quantize_tiles(w)[:2]
    del w
    c = mxq.fp8_gemm(A, sA, B, sB, m, n, k, b_scales=kind)
    mxq.check()
    i, j = max(m - 40, 0) // 4 * 4, (n - 128) // 128 * 128
    a = F.values(to_np(A[i:]), to_np(sA[:, i:m]), k, "e4m3", "line")
    sb = sB[:, j:n] if kind == "line" else sB[j // 128:]
    ref, S = F.gemm(a, F.values(to_np(B[j:]), to_np(sb), k, "e4m3", kind))
    tol = (k + k / 128 + 4) * 2.0 ** -23 * S
    tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert (np.abs(to_np(c[i:, j:].float()) - ref) <= tol).all()
