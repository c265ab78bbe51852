"""Layer norm and RMS norm on the GPU against float64.

Bounds, with u = 2^-24 and L = cols / 32 + 64 the longest chain of additions a
row sum can take (32 threads, each at most cols / 32 elements, then a tree):
* mean is off by at most dm = (L + 2) u mean|x|;
* rstd relatively by dr = (L + 8) u + dm rstd, the second term because the
  deviations it squares carry dm;
* y by |w| (2 |h| (dr + 4 u) + 2 dm rstd) + 4 u |y|, and the rounding to bf16;
* dx by rstd (8 u (|g| + |c1| + |h c2|) + (L + 6) u (mean|g| + |h| mean|g h|))
  with c1 = mean(g), c2 = mean(g h), and the rounding to bf16;
* dweight by (rows + 8) u sum|dy h|, dbias by (rows + 8) u sum|dy|.
"""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from precision_mx_quantize_gb300 import mxq
from tests.libutil import ensure_built, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _f(t):
    return to_np(t.float()).astype(np.float64)


def _inputs(rows, cols, dt, wdt, seed, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.5 * torch.randn(1, cols, generator=g))
    x = (x + offset * torch.randn(rows, 1, generator=g)).to(dt)
    w = (1 + 0.1 * torch.randn(cols, generator=g)).to(wdt)
    b = (0.1 * torch.randn(cols, generator=g)).to(wdt)
    dy = torch.randn(rows, cols, generator=g).to(dt)
    return x, w, b, dy


def _call(kind, x, w, b, fused=False, fmt="e4m3"):
    x, w = x.cuda(), w.cuda()
    b = None if b is None else b.cuda()
    if kind == "layer":
        return (mxq.layer_norm_quantize(x, w, b, EPS, fmt) if fused
                else mxq.layer_norm(x, w, b, EPS))
    if fused:
        c, s, rstd = mxq.rms_norm_quantize(x, w, EPS, fmt)
        return c, s, None, rstd
    y, rstd = mxq.rms_norm(x, w, EPS)
    return y, None, rstd


def _chain(cols):
    return cols / 32 + 64


def _bounds(x, w, b, kind):
    """float64 (y, mean, rstd) and the bounds of y, mean and the relative one of rstd."""
    xn, wn = _f(x), _f(w)
    y, mean, rstd = F.norm(xn, wn, None if b is None else _f(b), EPS, kind)
    L = _chain(xn.shape[1])
    dm = (L + 2) * U * np.abs(xn).mean(1) if kind == "layer" else np.zeros(xn.shape[0])
    dr = (L + 8) * U + dm * rstd
    h = np.abs((xn - mean[:, None] if kind == "layer" else xn) * rstd[:, None])
    ty = np.abs(wn) * (2 * h * (dr + 4 * U)[:, None] + 2 * (dm * rstd)[:, None]) + 4 * U * np.abs(y)
    if b is not None:
        ty += 4 * U * np.abs(_f(b))
    return y, mean, rstd, ty, dm, dr


SIZES = [(1, 1), (1, 8), (2, 7), (3, 64), (5, 129), (7, 1000), (33, 1024), (4, 1001), (9, 4096),
         (3, 8200), (2, 16384), (2, 16392), (2, 20001), (1, 40000), (700, 256), (301, 2048)]
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
         (torch.float32, torch.bfloat16), (torch.float32, torch.float32)]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, types, kind):
    x, w, b, _ = _inputs(*size, *types, seed=sum(size))
    for bias in ((None, b) if kind == "layer" else (None,)):
        y, mean, rstd = _call(kind, x, w, bias)
        mxq.check()
        ey, em, er, ty, dm, dr = _bounds(x, w, bias, kind)
        if types[0] is torch.bfloat16:
            ty = ty + 2.0 ** -8 * (np.abs(ey) + ty)
        assert y.dtype == x.dtype
        assert (np.abs(_f(y) - ey) <= ty).all()
        assert (np.abs(_f(rstd) - er) <= dr * er).all()
        if kind == "layer":
            assert (np.abs(_f(mean) - em) <= dm).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("types", TYPES[:1] + TYPES[3:], ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward_to_codes(size, types, fmt, kind):
    # the codes stand for a value within a code step of y: the scale is that of
    # y's amax within its bound, each code a rounding of y / scale within it
    x, w, b, _ = _inputs(*size, *types, seed=sum(size))
    b = b if kind == "layer" else None
    c, s, mean, rstd = _call(kind, x, w, b, True, fmt)
    mxq.check()
    rows, cols = size
    ey, _, er, ty, _, dr = _bounds(x, w, b, kind)
    assert (np.abs(_f(rstd) - er) <= dr * er).all()
    cs, ss = mxq.fp8_shapes(rows, cols)
    assert tuple(c.shape) == cs and tuple(s.shape) == ss
    assert (to_np(c)[:, cols:] == 0).all()
    assert (to_np(s)[:, rows:] == F.TINY).all()
    fmax = {"e4m3": 448.0, "e5m2": 57344.0}[fmt]
    pad = F.up(cols, 128) - cols
    blocks = lambda t: np.pad(t, ((0, 0), (0, pad))).reshape(rows, -1, 128)
    amax, tmax = np.abs(blocks(ey)).max(2), blocks(ty).max(2)
    sc = to_np(s)[:, :rows].T.astype(np.float64)
    assert (np.abs(sc - np.maximum(amax / fmax, F.TINY)) <= tmax / fmax + 2 * U * sc).all()
    got = F.values(to_np(c), to_np(s), cols, fmt, "line")
    full = np.repeat(sc, 128, 1)[:, :cols]
    # half a step of a code at |y|: relative 2^-4 (E4M3), 2^-3 (E5M2), or half
    # the subnormal step 2^-9 / 2^-16 times the scale
    rel, sub = {"e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}[fmt]
    tol = np.maximum(rel * (np.abs(ey) + ty), sub * full) + ty + 4 * U * np.abs(ey)
    assert (np.abs(got - ey) <= tol).all()


def test_fused_codes_are_the_quantizers_on_exact_values():
    # rows of +-1 with weight 1 and RMS norm: rstd rounds once, every |y| is the
    # same fp32 value, and the codes are +-448 exactly
    x = torch.ones(5, 300).to(torch.bfloat16)
    x[:, ::3] = -1
    c, s, rstd = mxq.rms_norm_quantize(x.cuda(), torch.ones(300, device="cuda"), 0.0)
    assert (to_np(c)[:, :300] == np.where(to_np(x.float()) > 0, 0x7E, 0xFE)).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES + [(3001, 128), (1100, 1001)], ids=str)
def test_backward(size, types, kind):
    x, w, _, dy = _inputs(*size, *types, seed=sum(size) + 1)
    rows, cols = size
    _, em, er = F.norm(_f(x), _f(w), None, EPS, kind)
    rstd = torch.from_numpy(er.astype(np.float32)).cuda()
    if kind == "layer":
        mean = torch.from_numpy(em.astype(np.float32)).cuda()
        dx, dw, db = mxq.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    else:
        mean = None
        dx, dw = mxq.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), rstd)
    mxq.check()
    xn, dyn, wn, rn = _f(x), _f(dy), _f(w), _f(rstd)
    mn = None if mean is None else _f(mean)
    edx, edw, edb = F.norm_backward(dyn, xn, wn, mn, rn, kind)
    L = _chain(cols)
    h = (xn - mn[:, None] if kind == "layer" else xn) * rn[:, None]
    g = dyn * wn
    c1 = g.mean(1, keepdims=True) if kind == "layer" else 0.0
    c2 = (g * h).mean(1, keepdims=True)
    t = rn[:, None] * (8 * U * (np.abs(g) + np.abs(c1) + np.abs(h * c2)) + (L + 6) * U * (
        np.abs(g).mean(1, keepdims=True) + np.abs(h) * np.abs(g * h).mean(1, keepdims=True)))
    if types[0] is torch.bfloat16:
        t = t + 2.0 ** -8 * (np.abs(edx) + t)
    assert dx.dtype == x.dtype and dw.dtype == torch.float32
    assert (np.abs(_f(dx) - edx) <= t).all()
    assert (np.abs(_f(dw) - edw) <= (rows + 8) * U * np.abs(dyn * h).sum(0)).all()
    if kind == "layer":
        assert (np.abs(_f(db) - edb) <= (rows + 8) * U * np.abs(dyn).sum(0)).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradients_against_differences(kind):
    # central differences of the float64 forward pass, step d: their error is
    # O(d^2) third derivatives, below 1e-7 here; the GPU's statistics are those
    # of its own forward pass, whose fp32 errors the backward bound covers
    rows, cols, d = 3, 24, 1e-4
    x, w, b, dy = _inputs(rows, cols, torch.float32, torch.float32, 4)
    y, mean, rstd = _call(kind, x, w, b if kind == "layer" else None)
    if kind == "layer":
        dx, dw, db = mxq.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    else:
        dx, dw = mxq.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), rstd)
    mxq.check()
    xn, wn, bn, dyn = _f(x), _f(w), _f(b), _f(dy)

    def loss(xv, wv, bv):
        return (F.norm(xv, wv, bv if kind == "layer" else None, EPS, kind)[0] * dyn).sum()

    def diff(of, args):
        out = np.zeros(args[of].shape)
        for i in np.ndindex(out.shape):
            lo, hi = [a.copy() for a in args], [a.copy() for a in args]
            hi[of][i] += d
            lo[of][i] -= d
            out[i] = (loss(*hi) - loss(*lo)) / (2 * d)
        return out

    args = [xn, wn, bn]
    np.testing.assert_allclose(_f(dx), diff(0, args), rtol=0, atol=2e-5)
    np.testing.assert_allclose(_f(dw), diff(1, args), rtol=0, atol=2e-5)
    if kind == "layer":
        np.testing.assert_allclose(_f(db), diff(2, args), rtol=0, atol=2e-5)


def test_large_common_offset():
    # a mean 1000 times the deviation: the variance is taken about the mean
    x, w, b, _ = _inputs(4, 4096, torch.float32, torch.float32, 2, offset=0.0)
    x = x + 1000.0
    y, mean, rstd = _call("layer", x, w, b)
    ey, _, er, ty, _, dr = _bounds(x, w, b, "layer")
    assert (np.abs(_f(y) - ey) <= ty).all() and (np.abs(_f(rstd) - er) <= dr * er).all()


def test_constant_rows_and_zero_eps():
    x = torch.full((3, 256), 2.5).to(torch.bfloat16).cuda()
    w = torch.ones(256, device="cuda")
    y, mean, rstd = mxq.layer_norm(x, w, None, EPS)
    assert (y == 0).all() and (mean == 2.5).all()
    np.testing.assert_allclose(to_np(rstd), EPS ** -0.5, rtol=4 * U * 2)
    y, rstd = mxq.rms_norm(x, w, 0.0)
    assert (to_np(rstd) == np.float32(0.4)).all() and (y == 1).all()


def test_non_finite_rows_stay_in_their_row():
    x, w, b, dy = _inputs(6, 520, torch.bfloat16, torch.float32, 8)
    x[2, 5], x[4, 100] = float("nan"), float("inf")
    y, mean, rstd = _call("layer", x, w, b)
    bad = torch.tensor([False, False, True, False, True, False])
    assert torch.equal(y.isfinite().all(1).cpu(), ~bad)
    c, s, _, _ = _call("layer", x, w, b, True)
    assert s[:, :6].isnan().all(0).cpu().equal(bad) and (c[bad.cuda()] == 0).all()
    dx, _, _ = mxq.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    assert torch.equal(dx.isfinite().all(1).cpu(), ~bad)


def test_empty():
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    y, mean, rstd = mxq.layer_norm(x, w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = mxq.layer_norm_backward(x, x, w, mean, rstd)
    assert (dw == 0).all() and (db == 0).all()
    z = torch.empty(3, 0, device="cuda", dtype=torch.bfloat16)
    mxq.rms_norm(z, torch.empty(0, device="cuda"))
    mxq.check()


def test_same_inputs_give_the_same_bits():
    x, w, b, dy = (t.cuda() for t in _inputs(777, 1544, torch.bfloat16, torch.float32, 8))
    y, mean, rstd = mxq.layer_norm(x, w, b)
    first = mxq.layer_norm_backward(dy, x, w, mean, rstd)
    for _ in range(3):
        again = mxq.layer_norm_backward(dy, x, w, mean, rstd)
        assert all(torch.equal(p, q) for p, q in zip(first, again))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("size", [(5, 64), (9, 1001), (2000, 2048), (1300, 4096), (6, 9000),
                                  (7, 20001), (4, 20000)], ids=str)
def test_in_place(size, dt):
    # y over x, dx over dy or x: the bits of separate buffers
    x, w, b, dy = (t.cuda() for t in _inputs(*size, dt, torch.float32, seed=3))
    y, mean, rstd = mxq.layer_norm(x, w, b)
    want = mxq.layer_norm_backward(dy, x, w, mean, rstd)
    for over in ("dy", "x"):
        t = {"dy": dy.clone(), "x": x.clone()}
        got = mxq.layer_norm_backward(t["dy"], t["x"], w, mean, rstd, out=t[over])
        assert got[0] is t[over]
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    t = x.clone()
    assert torch.equal(mxq.layer_norm(t, w, b, out=t)[0], y)
    mxq.check()


# Rows that start between 16-byte boundaries: enough of them for the persistent
# kernels, every place of the last chunk and of the last 16-byte word.
ODD = [(1000, 4097), (4900, 1003), (700, 8190), (3, 16383), (307, 15000)]
ODD += [(9, c) for c in range(513, 521)] + [(3, c) for c in range(9, 17)]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("types", [TYPES[1], TYPES[2]], ids=str)
@pytest.mark.parametrize("size", ODD, ids=str)
def test_unaligned_rows(size, types, kind):
    test_forward(size, types, kind)
    test_forward_to_codes(size, types, "e4m3", kind)
    test_backward(size, types, kind)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=str)
def test_unaligned_rows_leave_their_surroundings(dt):
    # x in a longer buffer: NaN right behind it changes nothing, and y and dx in
    # one write nothing behind them
    for rows, cols in ((1000, 4097), (9, 517), (12, 1001), (5, 77)):
        x, w, b, dy = (t.cuda() for t in _inputs(rows, cols, dt, torch.float32, seed=4))
        n = rows * cols

        def inside(t, value):
            long = torch.full((n + 64,), value, device="cuda", dtype=dt)
            long[:n] = t.flatten()
            return long, long[:n].view(rows, cols)

        y, mean, rstd = mxq.layer_norm(x, w, b)
        want = mxq.layer_norm_backward(dy, x, w, mean, rstd)
        (_, xl), (_, dyl) = inside(x, float("nan")), inside(dy, float("nan"))
        (yb, yl), (db, dl) = inside(x, 7.0), inside(x, 7.0)
        assert torch.equal(mxq.layer_norm(xl, w, b, out=yl)[0], y)
        got = mxq.layer_norm_backward(dyl, xl, w, mean, rstd, out=dl)
        mxq.check()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert (yb[n:] == 7).all() and (db[n:] == 7).all()
