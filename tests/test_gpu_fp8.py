"""The block-128 FP8 quantizers and their product on the GPU.

Quantizers: codes and scales equal to the oracle's, bit for bit (an amax is
exact whatever its order; the scale, its reciprocal and each product are single
fp32 operations).

Product: a term is scaled and added at most K times inside the tensor cores
and once per K block outside, so with u = 2^-23 per addition (truncation
allowed) an output is within (K + K / 128 + 4) u sum_k |a b| of the float64
product; bf16 output adds its rounding: 8 significant bits, 2^-8 |C|.
"""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from precision_mx_quantize_gb300 import mxq, synth
from tests.libutil import bf16_to_f32_np, ensure_built, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


SIZES = [(1, 1), (1, 128), (1, 4096), (3, 130), (4, 16), (127, 129), (128, 128), (129, 257),
         (130, 8), (300, 1001), (257, 136), (5, 1000)]


def _input(rows, cols, seed):
    """Heavy tails, an all-zero stretch, tiny and huge values, signed zeros."""
    rng = np.random.default_rng(seed)
    x = rng.standard_t(3, size=(rows, cols)) * np.exp(2 * rng.standard_normal((1, cols)))
    x[:, cols // 3:cols // 2] *= 0.0
    x[: rows // 2, -1] *= 1e-38
    x[rows // 2:, 0] *= 1e36
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def _eq(got, want):
    for g, w in zip(got, want):
        g = to_np(g)
        assert g.shape == w.shape and g.dtype == w.dtype
        np.testing.assert_array_equal(g, w)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_quantizers_match_the_definition(size, fmt):
    x = _input(*size, seed=sum(size))
    xn, xg = bf16_to_f32_np(x), x.cuda()
    row, col = F.quantize_lines(xn, fmt), F.quantize_lines(np.ascontiguousarray(xn.T), fmt)
    _eq(mxq.fp8_quantize(xg, "row", fmt), row)
    _eq(mxq.fp8_quantize(xg, "col", fmt), col)
    _eq(mxq.fp8_quantize_dual(xg, fmt, fmt), row + col)
    _eq(mxq.fp8_quantize_tiles(xg, fmt), F.quantize_tiles(xn, fmt))
    codes, scales, ct, st = mxq.fp8_quantize_tiles(
        xg, fmt, out=tuple(t.cuda() for t in (torch.empty(mxq.fp8_shapes(*size, "tile")[0],
                                                          dtype=torch.uint8),
                                              torch.empty(mxq.fp8_shapes(*size, "tile")[1])))
        + (None, None))
    assert ct is None and st is None
    _eq((codes, scales), F.quantize_tiles(xn, fmt)[:2])
    mxq.check()


def test_dual_takes_a_format_per_layout():
    x = _input(130, 260, 3)
    xn = bf16_to_f32_np(x)
    for fr, fc in (("e4m3", "e5m2"), ("e5m2", "e4m3")):
        _eq(mxq.fp8_quantize_dual(x.cuda(), fr, fc),
            F.quantize_lines(xn, fr) + F.quantize_lines(np.ascontiguousarray(xn.T), fc))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_blocks(value):
    # one bad element spoils its own row block, column block and tile only
    x = synth.activation(260, 300, 5)
    x[140, 131] = value
    xn, xg = bf16_to_f32_np(x), x.cuda()
    got = mxq.fp8_quantize_dual(xg)
    _eq(got, F.quantize_lines(xn, "e4m3") + F.quantize_lines(np.ascontiguousarray(xn.T), "e4m3"))
    assert int(got[1].isnan().sum()) == 1 and int(got[3].isnan().sum()) == 1
    tiles = mxq.fp8_quantize_tiles(xg)
    _eq(tiles, F.quantize_tiles(xn, "e4m3"))
    assert int(tiles[1].isnan().sum()) == 1
    # and reaches exactly the outputs that read it
    w = synth.weight(40, 300, 6)
    ws = mxq.fp8_quantize_tiles(w.cuda())
    c = mxq.fp8_gemm(got[0], got[1], ws[0], ws[1], 260, 40, 300, out_dtype=torch.float32)
    mxq.check()
    assert c[140].isnan().all() and int(c.isnan().any(1).sum()) == 1


def test_values_past_the_largest_code_saturate_to_it():
    # bf16's largest values: scale is finite, the block's maximum encodes as fmax
    x = torch.full((2, 128), 3.3895e38).to(torch.bfloat16)
    x[1] = -x[1]
    for fmt, code in (("e4m3", 0x7E), ("e5m2", 0x7B)):
        c, s = mxq.fp8_quantize(x.cuda(), "row", fmt)
        assert s[0, 0].isfinite()
        assert (to_np(c)[0] == code).all() and (to_np(c)[1] == (code | 0x80)).all()


def test_empty_tensors():
    for r, c in ((0, 64), (64, 0), (0, 0)):
        x = torch.empty(r, c, dtype=torch.bfloat16, device="cuda")
        mxq.fp8_quantize(x, "row")
        mxq.fp8_quantize(x, "col")
        mxq.fp8_quantize_dual(x)
        mxq.fp8_quantize_tiles(x)
    mxq.check()


# ---- the product ------------------------------------------------------------------

def _operands(m, n, k, fa, fb, kind, seed):
    rng = np.random.default_rng(seed)
    to = lambda a: bf16_to_f32_np(torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16))
    a = to(rng.standard_t(3, size=(m, k)) * np.exp(rng.standard_normal((1, k))))
    b = to(rng.standard_normal((n, k)) * 0.02 * np.exp(rng.standard_normal((n, 1))))
    A, sA = F.quantize_lines(a, fa)
    B, sB = F.quantize_lines(b, fb) if kind == "line" else F.quantize_tiles(b, fb)[:2]
    return A, sA, B, sB


def _product(ops, m, n, k, fa, fb, kind, out_dtype):
    t = [torch.from_numpy(np.ascontiguousarray(o)).cuda() for o in ops]
    c = mxq.fp8_gemm(*t, m, n, k, fmt_a=fa, fmt_b=fb, b_scales=kind, out_dtype=out_dtype)
    mxq.check()
    return to_np(c.float()).astype(np.float64)


def _check(ops, m, n, k, fa, fb, kind, out_dtype):
    A, sA, B, sB = ops
    ref, S = F.gemm(F.values(A, sA, k, fa, "line"), F.values(B, sB, k, fb, kind))
    got = _product(ops, m, n, k, fa, fb, kind, out_dtype)
    tol = (k + k / 128 + 4) * 2.0 ** -23 * S
    if out_dtype is torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[0])
    return got


GEMMS = [(1, 1, 1), (1, 128, 128), (1, 300, 1000), (2, 129, 144), (16, 256, 2048), (17, 40, 130),
         (33, 1001, 257), (64, 384, 512), (65, 130, 640), (128, 128, 384), (129, 257, 300),
         (200, 72, 1100), (256, 256, 256), (257, 520, 900), (400, 771, 1234), (513, 1024, 512)]


@pytest.mark.parametrize("kind", ["tile", "line"])
@pytest.mark.parametrize("shape", GEMMS, ids=lambda s: "x".join(map(str, s)))
def test_product_matches_float64(shape, kind):
    m, n, k = shape
    ops = _operands(m, n, k, "e4m3", "e4m3", kind, m + n + k)
    for out_dtype in (torch.float32, torch.bfloat16):
        _check(ops, m, n, k, "e4m3", "e4m3", kind, out_dtype)


@pytest.mark.parametrize("kind", ["tile", "line"])
@pytest.mark.parametrize("fmts", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")], ids=str)
@pytest.mark.parametrize("shape", [(5, 200, 300), (300, 520, 700), (700, 600, 400)], ids=str)
def test_product_of_mixed_formats(shape, fmts, kind):
    m, n, k = shape
    ops = _operands(m, n, k, *fmts, kind, 11)
    _check(ops, m, n, k, *fmts, kind, torch.float32)


# enough 256x256 tiles for the CTA-pair kernel: ragged rows and columns, odd N,
# rows of C that allow 32-byte, 16-byte and single-element stores, one K block
PAIRS = [(1500, 1296, 200), (257, 6200, 100), (2000, 1001, 130), (900, 1672, 300),
         (6200, 260, 520), (1792, 1028, 1111), (1600, 1024, 1)]


@pytest.mark.parametrize("kind", ["tile", "line"])
@pytest.mark.parametrize("shape", PAIRS, ids=lambda s: "x".join(map(str, s)))
def test_product_of_many_tiles(shape, kind):
    m, n, k = shape
    ops = _operands(m, n, k, "e4m3", "e4m3", kind, m + n + k)
    for out_dtype in (torch.float32, torch.bfloat16):
        _check(ops, m, n, k, "e4m3", "e4m3", kind, out_dtype)
    ops = _operands(m, n, k, "e5m2", "e4m3", kind, m)
    _check(ops, m, n, k, "e5m2", "e4m3", kind, torch.float32)


def test_bytes_past_k_are_not_read():
    m, n, k = 70, 150, 200
    ops = list(_operands(m, n, k, "e4m3", "e4m3", "tile", 2))
    want = _product(ops, m, n, k, "e4m3", "e4m3", "tile", torch.float32)
    for i in (0, 2):
        ops[i] = ops[i].copy()
        ops[i][:, k:] = 0x7F   # NaN codes between K and the pitch
    got = _product(ops, m, n, k, "e4m3", "e4m3", "tile", torch.float32)
    np.testing.assert_array_equal(got, want)


def test_degenerate_sizes():
    z = torch.zeros(128, dtype=torch.uint8, device="cuda")
    f = torch.zeros(64, device="cuda")
    assert mxq.fp8_gemm(z, f, z, f, 0, 5, 8).shape == (0, 5)
    assert mxq.fp8_gemm(z, f, z, f, 5, 0, 8).shape == (5, 0)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.full((3, 5), 7.0, dtype=dt, device="cuda")
        mxq.fp8_gemm(z, f, z, f, 3, 5, 0, out_dtype=dt, out=out)
        mxq.check()
        assert (out == 0).all()


@pytest.mark.parametrize("shape", [(3, 4100, 2000), (700, 1030, 1500)], ids=str)
def test_same_inputs_give_the_same_bits(shape):
    m, n, k = shape
    ops = _operands(m, n, k, "e4m3", "e4m3", "line", 9)
    first = _product(ops, m, n, k, "e4m3", "e4m3", "line", torch.float32)
    for _ in range(3):
        np.testing.assert_array_equal(
            _product(ops, m, n, k, "e4m3", "e4m3", "line", torch.float32), first)


def test_large_shapes_sampled():
    # the CUDA quantizers feed the CUDA product; sampled rows and columns in float64
    for m, n, k, kind in ((4096, 6144, 4096, "tile"), (6144, 2056, 1000, "line"),
                          (1500, 4096, 14336, "tile")):
        x, w = synth.activation(m, k, 1).cuda(), synth.weight(n, k, 2).cuda()
        A, sA = mxq.fp8_quantize(x)
        B, sB = mxq.fp8_quantize(w) if kind == "line" else mxq.fp8_quantize_tiles(w)[:2]
        c = mxq.fp8_gemm(A, sA, B, sB, m, n, k, b_scales=kind, out_dtype=torch.float32)
        mxq.check()
        rng = np.random.default_rng(m)
        ri, ci = np.sort(rng.choice(m, 97, False)), np.sort(rng.choice(n, 101, False))
        a = F.values(to_np(A), to_np(sA), k, "e4m3", "line")[ri]
        b = F.values(to_np(B), to_np(sB), k, "e4m3", kind)[ci]
        ref, S = F.gemm(a, b)
        got = to_np(c)[np.ix_(ri, ci)].astype(np.float64)
        assert (np.abs(got - ref) <= (k + k / 128 + 4) * 2.0 ** -23 * S).all()


def test_runs_on_the_current_stream():
    # operands made on a side stream and consumed there, with no host wait
    s = torch.cuda.Stream()
    x, w = synth.activation(600, 512, 1).cuda(), synth.weight(384, 512, 2).cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            A, sA = mxq.fp8_quantize(x)
            B, sB, _, _ = mxq.fp8_quantize_tiles(w)
            c = mxq.fp8_gemm(A, sA, B, sB, 600, 384, 512, out_dtype=torch.float32)
        s.synchronize()
    A, sA = mxq.fp8_quantize(x)
    B, sB, _, _ = mxq.fp8_quantize_tiles(w)
    assert torch.equal(c, mxq.fp8_gemm(A, sA, B, sB, 600, 384, 512, out_dtype=torch.float32))
    mxq.check()


# few tiles and a long K: two, three and four CTA pairs share a tile
SHARED = [(1024, 2100, 2900), (500, 2600, 1700), (300, 520, 4096), (257, 513, 2061), (700, 2049, 3600)]


@pytest.mark.parametrize("kind", ["tile", "line"])
@pytest.mark.parametrize("shape", SHARED, ids=lambda s: "x".join(map(str, s)))
def test_product_of_few_tiles_and_long_k(shape, kind):
    m, n, k = shape
    ops = _operands(m, n, k, "e4m3", "e5m2", kind, m + n)
    first = _check(ops, m, n, k, "e4m3", "e5m2", kind, torch.float32)
    _check(ops, m, n, k, "e4m3", "e5m2", kind, torch.bfloat16)
    assert np.array_equal(_product(ops, m, n, k, "e4m3", "e5m2", kind, torch.float32), first)
