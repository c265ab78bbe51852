"""The product with scales at the ends of their range, in every kernel.

Where the product of the two scales of a block is a normal fp32 value, the bound
of the other product tests holds.  Below, that product may have been rounded to
a multiple of 2^-149, so an output may be off by 2^-150 times the sum of its
blocks' |codes' products|; zeros stay zeros.  Subnormal results add half a
subnormal step, 2^-150, for each rounding."""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from precision_mx_quantize_gb300 import mxq
from tests.libutil import ensure_built, to_np
from tests.test_gpu_fp8_forms import FORMS, call
from tests.test_gpu_fp8_whole import guarded

pytestmark = pytest.mark.gpu
M, N, K = 270, 330, 520
KB, LINES_A, LINES_B = 5, 272, 332


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _check(A, sA, B, sB, fmt, kind, below=False):
    t = [torch.from_numpy(o).cuda() for o in (A, sA, B, sB)]
    ref, S = F.gemm(F.values(A, sA, K, fmt, "line"), F.values(B, sB, K, fmt, kind))
    # two multiplications and an addition a block, and C's own rounding
    tol = (K + K / 128 + 4) * 2.0 ** -23 * S + (3 * KB + 1) * 2.0 ** -150
    if below:
        tol = tol + 2.0 ** -150 * F.gemm(F.values(A, np.ones_like(sA), K, fmt, "line"),
                                         F.values(B, np.ones_like(sB), K, fmt, kind))[1]
    for pairs in FORMS:
        for dtype in (torch.bfloat16, torch.float32):
            long, c = guarded(M, N, dtype)
            assert call(t, M, N, K, fmt, fmt, kind, c, pairs) == 0
            mxq.check()
            got, bound = to_np(c.float()).astype(np.float64), tol
            if dtype is torch.bfloat16:
                bound = tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -134
            bad = ~(np.abs(got - ref) <= bound)
            assert not bad.any(), (pairs, dtype, int(bad.sum()), np.argwhere(bad)[0])
            assert (long[M * N:] == 7).all()


def _tiny(rng, fmt, kind, low, high):
    """Operands of one sign, so that a sum is as large as its terms, with scales of
    A from 2^-126 on beside ordinary ones (whole rows of either kind and rows that
    change from block to block) and scales of B from 2^low to 2^high."""
    top = {"e4m3": 0x7E, "e5m2": 0x7B}[fmt]
    A = rng.integers(top - 40, top + 1, (M, 528)).astype(np.uint8)
    B = rng.integers(top - 40, top + 1, (N, 528)).astype(np.uint8)
    sA = (2.0 ** -126 * (1 + rng.random((KB, LINES_A)))).astype(np.float32)
    sA[:, 100:150] = 0.01
    sA[:, 150:] = np.where(rng.random((KB, LINES_A - 150)) < 0.5, sA[:, 150:], np.float32(2.0 ** -100))
    shape = (KB, LINES_B) if kind == "line" else ((N + 127) // 128, KB)
    sB = (2.0 ** rng.integers(low, high, shape) * (1 + rng.random(shape))).astype(np.float32)
    return A, sA, B, sB


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["tile", "line"])
def test_smallest_products_of_scales(kind, fmt):
    rng = np.random.default_rng(3)
    _check(*_tiny(rng, fmt, kind, 0, 8), fmt, kind)           # 2^-126 and more
    _check(*_tiny(rng, fmt, kind, -24, -16), fmt, kind, True)  # 2^-150 and more


@pytest.mark.parametrize("kind", ["tile", "line"])
def test_largest_products_of_scales(kind):
    # products of up to 2^128; a row's block holds one code of 2^-9, or none, and
    # B's values are at most 1: C stays below 2^122
    rng = np.random.default_rng(4)
    A = np.zeros((M, 528), np.uint8)
    for kb in range(KB):
        at = kb * 128 + rng.integers(0, min(128, K - kb * 128), M)
        A[np.arange(M), at] = np.where(np.arange(M) % 5 == 0, 0, 1).astype(np.uint8)
    B = (rng.integers(0, 0x39, (N, 528)) | (rng.integers(0, 2, (N, 528)) << 7)).astype(np.uint8)
    sA = np.where(rng.random((KB, LINES_A)) < 0.5, 2.0 ** 87, 2.0 ** -60).astype(np.float32)
    shape = (KB, LINES_B) if kind == "line" else ((N + 127) // 128, KB)
    sB = (2.0 ** 40 * (1 + 0.5 * rng.random(shape))).astype(np.float32)
    _check(A, sA, B, sB, "e4m3", kind)


@pytest.mark.parametrize("pairs", FORMS)
def test_rows_of_zeros(pairs):
    # an all-zero block's scale, 2^-126, times a weight's is subnormal: zeros stay zeros
    g = torch.Generator().manual_seed(1)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    x[5:60], x[200], x[:, 128:256] = 0, 0, 0
    w = (0.02 * torch.randn(N, K, generator=g)).to(torch.bfloat16).cuda()
    a, b = mxq.fp8_quantize(x.cuda()), mxq.fp8_quantize_tiles(w)[:2]
    out = torch.empty(M, N, device="cuda")
    assert call([*a, *b], M, N, K, "e4m3", "e4m3", "tile", out, pairs) == 0
    mxq.check()
    assert (out[5:60] == 0).all() and (out[200] == 0).all()
    ref, S = F.gemm(F.values(to_np(a[0]), to_np(a[1]), K, "e4m3", "line"),
                    F.values(to_np(b[0]), to_np(b[1]), K, "e4m3", "tile"))
    assert (np.abs(to_np(out) - ref) <= (K + K / 128 + 4) * 2.0 ** -23 * S).all()
