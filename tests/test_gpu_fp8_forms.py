"""Every kernel of the block-128 FP8 product by name, whatever sizes the library
would choose it for: a few lines of A (pairs 0), 256x256 tiles with one to four
CTA pairs each.  Every element of C and the memory behind it; the bound is the
one of the other product tests."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from precision_mx_quantize_gb300 import mxq
from tests.libutil import ensure_built
from tests.test_gpu_fp8 import _operands
from tests.test_gpu_fp8_whole import check_whole, guarded

pytestmark = pytest.mark.gpu
FORMS = (0, 1, 2, 3, 4)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def call(t, m, n, k, fa, fb, kind, out, pairs):
    """mxq_debug_fp8_gemm on CUDA tensors (codes A, scales A, codes B, scales B)."""
    p = [x.data_ptr() for x in t]
    return mxq.lib().mxq_debug_fp8_gemm(
        p[0], p[1], mxq.FP8_FMTS[fa], p[2], p[3], mxq.FP8_FMTS[fb], mxq.B_SCALES[kind], m, n, k,
        out.data_ptr(), mxq._out_code(out.dtype), pairs, mxq._stream(out.get_device()))


def check_forms(m, n, k, fa, fb, kind, forms=FORMS, ops=None):
    ops = _operands(m, n, k, fa, fb, kind, m + n + k) if ops is None else ops
    t = [torch.from_numpy(np.ascontiguousarray(o)).cuda() for o in ops]
    ref, S = F.gemm(F.values(ops[0], ops[1], k, fa, "line"), F.values(ops[2], ops[3], k, fb, kind))
    for pairs in forms:
        for dtype in (torch.bfloat16, torch.float32):
            long, c = guarded(m, n, dtype)
            assert call(t, m, n, k, fa, fb, kind, c, pairs) == 0, pairs
            check_whole(c, long, ref, S, k)
            again = torch.empty_like(c)
            call(t, m, n, k, fa, fb, kind, again, pairs)
            assert torch.equal(again, c), pairs   # sums in a fixed order


# rows of C: odd, even, 8- and 16-byte multiples; N mod 256 of 1, 81, 127, 129,
# 255 and whole tiles; odd and even M on both sides of a tile's halves
SHAPES = [(300, 513, 600), (257, 593, 1100), (130, 383, 512), (512, 641, 700), (511, 511, 515),
          (129, 770, 1000), (385, 516, 520), (256, 520, 1111), (256, 512, 1024), (1, 257, 640)]


@pytest.mark.parametrize("kind", ["tile", "line"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forms(shape, kind):
    check_forms(*shape, "e4m3", "e4m3", kind)


@pytest.mark.parametrize("kind", ["tile", "line"])
@pytest.mark.parametrize("fmts", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")], ids=str)
def test_forms_of_mixed_formats(fmts, kind):
    check_forms(300, 641, 1000, *fmts, kind)
    check_forms(260, 264, 530, *fmts, kind)


@pytest.mark.parametrize("kind", ["tile", "line"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 300, 128), (300, 1, 200), (257, 257, 100)],
                         ids=lambda s: "x".join(map(str, s)))
def test_forms_of_few_k_blocks(shape, kind):
    kb = (shape[2] + 127) // 128
    check_forms(*shape, "e4m3", "e4m3", kind, [f for f in FORMS if f <= kb])


# more tiles than CTA pairs: every pair takes several in turn
@pytest.mark.parametrize("kind", ["tile", "line"])
@pytest.mark.parametrize("shape", [(2300, 2305, 260), (2303, 2423, 300), (2304, 2308, 200),
                                   (2304, 2312, 300)], ids=lambda s: "x".join(map(str, s)))
def test_forms_of_many_tiles(shape, kind):
    check_forms(*shape, "e4m3", "e4m3", kind, (0, 1))


def test_refused_forms():
    z = [torch.zeros(4096, dtype=torch.uint8, device="cuda"), torch.ones(64, device="cuda")] * 2
    out = torch.empty(3, 5, device="cuda")
    for pairs in (-1, 5):
        assert call(z, 3, 5, 128, "e4m3", "e4m3", "tile", out, pairs) == 1
    assert call(z, 3, 5, 128, "e4m3", "e4m3", "tile", out, 2) == 1   # one K block
    assert call(z, 3, 5, 0, "e4m3", "e4m3", "tile", out, 2) == 0     # no K block: zeros
    mxq.check()
    assert (out == 0).all()
    assert mxq.lib().mxq_debug_fp8_gemm(None, None, 0, None, None, 0, 0, 3, 5, 128,
                                        ctypes.c_void_p(out.data_ptr()), 0, 1, None) == 1
