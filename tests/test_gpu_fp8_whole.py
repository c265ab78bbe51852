"""The block-128 FP8 product, every element of C and the memory behind it.

Rows of C that no TMA store takes leave a tile in pieces: here they come in odd
and even numbers, with a last column tile whose right half holds a few columns,
one, or none.  The bound is the one of the other product tests: (K + K / 128 +
4) 2^-23 sum_k |a b|, and 2^-8 |C| for bf16.
"""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from precision_mx_quantize_gb300 import mxq
from tests.libutil import ensure_built, to_np
from tests.test_gpu_fp8 import _operands

pytestmark = pytest.mark.gpu
GUARD = 2048


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def guarded(m, n, dtype):
    """(a buffer of 7s, the [m, n] view at its start)."""
    long = torch.full((m * n + GUARD,), 7.0, device="cuda", dtype=dtype)
    return long, long[:m * n].view(m, n)


def check_whole(c, long, ref, S, k):
    """All of C within the bound, nothing written behind it."""
    mxq.check()
    got = to_np(c.float()).astype(np.float64)
    tol = (k + k / 128 + 4) * 2.0 ** -23 * S
    if c.dtype is torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0])
    assert (long[c.numel():] == 7).all()


@pytest.mark.parametrize("kind", ["tile", "line"])
@pytest.mark.parametrize("shape", [(2048, 4097, 300), (4096, 4097, 512), (4095, 4223, 512),
                                   (4096, 4177, 640)], ids=str)
def test_right_half_of_the_last_tile_past_n(shape, kind):
    m, n, k = shape
    ops = _operands(m, n, k, "e4m3", "e4m3", kind, m + n)
    t = [torch.from_numpy(np.ascontiguousarray(o)).cuda() for o in ops]
    ref, S = F.gemm(F.values(ops[0], ops[1], k, "e4m3", "line"),
                    F.values(ops[2], ops[3], k, "e4m3", kind))
    for dtype in (torch.bfloat16, torch.float32):
        long, c = guarded(m, n, dtype)
        mxq.fp8_gemm(*t, m, n, k, b_scales=kind, out_dtype=dtype, out=c)
        check_whole(c, long, ref, S, k)
