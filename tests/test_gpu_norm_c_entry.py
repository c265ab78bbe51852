"""mxq_norm_forward in the forms that the header promises and no tensor-level
helper takes, against float64 within the bounds of the other norm tests."""

import numpy as np
import pytest
import torch

from precision_mx_quantize_gb300 import mxq
from tests.libutil import ensure_built
from tests.test_gpu_norm import EPS, TYPES, _bounds, _f, _inputs

pytestmark = pytest.mark.gpu
KINDS = {"layer": mxq.NORM_LAYER, "rms": mxq.NORM_RMS}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _forward(kind, x, w, b, with_y, fmt):
    """(y, codes, scales, rstd) on the GPU, those not asked for None."""
    rows, cols = x.shape
    code = {torch.bfloat16: mxq.OUT_BF16, torch.float32: mxq.OUT_F32}
    ptr = lambda t: 0 if t is None else t.data_ptr()
    y = torch.empty_like(x) if with_y else None
    codes, scales = mxq._fp8_buffers(rows, cols, "line", x.device) if fmt else (None, None)
    rstd = torch.empty(rows, device="cuda")
    a = mxq._NORM_ARGS.pack(ptr(x), ptr(w), ptr(b), ptr(y), 0, ptr(rstd), ptr(codes), ptr(scales),
                            rows, cols, EPS, KINDS[kind], code[x.dtype], code[w.dtype],
                            mxq.FP8_FMTS[fmt] if fmt else 0)
    assert mxq.mxq_norm_forward(a, mxq._stream(x.get_device())) == 0
    mxq.check()
    return y, codes, scales, rstd


# a warp a row, a CTA a row, the ring, rows that one CTA reads again; aligned and not
SIZES = [(5, 64), (9, 1001), (7, 4096), (3000, 1024), (1300, 4096), (700, 4097), (2, 16392),
         (2, 20001)]


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_rms_norm_with_a_bias(size, types):
    x, w, b, _ = _inputs(*size, *types, seed=sum(size))
    b = b + 3.0   # larger than any rounding of y
    y, _, _, rstd = _forward("rms", x.cuda(), w.cuda(), b.cuda(), True, None)
    ey, _, er, ty, _, dr = _bounds(x, w, b, "rms")
    if types[0] is torch.bfloat16:
        ty = ty + 2.0 ** -8 * (np.abs(ey) + ty)
    assert (np.abs(_f(y) - ey) <= ty).all()
    assert (np.abs(_f(rstd) - er) <= dr * er).all()


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_rms_norm_with_a_bias_to_codes(size):
    # each code is within half a step of y / scale (E4M3: 2^-4 |y|, or half the
    # subnormal step 2^-9 times the scale)
    from oracle import fp8_oracle as F
    from tests.libutil import to_np
    x, w, b, _ = _inputs(*size, torch.bfloat16, torch.float32, seed=sum(size))
    b = b + 3.0
    _, codes, scales, _ = _forward("rms", x.cuda(), w.cuda(), b.cuda(), False, "e4m3")
    ey, _, _, ty, _, _ = _bounds(x, w, b, "rms")
    got = F.values(to_np(codes), to_np(scales), size[1], "e4m3", "line")
    step = np.repeat(to_np(scales)[:, :size[0]].T.astype(np.float64), 128, 1)[:, :size[1]]
    tol = np.maximum(2.0 ** -4 * (np.abs(ey) + ty), 2.0 ** -10 * step) + ty + 4 * 2.0 ** -24 * np.abs(ey)
    assert (np.abs(got - ey) <= tol).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("types", [TYPES[0], TYPES[3]], ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_output_and_codes_from_one_call(size, types, kind):
    # y within its bound, the codes those of the call that writes codes alone
    x, w, b, _ = _inputs(*size, *types, seed=sum(size))
    b = b if kind == "layer" else None
    xg, wg, bg = x.cuda(), w.cuda(), None if b is None else b.cuda()
    y, codes, scales, rstd = _forward(kind, xg, wg, bg, True, "e4m3")
    ey, _, er, ty, _, dr = _bounds(x, w, b, kind)
    if types[0] is torch.bfloat16:
        ty = ty + 2.0 ** -8 * (np.abs(ey) + ty)
    assert (np.abs(_f(y) - ey) <= ty).all()
    assert (np.abs(_f(rstd) - er) <= dr * er).all()
    _, alone, alone_scales, _ = _forward(kind, xg, wg, bg, False, "e4m3")
    assert torch.equal(codes, alone) and torch.equal(scales, alone_scales)
