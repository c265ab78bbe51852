"""The binding refuses buffers whose rows have another length than the call reads
or writes them with (CPU; recorders in place of the library)."""

import pytest
import torch

from precision_mx_quantize_gb300 import mxq
from tests.test_fp8_checks import fake, lib   # noqa: F401  (fixtures)

BF = torch.bfloat16


def _operands(rows, k, axis="line"):
    cs, ss = mxq.fp8_shapes(rows, k, axis)
    return torch.zeros(cs, dtype=torch.uint8), torch.zeros(ss)


def test_buffers_of_another_row_length_are_refused(fake):
    x, v = torch.zeros(70, 130, dtype=BF), torch.ones(130)
    mean = rstd = torch.zeros(70)
    a, w, l = _operands(70, 130), _operands(60, 130, "tile"), _operands(60, 130)
    wide, more = _operands(70, 200), _operands(200, 130)
    dual = _operands(70, 130) + _operands(130, 70)
    tiles = _operands(70, 130, "tile") + _operands(130, 70, "tile")
    bad = {
        "codes of a longer K": lambda: mxq.fp8_gemm(wide[0], wide[1], *w, 70, 60, 130),
        "K shorter than the codes'": lambda: mxq.fp8_gemm(*a, *w, 70, 60, 128),
        "fewer lines than the scales'": lambda: mxq.fp8_gemm(a[0][:40], a[1], *w, 40, 60, 130),
        "codes of B": lambda: mxq.fp8_gemm(*a, wide[0], w[1], 70, 60, 130),
        "tile scales of B": lambda: mxq.fp8_gemm(*a, w[0], torch.zeros(1, 3), 70, 60, 130),
        "line scales of B": lambda: mxq.fp8_gemm(*a, l[0], more[1], 70, 60, 130, b_scales="line"),
        "C transposed": lambda: mxq.fp8_gemm(*a, *w, 70, 60, 130, out=torch.zeros(60, 70, dtype=BF)),
        "quantizer's codes": lambda: mxq.fp8_quantize(x, out=(wide[0], a[1])),
        "quantizer's scales": lambda: mxq.fp8_quantize(x, out=(a[0], more[1])),
        "both layouts": lambda: mxq.fp8_quantize_dual(x, out=dual[:2] + (dual[2].view(65, 160),
                                                                         dual[3])),
        "tiles": lambda: mxq.fp8_quantize_tiles(x, out=(tiles[0], tiles[1].t().contiguous())
                                                + tiles[2:]),
        "norm's output": lambda: mxq.layer_norm(x, v, out=torch.zeros(130, 70, dtype=BF)),
        "norm's codes": lambda: mxq.rms_norm_quantize(x, v, out=(wide[0], a[1])),
        "dy transposed": lambda: mxq.layer_norm_backward(torch.zeros(130, 70, dtype=BF), x, v,
                                                         mean, rstd),
        "dx transposed": lambda: mxq.rms_norm_backward(x, x, v, rstd,
                                                       out=torch.zeros(130, 70, dtype=BF)),
    }
    for name, f in bad.items():
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"{name} was accepted")
    assert not fake


def test_flat_and_longer_buffers_are_taken(fake):
    x, v = torch.zeros(70, 130, dtype=BF), torch.ones(130)
    a, w, l = _operands(70, 130), _operands(60, 130, "tile"), _operands(60, 130)
    more = torch.zeros(500, 144, dtype=torch.uint8)   # codes of more lines
    flat = lambda t: torch.zeros(t.numel() + 5, dtype=t.dtype)
    mxq.fp8_gemm(*a, *w, 70, 60, 130)
    mxq.fp8_gemm(more, a[1], more, w[1], 70, 60, 130)
    mxq.fp8_gemm(*map(flat, a + l), 70, 60, 130, b_scales="line", out=torch.zeros(9999, dtype=BF))
    mxq.fp8_gemm(*a, *w, 70, 60, 130, out=torch.zeros(80, 60, dtype=BF))
    mxq.fp8_quantize(x, out=tuple(map(flat, a)))
    mxq.layer_norm(x, v, out=torch.zeros(80, 130, dtype=BF))
    mxq.layer_norm_backward(torch.zeros(10, 7, 130, dtype=BF), x, v, torch.zeros(70),
                            torch.zeros(70), out=flat(x))
    b = _operands(9, 100)
    mxq.fp8_gemm(*_operands(70, 100), b[0], torch.tensor(1.0), 70, 9, 100)   # one tile's scale
    assert len(fake) == 8
