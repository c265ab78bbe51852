"""The pre-norm FP8 linear layer on an fp32 residual stream, within the bounds of
the bf16 one's tests (the norm's output is rounded to bf16 in both)."""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from precision_mx_quantize_gb300 import mxq, synth
from tests.libutil import ensure_built, to_np
from tests.test_gpu_fp8_layer import _f, _layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _x(tokens, in_f):
    g = torch.Generator().manual_seed(7)
    return torch.randn(tokens, in_f, generator=g).cuda()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("shape", [(1, 256, 384), (77, 130, 200), (700, 512, 640)], ids=str)
def test_forward_and_infer(shape, kind):
    tokens, in_f, out_f = shape
    layer, x = _layer(kind, in_f, out_f), _x(tokens, in_f)
    h = F.norm(_f(x), _f(layer.norm_weight),
               None if layer.norm_bias is None else _f(layer.norm_bias), layer.eps, kind)[0]
    ref, S = F.gemm(h, _f(layer.weight))
    tol = (2.0 ** -3 + 2.0 ** -8 + 2.0 ** -7) * S + 2.0 ** -8 * np.abs(ref)
    for y in (layer.forward(x)[0], layer.infer(x)):
        mxq.check()
        assert y.dtype == torch.bfloat16 and tuple(y.shape) == (tokens, out_f)
        assert (np.abs(_f(y) - ref) <= tol).all()


@pytest.mark.parametrize("kind, grad_fmt", [("rms", "e4m3"), ("layer", "e5m2")])
@pytest.mark.parametrize("shape", [(33, 130, 200), (600, 512, 384)], ids=str)
def test_backward(shape, kind, grad_fmt):
    tokens, in_f, out_f = shape
    layer, x = _layer(kind, in_f, out_f, grad_fmt), _x(tokens, in_f)
    dy = synth.out_grad(tokens, out_f, 2).cuda()
    y, saved = layer.forward(x)
    dx, dw, dnw, dnb = layer.backward(dy, saved)
    mxq.check()
    assert dx.dtype == torch.float32 and dx.shape == x.shape
    # the input gradient's product, in fp32, and the norm's gradients of it
    dr, drs = mxq.fp8_quantize(dy, "row", grad_fmt)
    wt, wts = layer.operands[2:]
    dh = mxq.fp8_gemm(dr, drs, wt, wts, tokens, in_f, out_f, fmt_a=grad_fmt,
                      out_dtype=torch.float32)
    ref, S = F.gemm(F.values(to_np(dr), to_np(drs), out_f, grad_fmt, "line"),
                    F.values(to_np(wt), to_np(wts), out_f, "e4m3", "tile"))
    assert (np.abs(_f(dh) - ref) <= (out_f + out_f / 128 + 4) * 2.0 ** -23 * S).all()
    if kind == "layer":
        want = mxq.layer_norm_backward(dh, x, layer.norm_weight, saved[1], saved[2])
        assert torch.equal(dnb, want[2])
    else:
        want = mxq.rms_norm_backward(dh, x, layer.norm_weight, saved[2])
        assert dnb is None
    assert torch.equal(dx, want[0]) and torch.equal(dnw, want[1])
    hc, hcs = saved[3:]
    dc, dcs = mxq.fp8_quantize(dy, "col", grad_fmt)
    ref, S = F.gemm(F.values(to_np(dc), to_np(dcs), tokens, grad_fmt, "line"),
                    F.values(to_np(hc), to_np(hcs), tokens, "e4m3", "line"))
    assert (np.abs(_f(dw) - ref) <= (tokens + tokens / 128 + 4) * 2.0 ** -23 * S).all()


def test_no_tokens():
    layer = _layer("layer", 256, 128)
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.empty(0, 256, device="cuda", dtype=dtype)
        y, saved = layer.forward(x)
        dx, dw, dnw, dnb = layer.backward(torch.empty(0, 128, device="cuda", dtype=torch.bfloat16), saved)
        mxq.check()
        assert y.shape == (0, 128) and dx.shape == (0, 256) and dx.dtype == dtype
        assert (dw == 0).all() and (dnw == 0).all() and (dnb == 0).all()
        assert layer.infer(x).shape == (0, 128)


def test_replays_in_a_graph():
    layer, x = _layer("rms", 384, 512), _x(200, 384)
    dy = synth.out_grad(200, 512, 2).cuda()
    step = lambda: layer.backward(dy, layer.forward(x)[1])[:3] + (layer.infer(x),)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.add_(0.5)
    dy.copy_(synth.out_grad(200, 512, 8).cuda())
    graph.replay()
    want = step()
    mxq.check()
    for a, b in zip(out, want):
        assert torch.equal(a, b)
