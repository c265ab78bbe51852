"""The pre-norm FP8 linear layer: its products against float64 products of the
operands they read, its result against the unquantized layer, and the example.

Against the unquantized layer: an E4M3 code is within 2^-4 of its value (half a
step of three mantissa bits; E5M2 2^-3), or half a subnormal step, 2^-10 of the
block's maximum over 448, which the sum over a block of 128 keeps far below the
first term for these inputs; the norm's bf16 rounding adds 2^-8.  So an element
of a product of a by b is within r sum |a b|, r = 2 * 2^-4 + 2^-8 + 2^-7 (the
product of both errors, and the subnormal codes), and 2^-8 |y| for its own
rounding."""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from precision_mx_quantize_gb300 import mxq, synth
from precision_mx_quantize_gb300.fp8_layer import Fp8NormLinear
from tests.libutil import ensure_built, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _f(t):
    return to_np(t.float()).astype(np.float64)


def _layer(kind, in_f, out_f, grad_fmt="e4m3"):
    g = torch.Generator().manual_seed(5)
    nw = (1 + 0.1 * torch.randn(in_f, generator=g)).cuda()
    nb = (0.1 * torch.randn(in_f, generator=g)).cuda() if kind == "layer" else None
    return Fp8NormLinear(synth.weight(out_f, in_f, 3).cuda(), nw, nb, kind, grad_fmt=grad_fmt)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("shape", [(1, 256, 384), (77, 130, 200), (700, 512, 640)], ids=str)
def test_forward_and_infer(shape, kind):
    tokens, in_f, out_f = shape
    layer = _layer(kind, in_f, out_f)
    x = synth.normal((tokens, in_f), 1).cuda()
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
    layer = _layer(kind, in_f, out_f, grad_fmt)
    x, dy = synth.normal((tokens, in_f), 1).cuda(), synth.out_grad(tokens, out_f, 2).cuda()
    y, saved = layer.forward(x)
    dx, dw, dnw, dnb = layer.backward(dy, saved)
    mxq.check()
    # the weight gradient: the float64 product of the operands it read, exactly
    # as the product's own bound has it
    hc, hcs = saved[3:]
    dc, dcs = mxq.fp8_quantize(dy, "col", grad_fmt)
    ref, S = F.gemm(F.values(to_np(dc), to_np(dcs), tokens, grad_fmt, "line"),
                    F.values(to_np(hc), to_np(hcs), tokens, "e4m3", "line"))
    assert (np.abs(_f(dw) - ref) <= (tokens + tokens / 128 + 4) * 2.0 ** -23 * S).all()
    # the norm's gradients: those of the dh that the input-gradient product gives
    dr, drs = mxq.fp8_quantize(dy, "row", grad_fmt)
    wt, wts = layer.operands[2:]
    dh = mxq.fp8_gemm(dr, drs, wt, wts, tokens, in_f, out_f, fmt_a=grad_fmt)
    ref, S = F.gemm(F.values(to_np(dr), to_np(drs), out_f, grad_fmt, "line"),
                    F.values(to_np(wt), to_np(wts), out_f, "e4m3", "tile"))
    tol = (out_f + out_f / 128 + 4) * 2.0 ** -23 * S
    assert (np.abs(_f(dh) - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol)).all()
    if kind == "layer":
        want = mxq.layer_norm_backward(dh, x, layer.norm_weight, saved[1], saved[2])
        assert torch.equal(dnb, want[2])
    else:
        want = mxq.rms_norm_backward(dh, x, layer.norm_weight, saved[2])
        assert dnb is None
    assert torch.equal(dx, want[0]) and torch.equal(dnw, want[1])


def test_requantize_follows_the_weight():
    layer = _layer("rms", 256, 128)
    x = synth.normal((9, 256), 1).cuda()
    before = layer.forward(x)[0]
    buffers = [t.data_ptr() for t in layer.operands]
    layer.weight.mul_(2.0)
    assert torch.equal(layer.forward(x)[0], before)   # the operands are those of the old weight
    layer.requantize()
    assert [t.data_ptr() for t in layer.operands] == buffers
    torch.testing.assert_close(layer.forward(x)[0], before * 2.0, rtol=0, atol=0)


def test_replays_in_a_graph():
    # no call allocates, synchronizes or reads on the host: a step records into
    # a CUDA graph, and a replay on new inputs gives what the calls give
    layer = _layer("layer", 384, 512)
    x, dy = synth.normal((200, 384), 1).cuda(), synth.out_grad(200, 512, 2).cuda()
    step = lambda: layer.backward(dy, layer.forward(x)[1]) + (layer.infer(x),)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(synth.normal((200, 384), 7).cuda())
    dy.copy_(synth.out_grad(200, 512, 8).cuda())
    graph.replay()
    want = step()
    mxq.check()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


def test_refusals():
    w = synth.weight(64, 128, 1).cuda()
    v = torch.ones(128, device="cuda")
    with pytest.raises(ValueError):
        Fp8NormLinear(w, v, kind="batch")
    with pytest.raises(ValueError):
        Fp8NormLinear(w, v, v, kind="rms")
    with pytest.raises(ValueError):
        Fp8NormLinear(w.float(), v)


def test_example_learns_and_serves():
    import runpy
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "fp8_norm_linear.py")
    losses, gap = runpy.run_path(path)["main"](steps=25)
    assert losses[-1] < 0.2 * losses[0] and gap < 0.05
