"""The linear layer of experts: its products against float64 products of the operands
they read, the run of its operators as a training step uses them, and the example.

A product's K additions inside the tensor cores are each within 2^-23 of the sum of
magnitudes S, and a bf16 result is rounded by at most 2^-8 of its value."""

import os
import runpy

import numpy as np
import pytest
import torch

from oracle import expert_oracle as E
from oracle import mx_oracle as O
from precision_mx_quantize_gb300 import mxq, synth
from precision_mx_quantize_gb300.expert_layer import MxExpertLinear
from tests.libutil import ensure_built, to_np

pytestmark = pytest.mark.gpu

EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                       "mx_experts.py")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _f(t):
    return to_np(t.float()).astype(np.float64)


def _layer(experts, out_f, in_f, **kw):
    return MxExpertLinear(synth.weight(experts * out_f, in_f, 3).cuda().view(experts, out_f, in_f),
                          **kw)


def _ids(tokens, topk, experts, seed):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(experts)[:topk] for _ in range(tokens)])
    return torch.from_numpy(ids).cuda()


def _near(got, ref, S, k, rounded=True):
    tol = (k + 4) * 2.0 ** -23 * S
    if rounded:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert (np.abs(_f(got) - ref) <= tol).all()


@pytest.mark.parametrize("kw", [{}, {"wgrad_fmt": "e2m1"}, {"fmt": "e2m1"}, {"fmt": "e5m2"}], ids=str)
@pytest.mark.parametrize("shape", [(1, 4, 1, 64, 96), (90, 5, 2, 256, 512), (300, 3, 3, 160, 32)],
                         ids=str)
def test_forward_and_backward(shape, kw):
    tokens, experts, topk, out_f, in_f = shape
    layer = _layer(experts, out_f, in_f, **kw)
    x = synth.normal((tokens, in_f), 1).cuda()
    rows, (row_of, offsets, counts) = layer.dispatch(x, _ids(tokens, topk, experts, 2))
    y, saved = layer.forward(rows, offsets)
    off, end = to_np(offsets).astype(np.int64), int(offsets[-1])
    assert (off % layer.align == 0).all()
    w = _f(layer.weight)
    code = lambda v, axis, fmt, had=False: O.quantize_any(v.astype(np.float32), axis, fmt, had)
    weights = [code(w[e], "row", layer.fmt) for e in range(experts)]
    A, sA = code(_f(rows)[:end], "row", layer.fmt)
    ref, S = E.experts_product(A, sA, [q[0] for q in weights], [q[1] for q in weights], off,
                               layer.fmt, np.zeros((end, out_f)))
    _near(y[:end], ref, S, in_f)
    one = layer.infer(rows, offsets)
    assert torch.equal(one[:end], y[:end])

    dy = synth.out_grad(rows.shape[0], out_f, 4).cuda()
    for e in range(experts):       # the gradient of padding is zeros, as the combine gives it
        dy[int(off[e]) + int(counts[e]):int(off[e + 1])] = 0
    drows, dw = layer.backward(dy, saved, offsets)
    mxq.check()
    weights = [code(w[e], "col", layer.fmt) for e in range(experts)]
    A, sA = code(_f(dy)[:end], "row", layer.fmt)
    ref, S = E.experts_product(A, sA, [q[0] for q in weights], [q[1] for q in weights], off,
                               layer.fmt, np.zeros((end, in_f)))
    _near(drows[:end], ref, S, out_f)
    had = layer.wgrad_fmt == "e2m1"
    a, sa = code(_f(dy)[:end], "col", layer.wgrad_fmt, had)
    b, sb = code(_f(rows)[:end], "col", layer.wgrad_fmt, had)
    ref, S = E.experts_wgrad(a, sa, b, sb, off, layer.wgrad_fmt)
    _near(dw, ref, S, end, rounded=False)


def test_a_step_in_a_graph():
    # dispatch, forward, combine, its gradients, backward, AdamW and the quantizers in one
    # graph: replays follow new tokens, choices and the step's number
    tokens, experts, topk, out_f, in_f = 64, 4, 2, 128, 256
    x = synth.normal((tokens, in_f), 1).cuda()
    ids, gates = _ids(tokens, topk, experts, 2), torch.rand(tokens, topk, device="cuda")
    target = synth.normal((tokens, out_f), 5).cuda()
    number = torch.zeros(1, dtype=torch.int64, device="cuda")

    def make():
        layer = _layer(experts, out_f, in_f)
        master = layer.weight.float()
        plan = mxq.adamw_plan([master], [mxq.adamw_state(master, 8)], weights=[layer.weight])

        def step():
            number.add_(1)
            rows, (row_of, offsets, counts) = layer.dispatch(x, ids)
            y, saved = layer.forward(rows, offsets)
            out = mxq.expert_combine(y, row_of, gates)
            dy, dgates = mxq.expert_combine_backward(out - target, y, row_of, offsets, counts, gates)
            drows, dw = layer.backward(dy, saved, offsets)
            dx = mxq.expert_combine(drows, row_of)
            mxq.adamw_step(plan, [dw], number, 1e-3)
            layer.requantize()
            return out, dgates, dx
        return step, master, layer

    eager, m1, l1 = make()
    captured, m2, l2 = make()
    captured()                       # warm
    m2.copy_(l1.weight.float())
    l2.weight.copy_(l1.weight)
    l2.requantize()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = m2.clone()
    with torch.cuda.graph(graph):
        out = captured()
    assert torch.equal(m2, keep)     # a capture runs nothing
    # the eager layer gets the captured one's weights before every step
    for seed in (3, 4, 5):
        x.copy_(synth.normal((tokens, in_f), seed))
        ids.copy_(_ids(tokens, topk, experts, seed))
        before = [m2.clone(), l2.weight.clone()]
        l1.weight.copy_(l2.weight)
        l1.requantize()
        number.fill_(seed)
        graph.replay()
        got = [t.clone() for t in out]
        number.fill_(seed)
        want = eager()
        mxq.check()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert not torch.equal(m2, before[0])


@pytest.mark.parametrize("shape", [(1, 64, 8, 64, 256), (13, 9, 4, 96, 160)], ids=str)
def test_a_servers_tokens_without_padding(shape):
    tokens, experts, topk, out_f, in_f = shape
    layer = _layer(experts, out_f, in_f)
    x, ids = synth.normal((tokens, in_f), 1).cuda(), _ids(tokens, topk, experts, 2)
    rows, (row_of, offsets, counts) = layer.dispatch(x, ids, padded=False)
    assert rows.shape == (tokens * topk, in_f)
    for t, j in np.ndindex(tokens, topk):
        assert torch.equal(rows[int(row_of[t, j])], x[t])
    y = layer.infer(rows, offsets)
    mxq.check()
    w = _f(layer.weight)
    q = [O.quantize_any(w[e].astype(np.float32), "row", "e4m3", False) for e in range(experts)]
    A, sA = O.quantize_any(_f(rows).astype(np.float32), "row", "e4m3", False)
    ref, S = E.experts_product(A, sA, [v[0] for v in q], [v[1] for v in q],
                               to_np(offsets).astype(np.int64), "e4m3", np.zeros((rows.shape[0], out_f)))
    _near(y, ref, S, in_f)


def test_requantize_follows_the_weights():
    layer = _layer(3, 64, 128)
    rows = synth.normal((32, 128), 1).cuda()
    offsets = torch.tensor([0, 10, 10, 32], dtype=torch.int32, device="cuda")
    before = layer.infer(rows, offsets)
    layer.weight.mul_(2.0)
    assert torch.equal(layer.infer(rows, offsets), before)
    layer.requantize()
    assert torch.equal(layer.infer(rows, offsets), before * 2.0)


def test_no_tokens_and_one_expert_with_all():
    layer = _layer(4, 64, 96)
    rows, (row_of, offsets, counts) = layer.dispatch(
        torch.empty(0, 96, dtype=torch.bfloat16, device="cuda"),
        torch.empty(0, 2, dtype=torch.int64, device="cuda"))
    y, saved = layer.forward(rows, offsets)
    drows, dw = layer.backward(y, saved, offsets)
    assert rows.shape == drows.shape == (0, 96) and dw.eq(0).all()
    assert mxq.expert_combine(y, row_of).shape == (0, 64)
    x = synth.normal((50, 96), 1).cuda()
    ids = torch.full((50, 1), 2, device="cuda")
    rows, (row_of, offsets, counts) = layer.dispatch(x, ids)
    y, saved = layer.forward(rows, offsets)
    _, dw = layer.backward(y, saved, offsets)
    mxq.check()
    assert offsets.tolist() == [0, 0, 0, 64, 64] and torch.equal(rows[:50], x)
    assert dw[[0, 1, 3]].eq(0).all() and dw[2].ne(0).any()


def test_refusals():
    w = torch.zeros(2, 64, 48, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        MxExpertLinear(w)
    with pytest.raises(ValueError):
        MxExpertLinear(w[0])
    with pytest.raises(ValueError):
        MxExpertLinear(torch.zeros(2, 64, 64, device="cuda"))


@pytest.mark.parametrize("bits", [8, 32])
def test_example_runs(bits):
    losses, gap = runpy.run_path(EXAMPLE)["main"](steps=3, bits=bits)
    assert len(losses) == 3 and np.isfinite(losses).all() and np.isfinite(gap)


def test_weight_gradient_of_a_sum_of_experts():
    # the gradient of sum_t <dout_t, sum_j gate W x_t> in float64, without any rounding, and the
    # layer's, whose operands are rounded to E4M3 (2^-4 each) and dy to bf16
    tokens, experts, topk, out_f, in_f = 60, 3, 2, 64, 128
    layer = _layer(experts, out_f, in_f)
    x = synth.normal((tokens, in_f), 1).cuda()
    ids, gates = _ids(tokens, topk, experts, 2), torch.rand(tokens, topk, device="cuda")
    rows, (row_of, offsets, counts) = layer.dispatch(x, ids)
    y, saved = layer.forward(rows, offsets)
    dout = synth.normal((tokens, out_f), 4).cuda()
    dy, _ = mxq.expert_combine_backward(dout, y, row_of, offsets, counts, gates)
    _, dw = layer.backward(dy, saved, offsets)
    mxq.check()
    xs, d, g = _f(x), _f(dout), _f(gates)
    choice, grad = to_np(ids), _f(dw)
    want, size = np.zeros_like(grad), np.zeros_like(grad)
    for (t, j), e in np.ndenumerate(choice):
        v = g[t, j] * np.outer(d[t], xs[t])
        want[e] += v
        size[e] += np.abs(v)
    # E4M3: 2^-4 per operand (and their product), bf16 dy 2^-8; codes below the smallest
    # normal one are off by 2^-10 of a block's maximum at most, which 32 rows keep within
    # another 2^-4 of these sums
    assert (np.abs(grad - want) <= (3 * 2.0 ** -4 + 2.0 ** -7) * size).all()
