"""Layers of experts on the GPU: the order of the choices, gather, combine and its
gradients, and the MX products grouped by expert, against plain definitions in
float64.

Tolerances.  bf16 holds eight significant bits: its step at 1 is 2^-7, so a rounding is
off by at most 2^-8 of the value.  The order is whole numbers: equal.  gather without
weights copies; with them one fp32 product (2^-24) and one rounding.  combine: k products
and additions in fp32, each within 2^-24 of a value below the sum S of magnitudes: 2 k
2^-24 S, and 2^-8 for bf16.  dweights: a fused product and addition per column and a tree
of additions: (cols + 16) 2^-24 S.  Products: K additions inside the tensor cores, each
within 2^-23 of the sum of magnitudes (a truncation is a whole step): (K + 4) 2^-23 S, and
2^-8 of the value for bf16."""

import numpy as np
import pytest
import torch

from oracle import expert_oracle as E
from oracle import mx_oracle as O
from precision_mx_quantize_gb300 import mxq, synth
from tests.libutil import ensure_built, to_np

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _f(t):
    return to_np(t.float()).astype(np.float64)


def _ids(tokens, topk, experts, seed, dropped=0.0):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, experts, (tokens, topk))
    ids[rng.random(ids.shape) < dropped] = -1
    return ids


# ---- order ------------------------------------------------------------------------

@pytest.mark.parametrize("wide", [False, True], ids=["int32", "int64"])
@pytest.mark.parametrize("case", [
    (0, 4, 8, 1), (1, 1, 1, 1), (1, 8, 64, 32), (3, 5, 2, 7), (1000, 3, 7, 32), (4096, 1, 33, 64),
    (4097, 1, 5, 1), (777, 8, 1024, 16), (30000, 8, 64, 32), (9001, 2, 1, 128)], ids=str)
def test_order(case, wide):
    tokens, topk, experts, align = case
    ids = _ids(tokens, topk, experts, tokens, dropped=0.1)
    if tokens > 2:
        ids[1, 0], ids[2, 0] = experts, 2 ** 31 - 1      # outside: no expert
    t = torch.from_numpy(ids).cuda().to(torch.int64 if wide else torch.int32)
    row_of, offsets, counts = mxq.expert_order(t, experts, align)
    mxq.check()
    want = E.order(ids, experts, align)
    for got, ref in zip((row_of, offsets, counts), want):
        assert got.dtype == torch.int32 and np.array_equal(to_np(got), ref)
    assert want[1][-1] <= mxq.expert_rows(ids.size, experts, align)


def test_order_of_ids_past_32_bits():
    ids = torch.tensor([[2 ** 32, 1], [-2 ** 40, 0]], device="cuda")
    row_of, offsets, counts = mxq.expert_order(ids, 2, 4)
    assert row_of.tolist() == [[-1, 4], [-1, 0]]
    assert offsets.tolist() == [0, 4, 8] and counts.tolist() == [1, 1]


# ---- gather, combine ------------------------------------------------------------------

ROWS = [(1, 1, 1, 1, 1), (1, 8, 64, 256, 1), (5, 3, 4, 33, 32), (40, 2, 3, 1001, 32),
        (33, 9, 16, 64, 16), (64, 17, 5, 8, 1), (7, 4, 1024, 4096, 2), (3, 2, 2, 5000, 32),
        (20, 5, 8, 72, 1), (900, 6, 6, 128, 32), (12, 7, 9, 4104, 1), (700, 8, 20, 264, 64)]


def _routing(tokens, topk, experts, align, seed):
    ids = _ids(tokens, topk, experts, seed, dropped=0.15)
    if tokens > 3:
        ids[3] = -1                       # a token that no expert takes
    got = mxq.expert_order(torch.from_numpy(ids).cuda(), experts, align)
    rows = mxq.expert_rows(ids.size, experts, align) + 3
    w = torch.from_numpy(np.random.default_rng(seed + 1).standard_normal(ids.shape)).float()
    w[torch.from_numpy(ids) < 0] = float("nan")      # a dropped choice's weight is not read
    return got, tuple(to_np(t).astype(np.int64) for t in got), rows, w.cuda()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", ROWS, ids=str)
def test_gather(case, dtype):
    tokens, topk, experts, cols, align = case
    dev, ref, rows, w = _routing(tokens, topk, experts, align, 7)
    x = synth.normal((tokens, cols), 1).cuda().to(dtype)
    before = torch.full((rows, cols), 7.0, dtype=dtype, device="cuda")
    for weights in (None, w):
        out = mxq.expert_gather(x, *dev, rows, weights=weights, out=before.clone())
        mxq.check()
        want = E.gather(_f(x), *ref, _f(before), None if weights is None else _f(weights))
        tol = 0.0 if weights is None else (2.0 ** -24 + HALF[dtype]) * np.abs(want) + 1e-38
        assert (np.abs(_f(out) - want) <= tol).all()
        assert (_f(out)[ref[1][-1]:] == 7.0).all()          # rows behind the last expert


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", ROWS, ids=str)
def test_combine_and_its_gradients(case, dtype):
    tokens, topk, experts, cols, align = case
    dev, ref, rows, w = _routing(tokens, topk, experts, align, 11)
    y = synth.normal((rows, cols), 2).cuda().to(dtype)
    dout = synth.normal((tokens, cols), 3).cuda().to(dtype)
    for weights in (None, w):
        wn = None if weights is None else _f(weights)
        out = mxq.expert_combine(y, dev[0], weights)
        want, size = E.combine(_f(y), ref[0], wn)
        tol = 2 * topk * 2.0 ** -24 * size + HALF[dtype] * np.abs(want) * (1 + 1e-6) + 1e-38
        assert (np.abs(_f(out) - want) <= tol).all()
        before = torch.full((rows, cols), 7.0, dtype=dtype, device="cuda")
        dy, dw = mxq.expert_combine_backward(dout, y, *dev, weights, out=before.clone())
        mxq.check()
        want = E.gather(_f(dout), *ref, _f(before), wn)
        assert (np.abs(_f(dy) - want) <= (2.0 ** -24 + HALF[dtype]) * np.abs(want) + 1e-38).all()
        want, size = E.combine_dweights(_f(dout), _f(y), ref[0])
        assert (np.abs(_f(dw) - want) <= (cols + 16) * 2.0 ** -24 * size).all()
        again = mxq.expert_combine_backward(dout, y.clone(), *dev, weights)[1]
        assert torch.equal(again, dw)


def test_combine_backward_in_place():
    dev, ref, rows, w = _routing(50, 3, 6, 32, 5)
    y, dout = synth.normal((rows, 136), 2).cuda(), synth.normal((50, 136), 3).cuda()
    dy, dw = mxq.expert_combine_backward(dout, y, *dev, w, out=torch.zeros_like(y))
    buf = y.clone()
    dy2, dw2 = mxq.expert_combine_backward(dout, buf, *dev, w, out=buf)
    end = ref[1][-1]
    assert dy2 is buf and torch.equal(dw, dw2) and torch.equal(dy[:end], dy2[:end])
    assert torch.equal(buf[end:], y[end:])


def test_gradients_against_differences():
    # combine is linear in y and in the weights: a difference is a gradient, to rounding
    dev, ref, rows, w = _routing(6, 3, 4, 2, 9)
    w = torch.nan_to_num(w)
    y, dout = torch.randn(rows, 20, device="cuda"), torch.randn(6, 20, device="cuda")
    dy, dw = mxq.expert_combine_backward(dout, y, *dev, w, out=torch.zeros_like(y))
    loss = lambda y, w: (mxq.expert_combine(y, dev[0], w).double() * dout.double()).sum().item()
    rng = np.random.default_rng(0)
    for _ in range(12):
        u = torch.from_numpy(rng.standard_normal(y.shape)).cuda().float()
        v = torch.from_numpy(rng.standard_normal(tuple(w.shape))).cuda().float()
        d = (loss(y + u, w) - loss(y - u, w)) / 2
        assert abs(d - (dy.double() * u.double()).sum().item()) < 1e-4
        d = (loss(y, w + v) - loss(y, w - v)) / 2
        assert abs(d - (dw.double() * v.double()).sum().item()) < 1e-4


def test_empty_buffers():
    ids = torch.full((3, 2), -1, device="cuda")
    row_of, offsets, counts = mxq.expert_order(ids, 4)
    x, none = torch.ones(3, 8, device="cuda"), torch.empty(0, 8, device="cuda")
    assert mxq.expert_gather(x, row_of, offsets, counts, 0).shape == (0, 8)
    assert mxq.expert_combine(none, row_of).eq(0).all()
    dy, dw = mxq.expert_combine_backward(x, none, row_of, offsets, counts)
    assert dy.shape == (0, 8) and dw.eq(0).all()
    for rows, cols, tokens in ((4, 0, 3), (4, 8, 0)):
        x, y = torch.ones(tokens, cols, device="cuda"), torch.ones(rows, cols, device="cuda")
        choice = torch.zeros(tokens, 2, dtype=torch.int32, device="cuda")
        assert mxq.expert_gather(x, choice, offsets, counts, rows).shape == (rows, cols)
        assert mxq.expert_combine(y, choice).shape == (tokens, cols)
        assert mxq.expert_combine_backward(x, y, choice, offsets, counts)[1].eq(0).all()
    mxq.check()


def test_rows_outside_the_buffer_are_left_out_and_reported():
    row_of = torch.tensor([[0, 5], [9, -3]], dtype=torch.int32, device="cuda")
    x = torch.ones(2, 16, device="cuda")
    offsets = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    counts = torch.tensor([2], dtype=torch.int32, device="cuda")
    out = mxq.expert_gather(x, row_of, offsets, counts, 4, out=torch.zeros(4, 16, device="cuda"))
    with pytest.raises(mxq.MXQError, match="MXQ_ERR_ARG"):
        mxq.check()
    assert out[0].eq(1).all() and out[1:].eq(0).all()
    mxq.check()


# ---- products ----------------------------------------------------------------------------

def _codes(lines, blocked, fmt, seed):
    x = synth.normal((lines, blocked), seed).float().numpy()
    a, s = O.mx_quantize(x * np.exp(np.random.default_rng(seed).standard_normal((lines, 1))), "row",
                         fmt)
    return np.ascontiguousarray(a), np.ascontiguousarray(s)


def _gpu(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def _offsets(counts, first=0):
    return np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int64)


# rows of the experts, first row, rows behind them, N, K: few and many rows, short and long K
# take different kernels
PRODUCTS = [
    ([1], 0, 0, 8, 32), ([0, 3, 0], 0, 0, 264, 96), ([130, 1, 0, 257, 60], 0, 5, 136, 160),
    ([5, 127, 128, 129], 3, 0, 520, 512), ([300, 700], 0, 0, 256, 288), ([2] * 40, 1, 1, 24, 64),
    ([0] * 30 + [9] + [0] * 3, 0, 0, 1000, 1056), ([400, 0, 41], 0, 0, 264, 2208),
    ([70, 40, 100], 2, 1, 384, 4512), ([17, 0, 9, 70, 3], 0, 0, 136, 512),
    ([30, 2, 65, 0], 1, 3, 264, 288), ([40] + [0] * 5 + [1], 0, 0, 200, 256),
    ([33, 1, 70, 20, 0, 90], 3, 0, 136, 1056)]


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: f"{sum(c[0])}of{len(c[0])}x{c[3]}x{c[4]}")
def test_product(case, fmt, out):
    counts, first, behind, n, k = case
    off = _offsets(counts, first)
    rows, experts = int(off[-1]) + behind, len(counts)
    A, sA = _codes(rows, k, fmt, 1)
    B, sB = _codes(experts * n, k, fmt, 2)
    B, sB = B.reshape(experts, n, -1), sB.reshape(experts, n, -1)
    before = torch.full((rows, n), 7.0, dtype=out, device="cuda")
    o = torch.from_numpy(off).int().cuda()
    got = mxq.mx_gemm_experts(*_gpu(A, sA, B, sB), o, fmt, rows, n, k, out_dtype=out,
                              out=before.clone())
    mxq.check()
    ref, S = E.experts_product(A, sA, B, sB, off, fmt, _f(before))
    tol = (k + 4) * 2.0 ** -23 * S + (HALF[out] * (np.abs(ref) + S * 1e-4) if out is BF else 0.0)
    assert (np.abs(_f(got) - ref) <= np.where(S > 0, tol, 0.0)).all()
    if k % (256 if fmt == "e2m1" else 128) == 0:
        # the same with the weights' scales in the tensor cores' layout: the same bits
        w = [mxq.mx_quantize(synth.normal((n, k), 50 + e).cuda(), "row", fmt) for e in range(experts)]
        t = [mxq.mx_quantize(synth.normal((n, k), 50 + e).cuda(), "row", fmt, scale_layout="tc")
             for e in range(experts)]
        stack = lambda q, i: torch.stack([v[i] for v in q])
        a = _gpu(A, sA)
        one = mxq.mx_gemm_experts(*a, stack(w, 0), stack(w, 1), o, fmt, rows, n, k, out_dtype=out,
                                  out=before.clone())
        two = mxq.mx_gemm_experts(*a, stack(t, 0), stack(t, 1), o, fmt, rows, n, k, out_dtype=out,
                                  out=before.clone(), b_scale_layout="tc")
        mxq.check()
        assert torch.equal(one, two)


def test_product_is_the_single_product_of_each_expert():
    # same tiles, same order of additions: the bits of mx_gemm on each expert's rows
    counts, n, k = [300, 0, 77, 512], 384, 1024
    off = _offsets(counts)
    A, sA = _codes(int(off[-1]), k, "e4m3", 3)
    B, sB = _codes(4 * n, k, "e4m3", 4)
    A, sA, B, sB = _gpu(A, sA, B.reshape(4, n, -1), sB.reshape(4, n, -1))
    got = mxq.mx_gemm_experts(A, sA, B, sB, torch.from_numpy(off).int().cuda(), "e4m3",
                              int(off[-1]), n, k)
    for e, c in enumerate(counts):
        if c:
            s = slice(int(off[e]), int(off[e + 1]))
            want = mxq.mx_gemm(A[s].contiguous(), sA[s].contiguous(), B[e], sB[e], "e4m3", c, n, k)
            assert torch.equal(got[s], want)
    mxq.check()


WGRADS = [   # blocks of 64 rows of the experts, blocks before and behind, M, N
    ([1], 0, 0, 1, 8), ([0, 2, 0], 0, 1, 33, 264), ([3, 0, 5, 1, 1], 1, 0, 300, 136),
    ([9, 4], 0, 0, 129, 520), ([1] * 20, 0, 2, 64, 24), ([0, 0], 0, 1, 40, 16)]


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("case", WGRADS, ids=lambda c: f"{sum(c[0])}of{len(c[0])}x{c[3]}x{c[4]}")
def test_wgrad(case, fmt, out):
    blocks, first, behind, m, n = case
    unit = 64 if fmt == "e2m1" else 32
    off = _offsets(blocks, first) * unit
    rows = int(off[-1]) + behind * unit
    A, sA = _codes(m, rows, fmt, 1)
    B, sB = _codes(n, rows, fmt, 2)
    sA[:, off[-1] // 32:], sB[:, :off[0] // 32] = 255, 255   # rows of no expert: not read
    got = mxq.mx_gemm_experts_wgrad(*_gpu(A, sA, B, sB), torch.from_numpy(off).int().cuda(), fmt, m,
                                    n, rows, out_dtype=out)
    mxq.check()
    sA[:, off[-1] // 32:], sB[:, :off[0] // 32] = 127, 127
    ref, S = E.experts_wgrad(A, sA, B, sB, off, fmt)
    k = max(blocks) * unit
    tol = (k + 4) * 2.0 ** -23 * S + (HALF[out] * (np.abs(ref) + S * 1e-4) if out is BF else 0.0)
    assert got.shape == ref.shape and (np.abs(_f(got) - ref) <= tol).all()


def test_no_rows_at_all():
    o = torch.zeros(4, dtype=torch.int32, device="cuda")
    e = torch.empty(0, dtype=torch.uint8, device="cuda")
    c = mxq.mx_gemm_experts(e, e, torch.zeros(3 * 8 * 32, dtype=torch.uint8, device="cuda"),
                            torch.zeros(24, dtype=torch.uint8, device="cuda"), o, "e4m3", 0, 8, 32)
    g = mxq.mx_gemm_experts_wgrad(e, e, e, e, o, "e4m3", 5, 8, 0,
                                  out=torch.full((3, 5, 8), 7.0, device="cuda"))
    mxq.check()
    assert c.shape == (0, 8) and g.eq(0).all()


@pytest.mark.parametrize("offsets", [[0, 40, 20, 64], [-5, 10, 90, 64], [0, 1000, 1000, 1000],
                                     [2 ** 31 - 1, 0, 0, 0]], ids=str)
def test_offsets_that_fall_or_leave_are_reported(offsets):
    # the table that the kernels follow is put right before any tile goes by it
    A, sA = _codes(64, 64, "e4m3", 1)
    B, sB = _codes(3 * 16, 64, "e4m3", 2)
    a = _gpu(A, sA, B.reshape(3, 16, -1), sB.reshape(3, 16, -1))
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    out = mxq.mx_gemm_experts(*a, o, "e4m3", 64, 16, 64, out=torch.zeros(64, 16, device="cuda"))
    with pytest.raises(mxq.MXQError, match="MXQ_ERR_ARG"):
        mxq.check()
    assert out.isfinite().all()
    mxq.check()


def test_wgrad_offsets_inside_a_block_are_reported():
    A, sA = _codes(16, 64, "e4m3", 1)
    o = torch.tensor([0, 40, 64], dtype=torch.int32, device="cuda")
    a = _gpu(A, sA)
    mxq.mx_gemm_experts_wgrad(*a, *a, o, "e4m3", 16, 16, 64)
    with pytest.raises(mxq.MXQError, match="MXQ_ERR_ARG"):
        mxq.check()


def test_nan_scales_stay_in_their_expert():
    counts, n, k = [40, 50], 64, 128
    off = _offsets(counts)
    A, sA = _codes(90, k, "e4m3", 1)
    B, sB = _codes(2 * n, k, "e4m3", 2)
    B, sB = B.reshape(2, n, -1), sB.reshape(2, n, -1)
    sA[45, 2], sB[1, 5, 0] = 255, 255
    got = _f(mxq.mx_gemm_experts(*_gpu(A, sA, B, sB), torch.from_numpy(off).int().cuda(), "e4m3", 90,
                                 n, k))
    bad = np.zeros((90, n), bool)
    bad[45] = True
    bad[40:, 5] = True
    assert np.array_equal(np.isnan(got), bad)


def test_a_captured_layer_follows_the_routing():
    # order, gather, quantize, product, combine in one graph: replays read new choices
    tokens, topk, experts, n, k = 60, 3, 5, 128, 256
    rows = mxq.expert_rows(tokens * topk, experts, 32)
    ids = torch.from_numpy(_ids(tokens, topk, experts, 1)).cuda()
    x = synth.normal((tokens, k), 1).cuda()
    w = torch.rand(tokens, topk, device="cuda")
    B, sB = mxq.mx_quantize(synth.weight(experts * n, k, 2).cuda(), "row", "e4m3",
                            scale_layout="tc")

    def layer():
        row_of, offsets, counts = mxq.expert_order(ids, experts, 32)
        a = mxq.expert_gather(x, row_of, offsets, counts, rows)
        A, sA = mxq.mx_quantize(a, "row", "e4m3")
        y = mxq.mx_gemm_experts(A, sA, B, sB, offsets, "e4m3", rows, n, k, out_dtype=BF,
                                b_scale_layout="tc")
        return mxq.expert_combine(y, row_of, w)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for seed in (2, 3, 4):
        ids.copy_(torch.from_numpy(_ids(tokens, topk, experts, seed, dropped=0.2 * (seed - 2))))
        x.copy_(synth.normal((tokens, k), seed))
        graph.replay()
        want = layer()
        mxq.check()
        assert torch.equal(out, want)


def test_two_streams():
    counts, n, k = [100, 30, 0, 200], 256, 512
    off = _offsets(counts)
    o = torch.from_numpy(off).int().cuda()
    data = []
    for seed in (1, 2):
        A, sA = _codes(330, k, "e4m3", seed)
        B, sB = _codes(4 * n, k, "e4m3", seed + 10)
        data.append(_gpu(A, sA, B.reshape(4, n, -1), sB.reshape(4, n, -1)))
    want = [mxq.mx_gemm_experts(*d, o, "e4m3", 330, n, k) for d in data]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = mxq.mx_gemm_experts(*data[i], o, "e4m3", 330, n, k)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    mxq.check()
