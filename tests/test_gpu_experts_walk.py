"""Layers of experts at sizes where a team of threads takes several tokens, and a CTA or a
cluster several tiles, one after another: what is carried from one to the next (rings of
copies, buffers of sums, scale slots, accumulators) against float64 on the GPU.

Tolerances.  combine: k products and additions in fp32, each within 2^-24 of a value below
the sum S of magnitudes: 2 k 2^-24 S, and half a step of the output.  Its gradients: one
product and a rounding; a fused product and addition per column and a tree of additions,
(cols + 16) 2^-24 S.  Products: K additions inside the tensor cores, each within 2^-23 of S
(a truncation is a whole step): (K + 4) 2^-23 S, and half a step of bf16, 2^-8.  Sums that
start from codes below 2^-9 stay far above fp32's smallest values."""

import numpy as np
import pytest
import torch

from precision_mx_quantize_gb300 import mxq
from tests.libutil import ensure_built

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ---- order ------------------------------------------------------------------------

@pytest.mark.parametrize("wide", [False, True], ids=["int32", "int64"])
@pytest.mark.parametrize("case", [(100000, 8, 64, 32), (700001, 1, 1024, 1), (311297, 2, 3, 7)],
                         ids=str)
def test_order_of_many_choices(case, wide):
    # more than 152 blocks of 4096: each warp takes more than its first four steps
    tokens, topk, experts, align = case
    ids = np.random.default_rng(tokens).integers(-1, experts + 1, (tokens, topk))
    t = torch.from_numpy(ids).cuda().to(torch.int64 if wide else torch.int32)
    row_of, offsets, counts = mxq.expert_order(t, experts, align)
    mxq.check()
    flat = ids.reshape(-1)
    inside = np.flatnonzero((flat >= 0) & (flat < experts))
    by = inside[np.argsort(flat[inside], kind="stable")]
    n = np.bincount(flat[inside], minlength=experts)
    start = np.concatenate([[0], np.cumsum((n + align - 1) // align * align)])
    want = np.full(flat.size, -1)
    want[by] = start[flat[by]] + np.arange(by.size) - (np.cumsum(n) - n)[flat[by]]
    assert np.array_equal(row_of.cpu().numpy().reshape(-1), want)
    assert np.array_equal(offsets.cpu().numpy(), start) and np.array_equal(counts.cpu().numpy(), n)


# ---- rows ---------------------------------------------------------------------------

# tokens, choices, experts, columns, align: more tokens than the device holds teams
WALKS = [(6000, 8, 20, 264, 32), (6000, 8, 20, 4096, 32), (6000, 6, 20, 520, 1),
         (7000, 5, 9, 1032, 64), (9000, 3, 7, 1001, 32), (9000, 8, 7, 99, 16), (6000, 2, 5, 2048, 32),
         (5000, 4, 160, 1288, 32), (4000, 9, 16, 520, 32), (4000, 17, 24, 333, 1)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", WALKS, ids=str)
def test_rows_of_many_tokens(case, dtype):
    tokens, topk, experts, cols, align = case
    g = _gen(tokens + topk)
    ids = torch.randint(0, experts, (tokens, topk), device="cuda", generator=g)
    ids[torch.rand(tokens, topk, device="cuda", generator=g) < 0.1] = -1
    ids[5::97] = -1                                         # tokens that no expert takes
    dev = row_of, offsets, counts = mxq.expert_order(ids, experts, align)
    rows = mxq.expert_rows(ids.numel(), experts, align) + 3
    has = row_of >= 0
    w = torch.randn(tokens, topk, device="cuda", generator=g)
    w[~has] = float("nan")                                  # not read
    x = torch.randn(tokens, cols, device="cuda", generator=g).to(dtype)
    y = torch.randn(rows, cols, device="cuda", generator=g).to(dtype)
    at, wz = row_of.clamp_min(0).long(), torch.where(has, w, 0.0).to(F64)

    # what gather and the gradient write: their rows, zeros between, the rest as it was
    off, n = offsets.tolist(), counts.tolist()
    want = torch.full((rows, cols), 7.0, dtype=F64, device="cuda")
    want[:off[-1]] = 0.0
    for j in range(topk):
        h = has[:, j]
        want[at[h, j]] = x[h].to(F64) * wz[h, j:j + 1]
    tol = (2.0 ** -24 + HALF[dtype]) * want.abs() + 1e-38
    before = torch.full((rows, cols), 7.0, dtype=dtype, device="cuda")
    got = mxq.expert_gather(x, *dev, rows, weights=w, out=before.clone())
    assert ((got.to(F64) - want).abs() <= tol).all()
    dy, dw = mxq.expert_combine_backward(x, y, *dev, w, out=before.clone())
    assert torch.equal(dy, got)
    for e in range(experts):
        assert dy[off[e] + n[e]:off[e + 1]].eq(0).all()

    out = mxq.expert_combine(y, row_of, w)
    mxq.check()
    total, size = torch.zeros(tokens, cols, dtype=F64, device="cuda"), 0.0
    dwant, dsize = torch.zeros(tokens, topk, dtype=F64, device="cuda"), torch.zeros_like(wz)
    for j in range(topk):
        v = torch.where(has[:, j:j + 1], y[at[:, j]].to(F64), 0.0)
        total, size = total + v * wz[:, j:j + 1], size + (v * wz[:, j:j + 1]).abs()
        dwant[:, j], dsize[:, j] = (v * x.to(F64)).sum(1), (v * x.to(F64)).abs().sum(1)
    tol = 2 * topk * 2.0 ** -24 * size + HALF[dtype] * (1 + 1e-6) * total.abs() + 1e-38
    assert ((out.to(F64) - total).abs() <= tol).all()
    assert ((dw.to(F64) - dwant).abs() <= (cols + 16) * 2.0 ** -24 * dsize).all()

    # over y itself: the same bits
    buf = y.clone()
    dy2, dw2 = mxq.expert_combine_backward(x, buf, *dev, w, out=buf)
    mxq.check()
    assert dy2 is buf and torch.equal(dw2, dw) and torch.equal(buf[:off[-1]], dy[:off[-1]])
    assert torch.equal(buf[off[-1]:], y[off[-1]:])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", [(50, 2, 5, 264, 4096, 0), (3000, 8, 20, 72, 1000, 0), (40, 1, 9, 33, 511, 7),
                                  (700, 6, 30, 136, 2048, -3), (1, 1, 1024, 8, 64, 5000)], ids=str)
def test_long_padding(case, dtype):
    # several teams to an expert's padding, in buffers of the exact size, shorter or longer ones
    tokens, topk, experts, cols, align, more = case
    g = _gen(tokens)
    ids = torch.randint(-1, experts, (tokens, topk), device="cuda", generator=g)
    dev = row_of, offsets, counts = mxq.expert_order(ids, experts, align)
    off, n = offsets.tolist(), counts.tolist()
    end = off[-1]
    rows = max(end + more, 1)
    x = torch.randn(tokens, cols, device="cuda", generator=g).to(dtype)
    y = torch.randn(rows, cols, device="cuda", generator=g).to(dtype)
    want = torch.full((rows + 4, cols), 7.0, dtype=dtype, device="cuda")
    want[:min(end, rows)] = 0.0
    for j in range(topk):
        h = (row_of[:, j] >= 0) & (row_of[:, j] < rows)
        want[row_of[h, j].long()] = x[h]
    out = torch.full((rows + 4, cols), 7.0, dtype=dtype, device="cuda")
    mxq.expert_gather(x, *dev, rows, out=out)
    assert torch.equal(out, want)
    out.fill_(7.0)
    mxq.expert_combine_backward(x, y, *dev, out=out)
    assert torch.equal(out, want)
    mxq.check()


# ---- products -------------------------------------------------------------------------

BAD = {"e4m3": [0x7F, 0xFF], "e5m2": [c | s for c in (0x7C, 0x7D, 0x7E, 0x7F) for s in (0, 0x80)],
       "e2m1": []}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _table(fmt):
    if fmt == "e2m1":
        return torch.tensor(E2M1 + [-v for v in E2M1], dtype=F64, device="cuda")
    t = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    return torch.arange(256, dtype=torch.uint8).view(t).to(F64).cuda()


def _operand(lines, k, fmt, seed):
    """Random codes (numbers only) and scales of 2^-3 to 2^3."""
    g = _gen(seed)
    a = torch.randint(0, 256, (lines, k // 2 if fmt == "e2m1" else k), dtype=torch.uint8,
                      device="cuda", generator=g)
    for c in BAD[fmt]:
        a[a == c] = 0x35
    return a, torch.randint(124, 131, (lines, k // 32), dtype=torch.uint8, device="cuda", generator=g)


def _values(a, s, fmt):
    if fmt == "e2m1":
        a = torch.stack([a & 15, a >> 4], 2).flatten(1)
    return _table(fmt)[a.int()] * torch.exp2(s.to(F64) - 127.0).repeat_interleave(32, 1)


def _near(got, a, b, k, dtype):
    ref, S = a @ b.t(), a.abs() @ b.abs().t()
    tol = (k + 4) * 2.0 ** -23 * S
    if dtype is BF:
        tol = tol + HALF[BF] * (ref.abs() + tol)
    assert ((got.to(F64) - ref).abs() <= tol).all()


def _counts(experts, mean, seed):
    """Uneven, some empty, one with many, of about that mean."""
    r = np.random.default_rng(seed)
    n = r.integers(0, 2 * mean + 1, experts)
    n[r.integers(0, experts, max(1, experts // 8))] = 0
    n[int(r.integers(experts))] += 2 * mean
    return n


# name of the form, experts, mean rows, N, bytes of K: several tiles a CTA or cluster
FORMS = [("few, 16 rows", 40, 9, 3016, 672), ("few, 64 rows", 48, 34, 2008, 672),
         ("256 rows, staged", 30, 150, 2008, 720), ("256 rows", 30, 150, 2008, 1808),
         ("few, 16 rows, ring ends inside", 33, 10, 4008, 208), ("few of 1024", 1024, 9, 136, 160),
         ("64 rows of 900", 900, 30, 264, 96)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("case", FORMS, ids=lambda c: c[0])
def test_products_of_many_tiles(case, fmt, dtype):
    _, experts, mean, n, kb = case
    k = 2 * kb if fmt == "e2m1" else kb // 32 * 32
    counts = _counts(experts, mean, experts)
    off = np.concatenate([[0], np.cumsum(counts)])
    rows = int(off[-1])
    A, sA = _operand(rows, k, fmt, 1)
    B, sB = _operand(experts * n, k, fmt, 2)
    o = torch.from_numpy(off).int().cuda()
    call = lambda B, sB, **kw: mxq.mx_gemm_experts(
        A, sA, B.view(experts, n, -1), sB, o, fmt, rows, n, k, out_dtype=dtype,
        out=torch.full((rows + 1, n), 7.0, dtype=dtype, device="cuda"), **kw)
    c = call(B, sB)
    mxq.check()
    a = _values(A, sA, fmt)
    for e in range(experts):
        if counts[e]:
            b = _values(B[e * n:(e + 1) * n], sB[e * n:(e + 1) * n], fmt)
            _near(c[off[e]:off[e + 1]], a[off[e]:off[e + 1]], b, k, dtype)
    assert c[rows:].eq(7.0).all()
    assert torch.equal(c, call(B, sB))


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("case", [(40, 9, 3016, 768), (48, 34, 2008, 768), (30, 150, 2008, 768),
                                  (30, 150, 2008, 1792)], ids=str)
def test_products_of_many_tiles_with_scales_in_chunks(case, fmt):
    experts, mean, n, kb = case
    k = 2 * kb if fmt == "e2m1" else kb
    off = np.concatenate([[0], np.cumsum(_counts(experts, mean, experts))])
    rows = int(off[-1])
    A, sA = _operand(rows, k, fmt, 1)
    o = torch.from_numpy(off).int().cuda()
    w = torch.randn(experts, n, k, device="cuda", generator=_gen(3)).bfloat16()
    w.mul_(torch.randn(experts, n, 1, device="cuda", generator=_gen(4)).exp())
    got = []
    for layout in ("rowmajor", "tc"):
        q = [mxq.mx_quantize(v, "row", fmt, scale_layout=layout) for v in w]
        got.append(mxq.mx_gemm_experts(A, sA, torch.stack([v[0] for v in q]),
                                       torch.stack([v[1] for v in q]), o, fmt, rows, n, k,
                                       b_scale_layout=layout))
    mxq.check()
    assert torch.equal(*got)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("case", [(12, 5, 1000, 1304), (40, 2, 513, 264), (7, 40, 1500, 1544)], ids=str)
def test_weight_gradients_of_many_tiles(case, fmt, dtype):
    experts, mean, m, n = case
    unit = 64 if fmt == "e2m1" else 32
    off = np.concatenate([[0], np.cumsum(_counts(experts, mean, m))]) * unit
    rows = int(off[-1]) + unit
    A, sA = _operand(m, rows, fmt, 1)
    B, sB = _operand(n, rows, fmt, 2)
    o = torch.from_numpy(off).int().cuda()
    c = mxq.mx_gemm_experts_wgrad(A, sA, B, sB, o, fmt, m, n, rows, out_dtype=dtype)
    mxq.check()
    a, b = _values(A, sA, fmt), _values(B, sB, fmt)
    for e in range(experts):
        lo, hi = off[e], off[e + 1]
        _near(c[e], a[:, lo:hi], b[:, lo:hi], hi - lo, dtype)
    assert torch.equal(c, mxq.mx_gemm_experts_wgrad(A, sA, B, sB, o, fmt, m, n, rows, out_dtype=dtype))


# ---- offsets that no tile may follow -------------------------------------------------------

def _repaired(offsets, rows, unit):
    """The nearest offsets that neither fall, leave the rows nor split a unit."""
    placed = np.clip(np.array(offsets, np.int64), 0, rows) // unit * unit
    return np.maximum.accumulate(placed)


@pytest.mark.parametrize("case", [
    (64, [0, 40, 20, 64]), (64, [-5, 10, 90, 64]), (64, [0, 1000, 1000, 1000]),
    (64, [2 ** 31 - 1, 0, 0, 0]), (64, [7, 3, 50, -2 ** 31]), (30, [0, 12, 5, 30]),
    (700, [0, 400, 200, 650]), (700, [-9, 90, 800, 640]), (700, [300, 10, 690, 2 ** 31 - 1])], ids=str)
def test_products_by_repaired_offsets(case):
    rows, offsets = case
    n, k = 136, 288
    A, sA = _operand(rows, k, "e4m3", 1)
    B, sB = _operand(3 * n, k, "e4m3", 2)
    o = torch.tensor(offsets, dtype=torch.int64, device="cuda").int()
    c = mxq.mx_gemm_experts(A, sA, B.view(3, n, -1), sB, o, "e4m3", rows, n, k,
                            out=torch.full((rows, n), 7.0, device="cuda"))
    with pytest.raises(mxq.MXQError, match="MXQ_ERR_ARG"):
        mxq.check()
    off = _repaired(offsets, rows, 1)
    a, b = _values(A, sA, "e4m3"), _values(B, sB, "e4m3")
    for e in range(3):
        s = slice(off[e], off[e + 1])
        _near(c[s], a[s], b[e * n:(e + 1) * n], k, F32)
    assert c[:off[0]].eq(7.0).all() and c[off[-1]:].eq(7.0).all()
    mxq.check()


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("offsets", [[0, 40, 100, 192], [0, 130, 64, 192], [-64, 64, 500, 128],
                                     [2 ** 31 - 1, 0, 64, 128], [1, 2, 3, 200]], ids=str)
def test_weight_gradients_by_repaired_offsets(offsets, fmt):
    rows, m, n = 192, 40, 24
    A, sA = _operand(m, rows, fmt, 1)
    B, sB = _operand(n, rows, fmt, 2)
    o = torch.tensor(offsets, dtype=torch.int64, device="cuda").int()
    c = mxq.mx_gemm_experts_wgrad(A, sA, B, sB, o, fmt, m, n, rows)
    with pytest.raises(mxq.MXQError, match="MXQ_ERR_ARG"):
        mxq.check()
    off = _repaired(offsets, rows, 64 if fmt == "e2m1" else 32)
    a, b = _values(A, sA, fmt), _values(B, sB, fmt)
    for e in range(3):
        lo, hi = off[e], off[e + 1]
        _near(c[e], a[:, lo:hi], b[:, lo:hi], hi - lo, F32)
    mxq.check()
