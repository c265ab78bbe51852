"""Layers of experts and the AdamW step past 2^31 elements: rows, products and moments
behind the point where a 32-bit offset would wrap, against the same call on that part
alone (the same sums in the same order: the same bits)."""

import pytest
import torch

from precision_mx_quantize_gb300 import mxq
from tests.libutil import ensure_built

pytestmark = pytest.mark.gpu

BIG = 2 ** 31


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()
    yield
    torch.cuda.empty_cache()


def test_rows():
    # 2^31 elements and more of rows: two choices of each of the last tokens
    cols, tokens = 8192, 140000
    rows = 2 * tokens
    ids = torch.arange(2, device="cuda").expand(tokens, 2).contiguous()
    row_of, offsets, counts = mxq.expert_order(ids, 2)
    assert rows * cols > BIG and int(row_of[-1, 1]) == rows - 1
    x = torch.zeros(tokens, cols, dtype=torch.bfloat16, device="cuda")
    x[-50:] = torch.randn(50, cols, device="cuda")
    w = torch.rand(tokens, 2, device="cuda")
    y = mxq.expert_gather(x, row_of, offsets, counts, rows, w)
    last = slice(tokens - 50, tokens)
    for j in range(2):
        want = (x[last].float() * w[last, j:j + 1]).bfloat16()
        assert torch.equal(y[row_of[last, j].long()], want)
    out = mxq.expert_combine(y, row_of, w)
    part = torch.cat([y[row_of[last, j].long()] for j in range(2)])
    small = torch.arange(100, dtype=torch.int32, device="cuda").view(2, 50).t().contiguous()
    assert torch.equal(out[last], mxq.expert_combine(part, small, w[last]))
    dy, dw = mxq.expert_combine_backward(x, y, row_of, offsets, counts, w, out=y)
    two = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    n = torch.tensor([100], dtype=torch.int32, device="cuda")
    want = mxq.expert_combine_backward(x[last], part, small, two, n, w[last])
    assert torch.equal(dw[last], want[1])
    assert torch.equal(torch.cat([dy[row_of[last, j].long()] for j in range(2)]), want[0])
    mxq.check()


@pytest.mark.parametrize("tail", [3, 40, 700], ids=str)
def test_product(tail):
    # C of more than 2^31 elements: the last expert's rows lie behind
    n, k, first = 8192, 64, BIG // 8192 + 5
    rows = first + tail
    A = torch.randint(0, 120, (rows, k), dtype=torch.uint8, device="cuda")
    sA = torch.full((rows, 2), 127, dtype=torch.uint8, device="cuda")
    B = torch.randint(0, 120, (2, n, k), dtype=torch.uint8, device="cuda")
    sB = torch.full((2, n, 2), 127, dtype=torch.uint8, device="cuda")
    off = torch.tensor([0, first, rows], dtype=torch.int32, device="cuda")
    c = mxq.mx_gemm_experts(A, sA, B, sB, off, "e4m3", rows, n, k, out_dtype=torch.bfloat16)
    want = mxq.mx_gemm(A[first:].contiguous(), sA[first:].contiguous(), B[1], sB[1], "e4m3", tail, n,
                       k, out_dtype=torch.bfloat16)
    mxq.check()
    assert torch.equal(c[first:], want)


def test_few_rows_of_many_experts():
    # 1024 experts' rows in C of more than 2^31 elements, few to each
    n, k, experts = 262144, 32, 1024
    off = torch.arange(experts + 1, device="cuda").mul_(8).add_(2).int()
    rows = int(off[-1])
    assert rows * n > BIG
    A = torch.randint(0, 120, (rows, k), dtype=torch.uint8, device="cuda")
    sA = torch.full((rows, 1), 127, dtype=torch.uint8, device="cuda")
    B = torch.randint(0, 120, (experts, n, k), dtype=torch.uint8, device="cuda")
    sB = torch.full((experts, n, 1), 127, dtype=torch.uint8, device="cuda")
    c = mxq.mx_gemm_experts(A, sA, B, sB, off, "e4m3", rows, n, k, out_dtype=torch.bfloat16)
    for e in (0, 511, 1023):
        s = slice(int(off[e]), int(off[e + 1]))
        want = mxq.mx_gemm(A[s].contiguous(), sA[s].contiguous(), B[e], sB[e], "e4m3", 8, n, k,
                           out_dtype=torch.bfloat16)
        assert torch.equal(c[s], want)
    mxq.check()


def test_wgrad():
    m, n, experts, rows = 8192, 8192, 33, 33 * 64
    A = torch.randint(0, 120, (m, rows), dtype=torch.uint8, device="cuda")
    sA = torch.full((m, rows // 32), 127, dtype=torch.uint8, device="cuda")
    B = torch.randint(0, 120, (n, rows), dtype=torch.uint8, device="cuda")
    sB = torch.full((n, rows // 32), 127, dtype=torch.uint8, device="cuda")
    off = torch.arange(experts + 1, device="cuda").mul_(64).int()
    c = mxq.mx_gemm_experts_wgrad(A, sA, B, sB, off, "e4m3", m, n, rows)
    assert c.numel() > BIG
    for e in (0, 31, 32):
        s, q = slice(64 * e, 64 * e + 64), slice(2 * e, 2 * e + 2)
        want = mxq.mx_gemm(A[:, s].contiguous(), sA[:, q].contiguous(), B[:, s].contiguous(),
                           sB[:, q].contiguous(), "e4m3", m, n, 64)
        assert torch.equal(c[e], want)
    mxq.check()


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw(bits):
    n, part = BIG + 1000, 4096
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    state = mxq.adamw_state(p, bits)
    cut = n // 128 * 128 - part       # whole blocks from here on
    p[cut:], g[cut:] = torch.randn(n - cut, device="cuda"), torch.randn(n - cut, device="cuda")
    p2, g2 = p[cut:].clone(), g[cut:].clone()
    state2 = mxq.adamw_state(p2, bits)
    for q, d, s in ((p, g, state), (p2, g2, state2)):
        mxq.adamw_step(mxq.adamw_plan([q], [s], weight_decay=0.1), [d], 1, 1e-3)
    mxq.check()
    assert torch.equal(p[cut:], p2) and p[:cut].count_nonzero() == 0
    for a, b in zip(state, state2):
        if bits == 32:
            assert torch.equal(a[cut:], b)
        else:
            assert torch.equal(a[0][cut:], b[0]) and torch.equal(a[1][cut // 128:], b[1])
