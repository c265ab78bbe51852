"""Refusals of the experts' operators and the AdamW step (CPU): the C entry points reject
bad arguments before any device work, the binding rejects tensors that do not fit the
sizes, the argument structures have the C layout, and the oracle's definitions hold."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import expert_oracle as E
from precision_mx_quantize_gb300 import mxq
from precision_mx_quantize_gb300.expert_layer import MxExpertLinear
from tests.libutil import ensure_built

P, ODD = 16 * 1024, 16 * 1024 + 2   # never dereferenced: every call fails its checks
U8, I32, F32, BF = torch.uint8, torch.int32, torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_built()


# ---- the C entry points ----------------------------------------------------------------

def test_order_refusals():
    def call(**kw):
        a = dict(ids=P, bytes=4, n=8, experts=4, align=1, row_of=P, offsets=P, counts=P, ws=None,
                 size=0)
        a.update(kw)
        return mxq.mxq_expert_order(*a.values(), None)

    for kw in (dict(n=-1), dict(bytes=2), dict(experts=0), dict(experts=1025), dict(align=0),
               dict(align=4097), dict(n=2 ** 31), dict(ids=None), dict(row_of=None),
               dict(offsets=None), dict(counts=None), dict(n=2 ** 31 - 5, align=4096)):
        assert call(**kw) == 1, kw
    for kw in (dict(ids=ODD), dict(ids=P + 4, bytes=8), dict(row_of=ODD), dict(offsets=ODD),
               dict(counts=ODD)):
        assert call(**kw) == 2, kw
    need = mxq.mxq_expert_order_workspace_size(100000, 64)
    assert need > 0 and call(n=100000, experts=64, ws=P, size=need - 1) == 6
    assert call(n=100000, experts=64) == 6
    assert mxq.mxq_expert_order_workspace_size(4096, 64) == 0
    assert mxq.mxq_expert_order_workspace_size(-1, 64) == 0


ROWS = dict(x=P, y=P, out=P, row_of=P, offsets=P, counts=P, weights=P, dweights=P, tokens=4, rows=8,
            cols=16, topk=2, experts=3, dtype=1)


def _rows(fn, **kw):
    args = mxq.ExpertRowsArgs(**{**ROWS, **kw})
    return fn(ctypes.addressof(args), None)


def test_rows_refusals():
    gather, combine = mxq.mxq_expert_gather, mxq.mxq_expert_combine
    back = mxq.mxq_expert_combine_backward
    for fn in (gather, combine, back):
        assert fn(None, None) == 1
        for kw in (dict(tokens=-1), dict(rows=-1), dict(cols=-1), dict(topk=0), dict(topk=1025),
                   dict(tokens=2 ** 31), dict(rows=2 ** 31), dict(cols=2 ** 31), dict(dtype=2),
                   dict(tokens=2 ** 30, topk=4), dict(row_of=None), dict(out=None)):
            assert _rows(fn, **kw) == 1, (fn, kw)
        for kw in (dict(row_of=ODD), dict(out=ODD), dict(weights=ODD)):
            assert _rows(fn, **kw) == 2, (fn, kw)
        assert _rows(fn, tokens=0, rows=0) == 0
    for fn in (gather, back):
        for kw in (dict(experts=0), dict(experts=1025), dict(offsets=None), dict(counts=None),
                   dict(x=None)):
            assert _rows(fn, **kw) == 1, kw
        assert _rows(fn, x=P + 8) == 2 and _rows(fn, counts=ODD) == 2
    for fn in (combine, back):
        assert _rows(fn, y=None) == 1 and _rows(fn, y=P + 8) == 2
    assert _rows(back, dweights=None) == 1 and _rows(back, dweights=ODD) == 2
    assert _rows(gather, cols=0) == 0 and _rows(combine, cols=0) == 0


EXPERTS = dict(A=P, sA=P, B=P, sB=P, offsets=P, C=P, workspace=P, workspace_bytes=1 << 40, rows=64,
               M=64, N=64, K=256, experts=4, fmt=0, out_dtype=0, b_scale_layout=0)


def _experts(fn, **kw):
    args = mxq.ExpertsArgs(**{**EXPERTS, **kw})
    return fn(ctypes.addressof(args), None)


def test_product_refusals():
    rows, wgrad = mxq.mxq_gemm_experts, mxq.mxq_gemm_experts_wgrad
    for fn in (rows, wgrad):
        assert fn(None, None) == 1
        for kw in (dict(rows=-32), dict(rows=2 ** 31), dict(N=0), dict(N=2 ** 31), dict(experts=0),
                   dict(experts=1025), dict(fmt=3), dict(out_dtype=2), dict(A=None), dict(sA=None),
                   dict(B=None), dict(sB=None), dict(offsets=None), dict(C=None),
                   dict(workspace=None)):
            assert _experts(fn, **kw) == 1, kw
        for kw in (dict(A=ODD), dict(B=ODD), dict(C=ODD), dict(offsets=ODD), dict(workspace=P + 16),
                   dict(N=66), dict(N=60, out_dtype=1)):
            assert _experts(fn, **kw) == 2, kw
        assert _experts(fn, workspace_bytes=16) == 6
    for kw in (dict(K=0), dict(K=48), dict(K=2 ** 31), dict(b_scale_layout=2),
               dict(b_scale_layout=1, K=96), dict(b_scale_layout=1, K=128, fmt=1),
               dict(experts=1024, N=2 ** 22)):
        assert _experts(rows, **kw) == 1, kw
    assert _experts(rows, b_scale_layout=1, sB=P + 8) == 2
    assert _experts(rows, rows=0, A=None, C=None) == 0
    for kw in (dict(M=0), dict(M=2 ** 31), dict(rows=40)):
        assert _experts(wgrad, **kw) == 1, kw
    size = mxq.mxq_gemm_experts_workspace_size
    assert size(64, 64, 256, 4, 0, 0) > size(64, 64, 256, 4, 0, 1) > 0
    assert _experts(rows, workspace_bytes=size(64, 64, 256, 4, 0, 0) - 1) == 6
    assert size(64, 64, 250, 4, 0, 0) == 0 and size(64, 64, 256, 0, 0, 0) == 0
    size = mxq.mxq_gemm_experts_wgrad_workspace_size
    assert size(64, 64, 64, 4, 0) > 0 and size(65, 64, 64, 4, 0) == 0
    assert _experts(wgrad, workspace_bytes=size(64, 64, 64, 4, 0) - 1) == 6


@pytest.mark.parametrize("fmt", [0, 1])
def test_workspaces_hold_every_routing(fmt):
    # the chunks that the sizes allow for are those of the worst routing: the device packs
    # each expert's tail into a chunk of its own
    rng = np.random.default_rng(fmt)
    per = 256 if fmt else 128
    for _ in range(200):
        experts, unit = int(rng.integers(1, 40)), 64 if fmt else 32
        counts = rng.integers(0, 12, experts) * unit * (rng.random(experts) < 0.7)
        rows = int(counts.sum()) or unit
        chunks = sum(-(-int(c) // per) for c in counts) * (2 if fmt else 1)
        table = (3 * (experts + 1) * 4 + 255) // 256 * 256
        size = mxq.mxq_gemm_experts_wgrad_workspace_size(rows, 128, 128, experts, fmt)
        assert (size - table) // 512 >= 2 * chunks
        counts = rng.integers(0, 300, experts) * (rng.random(experts) < 0.5)
        rows = int(counts.sum()) or 1
        average = rows // max(1, min(experts, rows))
        tiles = sum(-(-int(c) // 128) for c in counts) if average > 48 else 0   # few: none
        kcs = 4 // (2 if fmt else 1) * (2 if fmt else 1)
        size = mxq.mxq_gemm_experts_workspace_size(rows, 128, 512, experts, fmt, 1)
        assert (size - table) // 512 >= tiles * kcs


ADAMW = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, lr_at=None, step_at=None,
             grad_scale_at=None, grad_dtype=0, state_bits=32)
TENSOR = dict(param=P, m=P, v=P, m_scale=P, r_scale=P, copy=P, n=4, weight_decay=0.0)


def _adamw(tensor=None, grad=P, count=1, **kw):
    t = mxq.AdamWTensor(**{**TENSOR, **(tensor or {})})
    g, args = (ctypes.c_void_p * 1)(grad), mxq.AdamWArgs(**{**ADAMW, **kw})
    return mxq.mxq_adamw(ctypes.addressof(t), ctypes.addressof(g), count, ctypes.addressof(args),
                         None)


def test_adamw_refusals():
    assert mxq.mxq_adamw(None, None, 0, None, None) == 1
    args = mxq.AdamWArgs(**ADAMW)
    assert mxq.mxq_adamw(None, None, 1, ctypes.addressof(args), None) == 1
    assert _adamw(count=-1) == 1
    nan = float("nan")
    for kw in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=nan), dict(eps=-1.0), dict(eps=nan),
               dict(step=0), dict(grad_dtype=2), dict(state_bits=16)):
        assert _adamw(**kw) == 1, kw
    assert _adamw(dict(n=2 ** 45)) == 1          # more chunks than a launch has
    for t in (dict(n=-1), dict(param=None), dict(m=None), dict(v=None)):
        assert _adamw(t) == 1, t
    assert _adamw(grad=None) == 1
    for t in (dict(m_scale=None), dict(r_scale=None)):
        assert _adamw(t, state_bits=8) == 1, t
    for t in (dict(param=ODD), dict(m=ODD), dict(v=ODD), dict(copy=P + 1)):
        assert _adamw(t) == 2, t
    assert _adamw(grad=ODD) == 2 and _adamw(grad=P + 1, grad_dtype=1) == 2
    assert _adamw(dict(m_scale=ODD), state_bits=8) == 2
    for kw in (dict(lr_at=ODD), dict(grad_scale_at=ODD), dict(step_at=P + 4)):
        assert _adamw(**kw) == 2, kw


@pytest.mark.parametrize("struct, name, packed", [
    (mxq.ExpertRowsArgs, "mxq_expert_rows_args", mxq._EXPERT_ROWS_ARGS),
    (mxq.ExpertsArgs, "mxq_experts_args", mxq._EXPERTS_ARGS),
    (mxq.AdamWTensor, "mxq_adamw_tensor", mxq._ADAMW_TENSOR),
    (mxq.AdamWArgs, "mxq_adamw_args", mxq._ADAMW_ARGS)], ids=lambda v: v if isinstance(v, str) else "")
def test_argument_structures_match_the_header(tmp_path, struct, name, packed):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    fields = [f for f, _ in struct._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"mxq.h\"\nint main(void) {\n"
                   f"  printf(\"%zu\", sizeof({name}));\n" +
                   "".join(f"  printf(\" %zu\", offsetof({name}, {f}));\n" for f in fields) +
                   "  return 0;\n}\n")
    subprocess.run([cc, "-I", inc, str(src), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True)
    want = [ctypes.sizeof(struct)] + [getattr(struct, f).offset for f in fields]
    assert [int(v) for v in got.stdout.split()] == want
    values = list(range(1, len(fields) + 1))
    assert packed.pack(*values) == bytes(struct(*values))


# ---- the binding's checks, against recorders in place of the library ------------------------

@pytest.fixture
def fake(monkeypatch):
    calls = []
    for name in ("mxq_expert_order", "mxq_expert_gather", "mxq_expert_combine",
                 "mxq_expert_combine_backward", "mxq_gemm_experts", "mxq_gemm_experts_wgrad",
                 "mxq_adamw", "mxq_quantize", "mxq_quantize_dual", "mxq_quantize_ex",
                 "mxq_quantize_dual_ex"):
        monkeypatch.setattr(mxq, name, lambda *a, _n=name: calls.append((_n, a)) or 0)
    monkeypatch.setattr(mxq, "_stream", lambda device=None: 0)
    monkeypatch.setattr(mxq, "_on_gpu", lambda t: True)
    return calls


def _refused(cases, kinds=(ValueError, TypeError)):
    for i, f in enumerate(cases):
        with pytest.raises(kinds):
            f()
            pytest.fail(f"case {i} was accepted")


def test_rows_bindings(fake):
    ids = torch.zeros(5, 2, dtype=torch.int64)
    row_of, offsets, counts = mxq.expert_order(ids, 4, 32)
    assert row_of.shape == (5, 2) and offsets.shape == (5,) and counts.shape == (4,)
    assert mxq.expert_rows(10, 4, 32) == 160 and mxq.expert_rows(10, 4) == 10
    assert mxq.expert_rows(0, 4, 32) == 0 and mxq.expert_rows(2, 4, 32) == 64
    x, w = torch.zeros(5, 33, dtype=BF), torch.zeros(5, 2)
    y = mxq.expert_gather(x, row_of, offsets, counts, 160, w)
    assert y.shape == (160, 33) and y.dtype is BF
    assert mxq.expert_combine(y, row_of, w).shape == (5, 33)
    dy, dw = mxq.expert_combine_backward(x, y, row_of, offsets, counts, w, out=y)
    assert dy is y and dw.shape == (5, 2)
    assert len(fake) == 4
    fake.clear()
    _refused([
        lambda: mxq.expert_order(ids.float(), 4), lambda: mxq.expert_order(ids[0], 4),
        lambda: mxq.expert_order(ids.t(), 4), lambda: mxq.expert_order(ids, 0),
        lambda: mxq.expert_order(ids, 1025),
        lambda: mxq.expert_gather(x.half(), row_of, offsets, counts, 160),
        lambda: mxq.expert_gather(x.t(), row_of, offsets, counts, 160),
        lambda: mxq.expert_gather(x[:4], row_of, offsets, counts, 160),
        lambda: mxq.expert_gather(x, row_of.long(), offsets, counts, 160),
        lambda: mxq.expert_gather(x, row_of[0], offsets, counts, 160),
        lambda: mxq.expert_gather(x, row_of, offsets[1:], counts, 160),
        lambda: mxq.expert_gather(x, row_of, offsets, counts[1:], 160),
        lambda: mxq.expert_gather(x, row_of, offsets, counts, 160, w.bfloat16()),
        lambda: mxq.expert_gather(x, row_of, offsets, counts, 160, w[:, :1].contiguous()),
        lambda: mxq.expert_gather(x, row_of, offsets, counts, 160, out=y[:159]),
        lambda: mxq.expert_gather(x, row_of, offsets, counts, 160, out=y.float()),
        lambda: mxq.expert_combine(y[0], row_of), lambda: mxq.expert_combine(y, row_of, w.double()),
        lambda: mxq.expert_combine(y, row_of, out=x[:4]),
        lambda: mxq.expert_combine_backward(x.float(), y, row_of, offsets, counts),
        lambda: mxq.expert_combine_backward(x, y[:, :32].contiguous(), row_of, offsets, counts),
        lambda: mxq.expert_combine_backward(x, y, row_of, offsets, counts, out=y[:3])])
    # reads and writes of one memory
    big = torch.zeros(400, 33, dtype=BF)
    _refused([
        lambda: mxq.expert_gather(big[:5], row_of, offsets, counts, 160, out=big[:160]),
        lambda: mxq.expert_gather(big[159:164], row_of, offsets, counts, 160, out=big[:160]),
        lambda: mxq.expert_combine(big[:160], row_of, out=big[:5]),
        lambda: mxq.expert_combine_backward(big[:5], y, row_of, offsets, counts, out=big[:160]),
        lambda: mxq.expert_combine_backward(x, big[:160], row_of, offsets, counts,
                                            out=big[1:161])])
    mxq.expert_gather(big[160:165], row_of, offsets, counts, 160, out=big[:160])
    fake.clear()
    assert not fake


def test_product_bindings(fake):
    for fmt, layout in (("e4m3", "rowmajor"), ("e2m1", "tc"), ("e5m2", "tc")):
        e, n, k, rows = 3, 72, 256, 50
        kb = k // 2 if fmt == "e2m1" else k
        A, sA = torch.zeros(rows, kb, dtype=U8), torch.zeros(rows, k // 32, dtype=U8)
        B = torch.zeros(e, n, kb, dtype=U8)
        sB = torch.zeros(e, n * k // 32 if layout == "rowmajor" else mxq.mxq_scales_tc_bytes(n, k),
                         dtype=U8)
        off = torch.zeros(e + 1, dtype=I32)
        call = lambda A=A, sA=sA, B=B, sB=sB, off=off, fmt=fmt, rows=rows, n=n, k=k, **kw: \
            mxq.mx_gemm_experts(A, sA, B, sB, off, fmt, rows, n, k,
                                **{"b_scale_layout": layout, **kw})
        assert call().shape == (rows, n) and call(out_dtype=BF).dtype is BF
        call(workspace=mxq.gemm_experts_workspace(rows, n, k, e, fmt, "cpu", layout),
             out=torch.zeros(rows, n))
        assert len(fake) == 3
        fake.clear()
        _refused([lambda: call(A=A[1:]), lambda: call(A=A.int()), lambda: call(sA=sA[1:]),
                  lambda: call(B=B[1:]), lambda: call(sB=sB[1:]), lambda: call(off=off.long()),
                  lambda: call(off=off[None]), lambda: call(off=None), lambda: call(rows=rows + 1),
                  lambda: call(k=k + 256), lambda: call(n=n + 8), lambda: call(A=A.t()),
                  lambda: call(out=torch.zeros(rows, n - 8)), lambda: call(out_dtype=torch.half),
                  lambda: call(out=torch.zeros(rows, n, dtype=BF)),
                  lambda: call(workspace=torch.zeros(9)),
                  lambda: call(k=96, b_scale_layout="tc")])
        _refused([lambda: call(fmt="e3m4"), lambda: call(b_scale_layout="cols")], KeyError)
        assert not fake


def test_wgrad_bindings(fake):
    for fmt in ("e4m3", "e2m1"):
        m, n, rows = 40, 24, 192
        rb = rows // 2 if fmt == "e2m1" else rows
        A, sA = torch.zeros(m, rb, dtype=U8), torch.zeros(m, rows // 32, dtype=U8)
        B, sB = torch.zeros(n, rb, dtype=U8), torch.zeros(n, rows // 32, dtype=U8)
        off = torch.zeros(4, dtype=I32)
        call = lambda A=A, sA=sA, B=B, sB=sB, off=off, fmt=fmt, m=m, n=n, rows=rows, **kw: \
            mxq.mx_gemm_experts_wgrad(A, sA, B, sB, off, fmt, m, n, rows, **kw)
        assert call().shape == (3, m, n)
        call(workspace=mxq.gemm_experts_wgrad_workspace(rows, m, n, 3, fmt, "cpu"),
             out=torch.zeros(3, m, n))
        assert len(fake) == 2
        fake.clear()
        _refused([lambda: call(A=A[1:]), lambda: call(sB=sB[1:]), lambda: call(rows=rows + 64),
                  lambda: call(off=off.float()), lambda: call(out=torch.zeros(3, m, n - 8)),
                  lambda: call(out=torch.zeros(2, m, n)), lambda: call(out_dtype=torch.half)])
        assert not fake


def test_layer_makes_the_operands_it_needs(fake):
    for fmt, out_f, in_f, layout in (("e4m3", 128, 256, "tc"), ("e4m3", 96, 256, "rowmajor"),
                                     ("e2m1", 256, 512, "tc"), ("e2m1", 128, 512, "rowmajor")):
        layer = MxExpertLinear(torch.zeros(3, out_f, in_f, dtype=BF), fmt)
        assert layer.layout == layout and layer.align == 32
        rows, (row_of, offsets, counts) = layer.dispatch(torch.zeros(7, in_f, dtype=BF),
                                                         torch.zeros(7, 2, dtype=torch.int64))
        assert rows.shape == (mxq.expert_rows(14, 3, 32), in_f)
        y, saved = layer.forward(rows, offsets)
        drows, dw = layer.backward(y, saved, offsets)
        assert drows.shape == rows.shape and dw.shape == (3, out_f, in_f) and dw.dtype is F32
        assert layer.infer(rows[:9], offsets).shape == (9, out_f)
    assert MxExpertLinear(torch.zeros(1, 32, 32, dtype=BF), wgrad_fmt="e2m1").align == 64


def test_layer_dispatches_a_servers_tokens_without_padding(fake):
    layer = MxExpertLinear(torch.zeros(64, 128, 256, dtype=BF))
    x, ids = torch.zeros(1, 256, dtype=BF), torch.zeros(1, 8, dtype=torch.int64)
    rows, (row_of, offsets, counts) = layer.dispatch(x, ids, padded=False)
    assert rows.shape == (8, 256) and fake[-2][0] == "mxq_expert_order" and fake[-2][1][4] == 1
    assert layer.infer(rows, offsets).shape == (8, 128)
    assert layer.dispatch(x, ids)[0].shape == (256, 256) and fake[-2][1][4] == 32


def test_adamw_bindings(fake):
    params = [torch.zeros(5, 7), torch.zeros(300), torch.zeros(0)]
    for bits in (32, 8):
        states = [mxq.adamw_state(p, bits) for p in params]
        copies = [torch.zeros(5, 7, dtype=BF), None, None]
        plan = mxq.adamw_plan(params, states, copies, weight_decay=[0.1, 0.0, 0.2])
        grads = [torch.zeros_like(p) for p in params]
        mxq.adamw_step(plan, grads, 3, 1e-3)
        mxq.adamw_step(plan, [g.bfloat16() for g in grads], torch.ones(1, dtype=torch.int64),
                       torch.ones(1), grad_scale=torch.ones(1))
        name, (table, places, count, args, _) = fake[-1]
        assert count == 3 and len(table) == 3 * ctypes.sizeof(mxq.AdamWTensor)
        a = mxq.AdamWArgs.from_buffer_copy(args)
        assert a.grad_dtype == 1 and a.state_bits == bits and a.lr_at and a.step_at
        t = (mxq.AdamWTensor * 3).from_buffer_copy(table)
        assert [v.n for v in t] == [35, 300, 0] and t[0].copy and not t[1].copy
        assert t[0].param == params[0].data_ptr() and abs(t[0].weight_decay - 0.1) < 1e-8
        fake.clear()
        one = torch.ones(1)
        _refused([
            lambda: mxq.adamw_step(plan, grads[:2], 1, 1e-3),
            lambda: mxq.adamw_step(plan, [g.half() for g in grads], 1, 1e-3),
            lambda: mxq.adamw_step(plan, [grads[0].bfloat16()] + grads[1:], 1, 1e-3),
            lambda: mxq.adamw_step(plan, [grads[0][1:]] + grads[1:], 1, 1e-3),
            lambda: mxq.adamw_step(plan, [grads[0].t()] + grads[1:], 1, 1e-3),
            lambda: mxq.adamw_step(plan, [None] + grads[1:], 1, 1e-3),
            lambda: mxq.adamw_step(plan, [params[0]] + grads[1:], 1, 1e-3),
            lambda: mxq.adamw_step(plan, grads, one, 1e-3),
            lambda: mxq.adamw_step(plan, grads, 1, one.double()),
            lambda: mxq.adamw_step(plan, grads, 1, 1e-3, grad_scale=one.half())])
        assert not fake
    s = [mxq.adamw_state(p) for p in params]
    q = [mxq.adamw_state(p, 8) for p in params]
    p0 = params[0]
    _refused([
        lambda: mxq.adamw_state(p0, 16),
        lambda: mxq.adamw_plan(params, s[:2]), lambda: mxq.adamw_plan(params, s, [None]),
        lambda: mxq.adamw_plan(params, s, weight_decay=[0.0]),
        lambda: mxq.adamw_plan([p0.bfloat16()], s[:1]), lambda: mxq.adamw_plan([p0.t()], s[:1]),
        lambda: mxq.adamw_plan(params[:2], [s[0], q[1]]),
        lambda: mxq.adamw_plan(params[1:2], s[:1]),
        lambda: mxq.adamw_plan([p0], [(q[0][0], (q[0][1][0], q[0][1][1][:0]))]),
        lambda: mxq.adamw_plan([p0], s[:1], [p0]),
        lambda: mxq.adamw_plan([p0, p0], [s[0], mxq.adamw_state(p0)]),       # one tensor twice
        lambda: mxq.adamw_plan([p0], [(s[0][0], s[0][0])]),
        lambda: mxq.adamw_plan([params[1], params[1][200:]], [s[1], mxq.adamw_state(params[1][200:])])])
    mxq.adamw_step(mxq.adamw_plan([], []), [], 1, 1e-3)      # nothing to do
    assert not fake


def test_a_parameter_that_moved(fake):
    p = torch.zeros(300)
    plan = mxq.adamw_plan([p], [mxq.adamw_state(p)])
    first = plan.table()
    assert plan.table() is first
    p.data = torch.zeros(300)
    assert plan.table() != first
    assert mxq.AdamWTensor.from_buffer_copy(plan.table()).param == p.data_ptr()
    p.data = torch.zeros(200)
    with pytest.raises(ValueError):
        mxq.adamw_plan([p], [mxq.adamw_state(torch.zeros(100))])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("how", ["data", "freed", "shrunk", "grown"])
def test_a_moment_that_moved(fake, bits, how):
    # no step writes where a moment was: its memory may be another tensor's by now
    p = torch.zeros(300)
    flat = lambda state: [t for x in state for t in (x if bits == 8 else (x,))]
    for k in range(2 if bits == 32 else 4):
        state = mxq.adamw_state(p, bits)
        plan = mxq.adamw_plan([p], [state])
        first = plan.table()
        assert plan.table() is first
        t = flat(state)[k]
        if how == "data":
            t.data = t.clone()
        else:
            t.untyped_storage().resize_(8 if how == "shrunk" else 0)
            if how == "grown":
                t.resize_(2000)
        if how in ("freed", "shrunk"):
            with pytest.raises(ValueError):
                mxq.adamw_step(plan, [torch.zeros(300)], 1, 1e-3)
            assert not fake
            continue
        row = mxq.AdamWTensor.from_buffer_copy(plan.table())
        names = ("m", "v") if bits == 32 else ("m", "m_scale", "v", "r_scale")
        assert [getattr(row, n) for n in names] == [x.data_ptr() for x in flat(state)]


def test_a_parameter_with_another_view_of_its_memory(fake):
    # the same address, but other elements or another order than the plan's
    for weight in (False, True):
        p, w = torch.zeros(20, 15), torch.zeros(20, 15, dtype=BF)
        plan = mxq.adamw_plan([p], [mxq.adamw_state(p)], [w])
        t, whole = (w, w.data) if weight else (p, p.data)
        grads = [torch.zeros(20, 15)]
        t.data = whole.t()
        _refused([lambda: mxq.adamw_step(plan, grads, 1, 1e-3)], ValueError)
        t.data = whole[:10]
        _refused([lambda: mxq.adamw_step(plan, grads, 1, 1e-3)], ValueError)
        assert not fake
        if not weight:      # a shorter parameter goes with gradients of its size
            mxq.adamw_step(plan, [torch.zeros(10, 15)], 1, 1e-3)
            assert mxq.AdamWTensor.from_buffer_copy(fake[-1][1][0]).n == 150
        t.data = whole
        mxq.adamw_step(plan, grads, 1, 1e-3)
        assert mxq.AdamWTensor.from_buffer_copy(fake[-1][1][0]).n == 300
        fake.clear()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_gradient_that_overlaps_what_is_written(fake, bits):
    # all of it from one buffer, 1200 bytes to a piece: parameter, gradient, weight, states
    byte = torch.zeros(20000, dtype=U8)
    cut = lambda at, n, dtype: byte[at:at + n * (torch.ones(1, dtype=dtype).element_size())].view(dtype)
    p, w = cut(1200, 300, F32), cut(3600, 300, BF)
    state = (cut(6000, 300, F32), cut(7200, 300, F32)) if bits == 32 else \
        ((cut(6000, 300, U8), cut(7200, 3, F32)), (cut(8400, 300, U8), cut(9600, 3, F32)))
    plan = mxq.adamw_plan([p], [state], [w])
    grad = lambda at, dtype=F32: mxq.adamw_step(plan, [cut(at, 300, dtype)], 1, 1e-3)
    for at in (0, 2400, 4800, 12000):      # between the pieces, up to their first bytes
        grad(at)
        grad(at)
    grad(600, BF)
    assert len(fake) == 9
    fake.clear()
    ends = (8396,) if bits == 32 else (6296, 7208, 8696, 9608)
    starts = (6000, 7200) if bits == 32 else (6000, 7200, 8400, 9600)
    _refused([lambda at=at: grad(at) for at in
              (4, 1196, 1200, 1204, 2396, 2404, 3600, 4196) + starts + ends
              + tuple(s - 1196 for s in starts)] + [lambda: grad(604, BF), lambda: grad(1796, BF)],
             ValueError)
    # numbers in device memory are read while the tensors are written
    one, step = torch.ones(1), torch.ones(2, dtype=torch.int64)
    g = [torch.zeros(300)]
    _refused([lambda: mxq.adamw_step(plan, g, 1, p[299:]), lambda: mxq.adamw_step(plan, g, 1, 1e-3,
                                                                              grad_scale=p[:1]),
              lambda: mxq.adamw_step(plan, g, cut(7200, 1, torch.int64), 1e-3)], ValueError)
    assert not fake
    mxq.adamw_step(plan, g, step, one, grad_scale=one)
    # an empty parameter's gradient is nowhere
    empty = mxq.adamw_plan([p, torch.zeros(0)], [state, mxq.adamw_state(torch.zeros(0), bits)])
    mxq.adamw_step(empty, [torch.zeros(300), p[:0]], 1, 1e-3)
    # the parameter moves to where the gradient is
    plan = mxq.adamw_plan([p], [state])
    mxq.adamw_step(plan, g, 1, 1e-3)
    p.data = g[0].data
    _refused([lambda: mxq.adamw_step(plan, g, 1, 1e-3)], ValueError)


def test_a_plan_keeps_the_states_it_was_given(fake):
    p, other = torch.zeros(300), torch.zeros(300)
    m, v = mxq.adamw_state(p)
    state = [m, v]
    plan = mxq.adamw_plan([p], [state])
    state[0] = other
    p.data = torch.zeros(300)
    assert mxq.AdamWTensor.from_buffer_copy(plan.table()).m == m.data_ptr()


# ---- the oracle itself ---------------------------------------------------------------------

def test_oracle_order_by_hand():
    ids = np.array([[1, 0], [1, 5], [0, 1]])
    row_of, offsets, counts = E.order(ids, 3, 4)
    assert counts.tolist() == [2, 3, 0] and offsets.tolist() == [0, 4, 8, 8]
    assert row_of.tolist() == [[4, 0], [5, -1], [1, 6]]


def test_oracle_adamw_by_hand():
    # first step: m / (1 - b1) = g, v / (1 - b2) = g^2, so p moves by lr sign(g) and decays
    p, m, v, u = E.adamw(np.array([1.0, -2.0]), np.array([0.5, -4.0]), np.zeros(2), np.zeros(2), 1,
                         0.1, 0.9, 0.99, 0.0, 0.01)
    assert np.allclose(p, [1 - 0.001 - 0.1, -2 + 0.002 + 0.1]) and np.allclose(u, 0.1)
    assert np.allclose(m, [0.05, -0.4]) and np.allclose(v, [0.0025, 0.16])


def test_oracle_combine_gradients_are_differences():
    rng = np.random.default_rng(0)
    row_of = np.array([[0, 3], [2, -1], [1, 4]])
    y, w, d = rng.standard_normal((5, 4)), rng.standard_normal((3, 2)), rng.standard_normal((3, 4))
    f = lambda y, w: (E.combine(y, row_of, w)[0] * d).sum()
    dy = E.gather(d, row_of, np.array([0, 5]), np.array([5]), np.zeros((5, 4)), w)
    dw = E.combine_dweights(d, y, row_of)[0]
    for i in np.ndindex(y.shape):
        h = np.zeros_like(y)
        h[i] = 1e-5
        assert abs((f(y + h, w) - f(y - h, w)) / 2e-5 - dy[i]) < 1e-8
    for i in np.ndindex(w.shape):
        h = np.zeros_like(w)
        h[i] = 1e-5
        assert abs((f(y, w + h) - f(y, w - h)) / 2e-5 - dw[i]) < 1e-8
