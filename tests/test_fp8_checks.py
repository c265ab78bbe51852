"""Refusals of the block-128 FP8 operators and the norms (CPU): the C entry
points reject bad arguments before any device work, the binding rejects
tensors that do not fit the sizes, and the argument structures have the C
layout."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from precision_mx_quantize_gb300 import mxq
from tests.libutil import ensure_built

P = ctypes.c_void_p(16 * 1024)   # never dereferenced: every call fails its checks
ODD = ctypes.c_void_p(16 * 1024 + 2)
ROW, COL, E4, E2, E5 = mxq.ROWWISE, mxq.COLWISE_T, mxq.E4M3, mxq.E2M1, mxq.E5M2


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_built()


def test_sizes():
    assert [mxq.lib().mxq_fp8_pitch(n) for n in (1, 16, 17, 4096)] == [16, 16, 32, 4096]
    assert mxq.lib().mxq_fp8_pitch(0) == mxq.lib().mxq_fp8_pitch(-3) == 0
    n = mxq.lib().mxq_fp8_scale_count
    for lines, blocked in ((1, 1), (5, 129), (128, 128), (300, 1000)):
        for name, kind in (("line", mxq.FP8_LINES), ("tile", mxq.FP8_TILES)):
            ss = mxq.fp8_shapes(lines, blocked, name)[1]
            assert n(lines, blocked, kind) == ss[0] * ss[1]
    assert n(0, 5, 0) == n(5, 0, 0) == n(5, 5, 2) == 0


def test_quantizer_refusals():
    q, d, t = mxq.mxq_fp8_quantize, mxq.mxq_fp8_quantize_dual, mxq.mxq_fp8_quantize_tiles
    assert q(P, 0, 64, ROW, E4, P, P, None) == 0 and q(None, 64, 0, ROW, E4, None, None, None) == 0
    for bad in ((P, -1, 64, ROW, E4, P, P), (P, 64, 2 ** 31, ROW, E4, P, P),
                (P, 64, 64, 2, E4, P, P), (P, 64, 64, ROW, E2, P, P), (P, 64, 64, ROW, 9, P, P),
                (None, 64, 64, ROW, E4, P, P), (P, 64, 64, COL, E4, None, P),
                (P, 64, 64, COL, E4, P, None)):
        assert q(*bad, None) == 1, bad
    for bad in ((ODD, 64, 64, ROW, E4, P, P), (P, 64, 64, ROW, E4, ODD, P),
                (P, 64, 64, ROW, E4, P, ODD)):
        assert q(*bad, None) == 2, bad
    assert d(P, 64, 64, E4, P, P, E2, P, P, None) == 1
    assert d(P, 64, 64, E4, P, P, E4, None, P, None) == 1
    assert d(P, 64, 64, E4, P, P, E4, ODD, P, None) == 2
    assert t(P, 64, 64, E2, P, P, P, P, None) == 1
    assert t(P, 64, 64, E4, P, P, P, None, None) == 1     # both transposed outputs or none
    assert t(P, 64, 64, E4, P, P, ODD, P, None) == 2
    assert t(P, 64, 64, E4, P, ODD, P, P, None) == 2


def test_product_refusals():
    g = mxq.mxq_fp8_gemm
    ok = dict(A=P, sA=P, fa=E4, B=P, sB=P, fb=E4, bs=1, M=8, N=8, K=8, C=P, od=0)

    def call(**kw):
        a = {**ok, **kw}
        return g(a["A"], a["sA"], a["fa"], a["B"], a["sB"], a["fb"], a["bs"], a["M"], a["N"],
                 a["K"], a["C"], a["od"], None)

    assert call(M=0) == 0 and call(N=0, C=None) == 0
    for kw in (dict(M=-1), dict(N=2 ** 31), dict(K=-5), dict(fa=E2), dict(fb=7), dict(bs=2),
               dict(od=2), dict(A=None), dict(sA=None), dict(B=None), dict(sB=None), dict(C=None)):
        assert call(**kw) == 1, kw
    for kw in (dict(A=ODD), dict(B=ODD), dict(C=ODD), dict(sA=ODD), dict(sB=ODD),
               dict(sB=ctypes.c_void_p(16 * 1024 + 4), bs=0)):
        assert call(**kw) == 2, kw


def _norm_args(**kw):
    a = mxq.NormArgs(P.value, P.value, None, P.value, P.value, P.value, None, None, 4, 64, 1e-5,
                     mxq.NORM_LAYER, 0, 0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return mxq.mxq_norm_forward(ctypes.addressof(a), None)


def test_norm_refusals():
    p, odd = P.value, ODD.value
    assert mxq.mxq_norm_forward(None, None) == 1
    assert _norm_args(rows=0) == 0 and _norm_args(cols=0) == 0
    for kw in (dict(rows=-1), dict(cols=2 ** 31), dict(kind=2), dict(x_dtype=2), dict(w_dtype=-1),
               dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(weight=None),
               dict(y=None), dict(codes=p), dict(codes=p, scales=p, fmt=E2),
               dict(kind=mxq.NORM_RMS)):    # RMS norm has no mean
        assert _norm_args(**kw) == 1, kw
    for kw in (dict(x=odd), dict(weight=odd), dict(bias=odd), dict(y=odd),
               dict(codes=odd, scales=p), dict(codes=p, scales=odd)):
        assert _norm_args(**kw) == 2, kw


def _grad_args(**kw):
    a = mxq.NormGradArgs(P.value, P.value, P.value, P.value, P.value, P.value, P.value, P.value,
                         P.value, 1 << 30, 4, 64, mxq.NORM_LAYER, 0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return mxq.mxq_norm_backward(ctypes.addressof(a), None)


def test_norm_backward_refusals():
    odd = ODD.value
    assert mxq.mxq_norm_backward(None, None) == 1
    assert _grad_args(cols=0) == 0
    for kw in (dict(rows=-1), dict(kind=5), dict(kind=mxq.NORM_RMS), dict(x_dtype=3), dict(dy=None), dict(x=None),
               dict(weight=None), dict(mean=None), dict(rstd=None), dict(dx=None),
               dict(dweight=None), dict(workspace=None)):
        assert _grad_args(**kw) == 1, kw
    for kw in (dict(dy=odd), dict(x=odd), dict(weight=odd), dict(dx=odd), dict(workspace=odd)):
        assert _grad_args(**kw) == 2, kw
    need = mxq.mxq_norm_backward_workspace_size(4, 64)
    assert need > 0 and _grad_args(workspace_bytes=need - 1) == 6
    assert mxq.mxq_norm_backward_workspace_size(0, 64) == 0
    assert mxq.mxq_norm_backward_workspace_size(-1, 64) == 0


@pytest.mark.parametrize("struct, name", [(mxq.NormArgs, "mxq_norm_args"),
                                          (mxq.NormGradArgs, "mxq_norm_grad_args")])
def test_argument_structures_match_the_header(tmp_path, struct, name):
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
    # the packed form the binding passes: the same bytes as the mirror's
    packed = {"mxq_norm_args": mxq._NORM_ARGS, "mxq_norm_grad_args": mxq._NORM_GRAD_ARGS}[name]
    values = list(range(1, len(fields) + 1))
    assert packed.pack(*values) == bytes(struct(*values))


# ---- the binding's buffer checks, against recorders in place of the library --------

@pytest.fixture
def fake(monkeypatch):
    calls = []
    for name in ("mxq_fp8_quantize", "mxq_fp8_quantize_dual", "mxq_fp8_quantize_tiles",
                 "mxq_fp8_gemm", "mxq_norm_forward", "mxq_norm_backward"):
        monkeypatch.setattr(mxq, name, lambda *a, _n=name: calls.append(_n) or 0)
    monkeypatch.setattr(mxq, "_stream", lambda device=None: 0)
    monkeypatch.setattr(mxq, "_on_gpu", lambda t: True)
    return calls


def test_binding_accepts_its_own_buffers(fake):
    x = torch.zeros(70, 130, dtype=torch.bfloat16)
    a = mxq.fp8_quantize(x)
    mxq.fp8_quantize(x, out=a)
    d = mxq.fp8_quantize_dual(x)
    mxq.fp8_quantize_dual(x, out=d)
    w = mxq.fp8_quantize_tiles(x)
    mxq.fp8_quantize_tiles(x, out=w[:2] + (None, None))
    assert mxq.fp8_gemm(*a, *w[:2], 70, 70, 130).shape == (70, 70)
    mxq.fp8_gemm(*a, *a, 70, 70, 130, b_scales="line", out_dtype=torch.float32)
    v = torch.ones(130)
    y, mean, rstd = mxq.layer_norm(x, v, v)
    mxq.layer_norm_quantize(x, v, v)
    mxq.rms_norm_quantize(x, v)
    mxq.layer_norm_backward(y, x, v, mean, rstd)
    mxq.rms_norm_backward(y, x, v, mxq.rms_norm(x, v)[1])
    assert len(fake) == 14


def test_binding_refusals(fake):
    x = torch.zeros(70, 130, dtype=torch.bfloat16)
    a, w, v = mxq.fp8_quantize(x), mxq.fp8_quantize_tiles(x), torch.ones(130)
    mean = rstd = torch.zeros(70)
    fake.clear()
    bad = [
        lambda: mxq.fp8_quantize(x.float()),
        lambda: mxq.fp8_quantize(x.t()),
        lambda: mxq.fp8_quantize(x[0]),
        lambda: mxq.fp8_quantize(x, out=(a[0][1:], a[1])),
        lambda: mxq.fp8_quantize(x, out=(a[0], a[1].double())),
        lambda: mxq.fp8_quantize_dual(x, out=a + a),
        lambda: mxq.fp8_quantize_tiles(x, out=(w[0], w[1], w[2], None)),
        lambda: mxq.fp8_gemm(*a, *w[:2], 71, 70, 130),
        lambda: mxq.fp8_gemm(*a, *w[:2], 70, 70, 160),
        lambda: mxq.fp8_gemm(*a, *w[:2], 70, 70, 130, b_scales="line"),
        lambda: mxq.fp8_gemm(*a, *w[:2], 70, 70, 130, out_dtype=torch.float16),
        lambda: mxq.fp8_gemm(*a, *w[:2], 70, 70, 130, out=torch.empty(70, 69, dtype=x.dtype)),
        lambda: mxq.layer_norm(x.half(), v),
        lambda: mxq.layer_norm(x.t(), torch.ones(70)),
        lambda: mxq.layer_norm(x, v[1:]),
        lambda: mxq.layer_norm(x, v, v.bfloat16()),
        lambda: mxq.rms_norm(x, v, out=torch.empty(70, 130)),
        lambda: mxq.rms_norm_quantize(x, v, out=(a[0], a[1][:1])),
        lambda: mxq.layer_norm_backward(x.float(), x, v, mean, rstd),
        lambda: mxq.layer_norm_backward(x, x, v, mean[1:], rstd),
        lambda: mxq.rms_norm_backward(x, x, v, rstd.double()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            pytest.fail(f"case {i} was accepted")
    for f in (lambda: mxq.fp8_quantize(x, "diag"), lambda: mxq.fp8_quantize(x, fmt="e2m1"),
              lambda: mxq.fp8_gemm(*a, *w[:2], 70, 70, 130, b_scales="rows")):
        with pytest.raises(KeyError):
            f()
    with pytest.raises(TypeError):
        mxq.fp8_gemm(a[0], None, *w[:2], 70, 70, 130)
    assert not fake


# ---- the oracle itself ---------------------------------------------------------------

def test_oracle_by_hand():
    # one block: amax 7, scale 7 / 448 = 1/64; 7 -> 448, 1 -> 64, -0.5 -> -32
    x = np.zeros((1, 128), np.float32)
    x[0, :3] = 7.0, 1.0, -0.5
    c, s = F.quantize_lines(x, "e4m3")
    assert s.shape == (1, 4) and s[0, 0] == 1 / 64 and (s[0, 1:] == F.TINY).all()
    assert list(c[0, :4]) == [0x7E, 0x68, 0xE0, 0x00]
    assert (F.values(c, s, 128, "e4m3", "line") == x).all()
    ct = F.quantize_tiles(x, "e4m3")
    assert ct[1][0, 0] == 1 / 64 and ct[2].shape == (128, 16) and ct[2][1, 0] == 0x68


def test_oracle_norm_gradient_is_the_derivative():
    rng = np.random.default_rng(0)
    x, dy, w = rng.standard_normal((2, 9)), rng.standard_normal((2, 9)), rng.standard_normal(9)
    for kind in ("layer", "rms"):
        f = lambda v: (F.norm(v, w, None, 1e-5, kind)[0] * dy).sum()
        _, mean, rstd = F.norm(x, w, None, 1e-5, kind)
        dx = F.norm_backward(dy, x, w, mean, rstd, kind)[0]
        for i in np.ndindex(x.shape):
            d = np.zeros_like(x)
            d[i] = 1e-5
            assert abs((f(x + d) - f(x - d)) / 2e-5 - dx[i]) < 1e-8
