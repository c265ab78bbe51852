"""Cases of the block-128 FP8 operators and of the norms that feed them.

Three groups of operators, as a quantized pre-norm linear layer uses them:

* quantization of a bf16 tensor to FP8 codes with one fp32 scale per block of
  128 (along rows, along columns stored transposed, both in one pass, or per
  128x128 tile with the transposed codes);
* the matrix product of such codes, C = dec(A) dec(B)^T, with the scales of B
  per tile (a weight) or per line and 128 elements (the weight gradient);
* layer norm and RMS norm: forward, forward straight to FP8 codes, backward
  with the gradients of weight and bias.

``own`` False computes a case in elementary torch operations in 32 bits;
``own`` True calls this repository's operators on the same state.
"""

import math

import torch

own = False

BLOCK = 128
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FLOATS = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 2.0 ** -126   # smallest scale
EPS = 1e-5


def listed():
    return [
        # a training layer's input activation: forward and weight-gradient operand in one pass
        {"name": "quantize-dual 8192x4096", "op": "quantize", "mode": "dual", "rows": 8192,
         "cols": 4096, "fmt": "e4m3"},
        # the gate+up weight after an optimizer step: forward and dgrad operand
        {"name": "quantize-tiles 28672x4096", "op": "quantize", "mode": "tiles", "rows": 28672,
         "cols": 4096, "fmt": "e4m3"},
        # one token's activation in front of the down projection: latency
        {"name": "quantize-row 1x14336", "op": "quantize", "mode": "row", "rows": 1,
         "cols": 14336, "fmt": "e4m3"},
        # an output gradient of a ragged micro-batch, wide range, as weight-gradient operand
        {"name": "quantize-col 1237x1001 e5m2", "op": "quantize", "mode": "col", "rows": 1237,
         "cols": 1001, "fmt": "e5m2"},
        # forward product of the QKV projection of a training step
        {"name": "gemm fwd 8192x6144x4096", "op": "gemm", "m": 8192, "n": 6144, "k": 4096,
         "fmt_a": "e4m3", "fmt_b": "e4m3", "scales": "tile", "out": "bf16"},
        # weight gradient of the gate+up projection, fp32 for the optimizer
        {"name": "gemm wgrad 28672x4096x8192", "op": "gemm", "m": 28672, "n": 4096, "k": 8192,
         "fmt_a": "e4m3", "fmt_b": "e4m3", "scales": "line", "out": "f32"},
        # one token through the down projection: the weight's bytes and latency
        {"name": "gemm decode 1x4096x14336", "op": "gemm", "m": 1, "n": 4096, "k": 14336,
         "fmt_a": "e4m3", "fmt_b": "e4m3", "scales": "tile", "out": "bf16"},
        # a ragged micro-batch's input gradient, E5M2 gradient against an E4M3 weight
        {"name": "gemm dgrad 333x1001x1234", "op": "gemm", "m": 333, "n": 1001, "k": 1234,
         "fmt_a": "e5m2", "fmt_b": "e4m3", "scales": "tile", "out": "bf16"},
        # the pre-attention norm of a training step
        {"name": "rms fwd 8192x4096", "op": "norm", "kind": "rms", "rows": 8192, "cols": 4096,
         "dtype": "bf16", "wdtype": "bf16"},
        # the norm of a decode batch, straight to the projection's operand
        {"name": "rms quantize 32x4096", "op": "norm_quantize", "kind": "rms", "rows": 32,
         "cols": 4096, "dtype": "bf16", "wdtype": "bf16"},
        # backward of the pre-attention norm of a training step
        {"name": "layer bwd 8192x4096", "op": "norm_backward", "kind": "layer", "rows": 8192,
         "cols": 4096, "dtype": "bf16", "wdtype": "f32"},
        # odd sizes, fp32 residual stream
        {"name": "layer bwd 517x1001 f32", "op": "norm_backward", "kind": "layer", "rows": 517,
         "cols": 1001, "dtype": "f32", "wdtype": "f32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "norm", "norm_quantize", "norm_backward"])
    if op == "quantize":
        # tokens x features, or a weight, up to the listed weight's size
        cols = _log_int(rng, 33, 28672)
        rows = _log_int(rng, 1, min(32768, 28672 * 4096 // cols))
        if rng.random() < 0.5:
            cols = (cols + 15) // 16 * 16
        return {"op": op, "mode": rng.choice(["row", "col", "dual", "tiles"]), "rows": rows,
                "cols": cols, "fmt": rng.choice(["e4m3", "e4m3", "e5m2"])}
    if op == "gemm":
        n = _log_int(rng, 40, 28672)
        k = _log_int(rng, 40, 16384)
        m = _log_int(rng, 1, min(28672, 28672 * 4096 * 8192 // (n * k)))
        if rng.random() < 0.5:
            n = (n + 7) // 8 * 8
        return {"op": op, "m": m, "n": n, "k": k, "fmt_a": rng.choice(["e4m3", "e5m2"]),
                "fmt_b": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "scales": rng.choice(["tile", "line"]), "out": rng.choice(["bf16", "f32"])}
    cols = _log_int(rng, 33, 16384)
    if rng.random() < 0.6:
        cols = (cols + 7) // 8 * 8
    rows = _log_int(rng, 1, min(32768, (1 << 26) // cols))
    return {"op": op, "kind": rng.choice(["rms", "layer"]), "rows": rows, "cols": cols,
            "dtype": rng.choice(["bf16", "bf16", "f32"]), "wdtype": rng.choice(["bf16", "f32"])}


# ---- inputs ---------------------------------------------------------------------

def _student(rows, cols, g):
    """Student-t(3) times a per-channel LogNormal(0, 1): heavy tails, outlier channels."""
    z = torch.randn(rows, cols, device="cuda", generator=g)
    v = torch.randn(rows, cols, device="cuda", generator=g).square_()
    v += torch.randn(rows, cols, device="cuda", generator=g).square_()
    v += torch.randn(rows, cols, device="cuda", generator=g).square_()
    col = torch.randn(1, cols, device="cuda", generator=g).exp_()
    return z.div_(v.div_(3.0).sqrt_().clamp_min_(1e-6)).mul_(col)


def _out_grad(rows, cols, g):
    """N(0, 1e-3) times a per-column LogNormal(0, 2)."""
    z = torch.randn(rows, cols, device="cuda", generator=g).mul_(1e-3)
    return z.mul_(torch.randn(1, cols, device="cuda", generator=g).mul_(2.0).exp_())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        if case["mode"] == "tiles":
            x = torch.randn(r, c, device="cuda", generator=g).mul_(0.02)
        elif case["fmt"] == "e5m2":
            x = _out_grad(r, c, g)
        else:
            x = _student(r, c, g)
        s["x"] = x.to(torch.bfloat16)
    elif case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        a = (_out_grad(m, k, g) if case["fmt_a"] == "e5m2" else _student(m, k, g))
        s["A"], s["sA"] = _quantize_lines(a.to(torch.bfloat16), case["fmt_a"])
        del a
        if case["scales"] == "tile":
            b = torch.randn(n, k, device="cuda", generator=g).mul_(0.02)
            s["B"], s["sB"] = _quantize_tiles(b.to(torch.bfloat16), case["fmt_b"])[:2]
        else:
            b = _student(n, k, g)
            s["B"], s["sB"] = _quantize_lines(b.to(torch.bfloat16), case["fmt_b"])
    else:
        r, c = case["rows"], case["cols"]
        dt, wdt = FLOATS[case["dtype"]], FLOATS[case["wdtype"]]
        x = torch.randn(r, c, device="cuda", generator=g)
        x.mul_(torch.randn(1, c, device="cuda", generator=g).mul_(0.5).exp_())
        x.add_(torch.randn(r, 1, device="cuda", generator=g).mul_(0.3))
        s["x"] = x.to(dt)
        s["weight"] = torch.randn(c, device="cuda", generator=g).mul_(0.1).add_(1.0).to(wdt)
        s["bias"] = None
        if case["kind"] == "layer":
            s["bias"] = torch.randn(c, device="cuda", generator=g).mul_(0.1).to(wdt)
        if case["op"] == "norm_backward":
            s["dy"] = torch.randn(r, c, device="cuda", generator=g).to(dt)
            s["mean"], s["rstd"] = _stats(s["x"].float(), case["kind"])
    return s


# ---- the plain forms ------------------------------------------------------------

def _up(n, m):
    return (n + m - 1) // m * m


def _scale(amax, fmt):
    return (amax / torch.full_like(amax, FMAX[fmt])).clamp_min(TINY)


def _encode(x, scale, fmt):
    q = x * (torch.ones_like(scale) / scale)
    return q.clamp(-FMAX[fmt], FMAX[fmt]).to(FP8[fmt]).view(torch.uint8)


def _padded(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[1], 0, rows - x.shape[0]))


def _quantize_lines(x, fmt):
    """Codes [lines][K up to 16] and scales [K blocks][lines up to 4] of x [lines][K]."""
    lines, k = x.shape
    kb = _up(k, BLOCK) // BLOCK
    v = _padded(x.float(), _up(lines, 4), kb * BLOCK).view(-1, kb, BLOCK)
    s = _scale(v.abs().amax(-1), fmt)
    q = _encode(v, s[:, :, None], fmt).view(-1, kb * BLOCK)
    return q[:lines, :_up(k, 16)].contiguous(), s.t().contiguous()


def _quantize_tiles(x, fmt):
    """Codes, scales [row tiles][column tiles], and both transposed, of x [rows][cols]."""
    r, c = x.shape
    rb, cb = _up(r, BLOCK) // BLOCK, _up(c, BLOCK) // BLOCK
    v = _padded(x.float(), rb * BLOCK, cb * BLOCK).view(rb, BLOCK, cb, BLOCK)
    s = _scale(v.abs().amax(3).amax(1), fmt)
    q = _encode(v, s[:, None, :, None], fmt).view(rb * BLOCK, cb * BLOCK)
    return (q[:r, :_up(c, 16)].contiguous(), s, q.t()[:c, :_up(r, 16)].contiguous(),
            s.t().contiguous())


def _decode_lines(codes, scales, k, fmt, dtype):
    v = codes.view(FP8[fmt])[:, :k].to(dtype)
    s = scales[:, :codes.shape[0]].t().to(dtype)
    return v * s.repeat_interleave(BLOCK, 1)[:, :k]


def _decode_tiles(codes, scales, k, fmt, dtype):
    n = codes.shape[0]
    v = codes.view(FP8[fmt])[:, :k].to(dtype)
    s = scales.to(dtype).repeat_interleave(BLOCK, 0)[:n]
    return v * s.repeat_interleave(BLOCK, 1)[:, :k]


def _product(s, dtype):
    a = _decode_lines(s["A"], s["sA"], s["k"], s["fmt_a"], dtype)
    decode = _decode_tiles if s["scales"] == "tile" else _decode_lines
    b = decode(s["B"], s["sB"], s["k"], s["fmt_b"], dtype)
    return a @ b.t()


def _stats(x, kind):
    mean = x.mean(1) if kind == "layer" else None
    d = x - mean[:, None] if kind == "layer" else x
    return mean, 1.0 / torch.sqrt((d * d).mean(1) + EPS)


def _norm(x, weight, bias, kind):
    mean, rstd = _stats(x, kind)
    d = x - mean[:, None] if kind == "layer" else x
    y = d * rstd[:, None] * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def _norm_backward(dy, x, weight, mean, rstd, kind):
    h = (x - mean[:, None] if kind == "layer" else x) * rstd[:, None]
    g = dy * weight
    dx = g - h * (g * h).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(1, keepdim=True)
    out = {"dx": dx * rstd[:, None], "dweight": (dy * h).sum(0)}
    if kind == "layer":
        out["dbias"] = dy.sum(0)
    return out


def _plain(s):
    op = s["op"]
    if op == "quantize":
        x, fmt, mode = s["x"], s["fmt"], s["mode"]
        if mode == "row":
            return _named(mode, _quantize_lines(x, fmt), fmt)
        if mode == "col":
            return _named(mode, _quantize_lines(x.t(), fmt), fmt)
        if mode == "dual":
            return _named(mode, _quantize_lines(x, fmt) + _quantize_lines(x.t(), fmt), fmt)
        return _named(mode, _quantize_tiles(x, fmt), fmt)
    if op == "gemm":
        return _product(s, torch.float32).to(FLOATS[s["out"]])
    x, w = s["x"].float(), s["weight"].float()
    b = None if s["bias"] is None else s["bias"].float()
    if op == "norm":
        y, mean, rstd = _norm(x, w, b, s["kind"])
        return _norm_out(y.to(s["x"].dtype), mean, rstd)
    if op == "norm_quantize":
        y, mean, rstd = _norm(x, w, b, s["kind"])
        codes, scales = _quantize_lines(y, "e4m3")
        return _norm_out((codes.view(FP8["e4m3"]), scales), mean, rstd)
    out = _norm_backward(s["dy"].float(), x, w, s["mean"], s["rstd"], s["kind"])
    out["dx"] = out["dx"].to(s["x"].dtype)
    return out


def _named(mode, out, fmt):
    """The quantizers' outputs, codes as the values they stand for."""
    return [t.view(FP8[fmt]) if t.dtype == torch.uint8 else t for t in out]


def _norm_out(y, mean, rstd):
    out = {"y": y, "rstd": rstd}
    if mean is not None:
        out["mean"] = mean
    return out


# ---- the framework's operators --------------------------------------------------

def _own(s):
    from precision_mx_quantize_gb300 import mxq
    op = s["op"]
    if op == "quantize":
        x, fmt, mode = s["x"], s["fmt"], s["mode"]
        if mode in ("row", "col"):
            return _named(mode, mxq.fp8_quantize(x, mode, fmt), fmt)
        if mode == "dual":
            return _named(mode, mxq.fp8_quantize_dual(x, fmt, fmt), fmt)
        return _named(mode, mxq.fp8_quantize_tiles(x, fmt), fmt)
    if op == "gemm":
        return mxq.fp8_gemm(s["A"], s["sA"], s["B"], s["sB"], s["m"], s["n"], s["k"],
                            fmt_a=s["fmt_a"], fmt_b=s["fmt_b"], b_scales=s["scales"],
                            out_dtype=FLOATS[s["out"]])
    layer = s["kind"] == "layer"
    if op == "norm":
        if layer:
            return _norm_out(*mxq.layer_norm(s["x"], s["weight"], s["bias"], EPS))
        y, rstd = mxq.rms_norm(s["x"], s["weight"], EPS)
        return _norm_out(y, None, rstd)
    if op == "norm_quantize":
        if layer:
            c, sc, mean, rstd = mxq.layer_norm_quantize(s["x"], s["weight"], s["bias"], EPS)
        else:
            c, sc, rstd = mxq.rms_norm_quantize(s["x"], s["weight"], EPS)
            mean = None
        return _norm_out((c.view(FP8["e4m3"]), sc), mean, rstd)
    if layer:
        dx, dw, db = mxq.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    dx, dw = mxq.rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"])
    return {"dx": dx, "dweight": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ---- bytes and operations -------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "quantize":
        r, c, mode = case["rows"], case["cols"], case["mode"]
        kb_r, kb_c = _up(c, BLOCK) // BLOCK, _up(r, BLOCK) // BLOCK
        row, col = r * _up(c, 16) + 4 * r * kb_r, c * _up(r, 16) + 4 * c * kb_c
        if mode == "tiles":
            out = r * _up(c, 16) + c * _up(r, 16) + 8 * kb_r * kb_c
        else:
            out = {"row": row, "col": col, "dual": row + col}[mode]
        return {"bytes": 2 * r * c + out, "flops": (6 if mode == "dual" else 4) * r * c}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = _up(k, BLOCK) // BLOCK
        sb = (_up(n, BLOCK) // BLOCK if case["scales"] == "tile" else n) * kb * 4
        out = m * n * (2 if case["out"] == "bf16" else 4)
        return {"bytes": (m + n) * k + m * kb * 4 + sb + out, "flops": 2 * m * n * k}
    r, c = case["rows"], case["cols"]
    e, we = (2 if case["dtype"] == "bf16" else 4), (2 if case["wdtype"] == "bf16" else 4)
    layer = case["kind"] == "layer"
    vec, stats = c * we * (2 if layer else 1), 4 * r * (2 if layer else 1)
    if op == "norm":
        return {"bytes": 2 * r * c * e + vec + stats, "flops": 8 * r * c}
    if op == "norm_quantize":
        out = r * _up(c, 16) + 4 * r * (_up(c, BLOCK) // BLOCK)
        return {"bytes": r * c * e + out + vec + stats, "flops": 12 * r * c}
    grads = 4 * c * (2 if layer else 1)
    return {"bytes": 3 * r * c * e + c * we + stats + grads, "flops": 14 * r * c}


# ---- the definitions in 64 bits -------------------------------------------------

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits: a code's place holds
    the value before its rounding to 8 bits."""
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "quantize":
        x, fmt, mode = s["x"].to(f64), case["fmt"], case["mode"]

        def blocks(v, br):
            """(v / scale with its zero padding, scales) for blocks of br x 128."""
            r, c = v.shape
            rp = _up(r, br if br > 1 else 4)
            nb, cb = rp // br, _up(c, BLOCK) // BLOCK
            full = torch.zeros(rp, cb * BLOCK, dtype=f64, device=v.device)
            full[:r, :c] = v
            t = full.view(nb, br, cb, BLOCK)
            sc = torch.clamp(t.abs().amax(dim=(1, 3)) / FMAX[fmt], min=TINY)
            q = (t / sc.view(nb, 1, cb, 1)).view(rp, cb * BLOCK)
            return q, sc

        if mode == "tiles":
            q, sc = blocks(x, BLOCK)
            r, c = x.shape
            return [q[:r, :_up(c, 16)], sc, q.t()[:c, :_up(r, 16)], sc.t()]
        out = []
        for v in {"row": [x], "col": [x.t()], "dual": [x, x.t()]}[mode]:
            q, sc = blocks(v, 1)
            out += [q[:v.shape[0], :_up(v.shape[1], 16)], sc.t()]
        return out
    if op == "gemm":
        k = case["k"]

        def decoded(codes, scales, fmt, tile):
            v = codes.view(FP8[fmt]).to(f64)[:, :k]
            at = torch.arange(k, device=v.device) // BLOCK
            if tile:
                rt = torch.arange(v.shape[0], device=v.device) // BLOCK
                return v.mul_(scales.to(f64)[rt][:, at])
            return v.mul_(scales.to(f64)[:, :v.shape[0]].t()[:, at])

        a = decoded(s["A"], s["sA"], case["fmt_a"], False)
        b = decoded(s["B"], s["sB"], case["fmt_b"], case["scales"] == "tile")
        return torch.mm(a, b.t())
    x, w = s["x"].to(f64), s["weight"].to(f64)
    c, layer = x.shape[1], case["kind"] == "layer"
    if op == "norm_backward":
        dy, rstd = s["dy"].to(f64), s["rstd"].to(f64)[:, None]
        h = ((x - s["mean"].to(f64)[:, None]) if layer else x) * rstd
        wdy = dy * w
        c2 = torch.einsum("rc,rc->r", wdy, h)[:, None] / c
        c1 = wdy.sum(1, keepdim=True) / c if layer else 0.0
        out = {"dx": rstd * (wdy - c1 - h * c2), "dweight": torch.einsum("rc,rc->c", dy, h)}
        if layer:
            out["dbias"] = dy.sum(0)
        return out
    mean = x.sum(1) / c if layer else None
    h = x - mean[:, None] if layer else x
    rstd = (torch.einsum("rc,rc->r", h, h) / c + EPS) ** -0.5
    y = h * rstd[:, None] * w
    if layer:
        y = y + s["bias"].to(f64)
    if op == "norm_quantize":
        r, kb = y.shape[0], _up(c, BLOCK) // BLOCK
        full = torch.zeros(_up(r, 4), kb * BLOCK, dtype=f64, device=y.device)
        full[:r, :c] = y
        t = full.view(-1, kb, BLOCK)
        sc = torch.clamp(t.abs().amax(2) / FMAX["e4m3"], min=TINY)
        q = (t / sc[:, :, None]).view(-1, kb * BLOCK)[:r, :_up(c, 16)]
        y = (q, sc.t())
    out = {"y": y, "rstd": rstd}
    if layer:
        out["mean"] = mean
    return out
