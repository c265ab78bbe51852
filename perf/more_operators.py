"""Cases of the operators around a layer of experts and of its optimizer step.

Three groups, as a mixture-of-experts layer on MX codes uses them:

* dispatch and combine: the rows of an expert-sorted buffer from the router's
  choices, the tokens gathered into it, the experts' outputs summed back with the
  router's weights, and the gradients of that sum;
* products grouped by expert: each row of A against the weight of the expert that
  holds it (forward and input gradient), and one product per expert over the rows
  that it holds (weight gradient), on MXFP8 or MXFP4 codes;
* an AdamW step over many tensors at once, with its two moments in fp32, or in
  8 bits with one fp32 scale per block of 128.

``own`` False computes a case in elementary torch operations in 32 bits;
``own`` True calls this repository's operators on the same state.
"""

import math

import torch

own = False

FLOATS = {"bf16": torch.bfloat16, "f32": torch.float32}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
EMAX = {"e4m3": 8, "e5m2": 15, "e2m1": 2}
VMAX = {"e4m3": 448.0, "e5m2": 57344.0, "e2m1": 6.0}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 128           # elements per scale of an 8-bit moment
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1


def listed():
    return [
        # the gate+up product of a training step: tokens of 8 choices each over 32 experts,
        # rows padded per expert for the weight gradient's blocks
        {"name": "experts fwd 4096x8 of 32", "op": "rows", "tokens": 4096, "topk": 8,
         "experts": 32, "n": 4096, "k": 4096, "fmt": "e4m3", "out": "bf16", "layout": "tc",
         "align": 32},
        # one token through its eight experts of 64, MXFP4 weights: their bytes and latency
        {"name": "experts token 1x8 of 64", "op": "rows", "tokens": 1, "topk": 8,
         "experts": 64, "n": 4096, "k": 4096, "fmt": "e2m1", "out": "bf16", "layout": "tc",
         "align": 1},
        # the input gradient of a ragged micro-batch, wide range, for an fp32 residual stream
        {"name": "experts dgrad 411x3 of 7", "op": "rows", "tokens": 411, "topk": 3,
         "experts": 7, "n": 1004, "k": 1056, "fmt": "e5m2", "out": "f32", "layout": "rowmajor",
         "align": 1},
        # weight gradients of all experts of a training step, MXFP4, fp32 for the optimizer
        {"name": "experts wgrad 4096x8 of 32", "op": "wgrad", "tokens": 4096, "topk": 8,
         "experts": 32, "m": 4096, "n": 2048, "fmt": "e2m1", "out": "f32", "align": 64},
        # weight gradients of a ragged micro-batch
        {"name": "experts wgrad 411x3 of 7", "op": "wgrad", "tokens": 411, "topk": 3,
         "experts": 7, "m": 1001, "n": 520, "fmt": "e4m3", "out": "bf16", "align": 32},
        # a training step's tokens to their experts' rows
        {"name": "dispatch 8192x8 of 64", "op": "dispatch", "tokens": 8192, "topk": 8,
         "experts": 64, "cols": 4096, "dtype": "bf16", "align": 32},
        # one token to its experts' rows: latency
        {"name": "dispatch 1x8 of 64", "op": "dispatch", "tokens": 1, "topk": 8, "experts": 64,
         "cols": 4096, "dtype": "bf16", "align": 1},
        # a training step's expert outputs back to their tokens
        {"name": "combine 8192x8 of 64", "op": "combine", "tokens": 8192, "topk": 8,
         "experts": 64, "cols": 4096, "dtype": "bf16", "align": 32},
        # gradients of that sum at odd sizes, fp32
        {"name": "combine bwd 4099x3 f32", "op": "combine_backward", "tokens": 4099, "topk": 3,
         "experts": 7, "cols": 1001, "dtype": "f32", "align": 32},
        # the optimizer step of a decoder block's weights and norms
        {"name": "adamw block 32-bit", "op": "adamw", "bits": 32, "grad": "f32", "copy": True,
         "shapes": "28672x4096,4096x14336,6144x4096,4096x4096,4096,4096"},
        # the optimizer step of 32 experts' weights with moments in 8 bits
        {"name": "adamw experts 8-bit", "op": "adamw", "bits": 8, "grad": "f32", "copy": True,
         "shapes": ",".join(["2048x1024"] * 32 + ["1001x517", "4096", "33"])},
        # norm weights and biases: many small tensors, latency
        {"name": "adamw norms 32-bit", "op": "adamw", "bits": 32, "grad": "bf16", "copy": False,
         "shapes": ",".join(["4096"] * 40 + ["1001"] * 8)},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rows", "rows", "wgrad", "dispatch", "combine", "combine_backward", "adamw"])
    if op == "adamw":
        # up to the listed block's size in up to 48 tensors
        left = _log_int(rng, 2000, 200_000_000)
        shapes = []
        while left > 0 and len(shapes) < 48:
            n = min(left, _log_int(rng, 1, 60_000_000))
            shapes.append(str(n))
            left -= n
        return {"op": op, "bits": rng.choice([8, 32]), "grad": rng.choice(["bf16", "f32"]),
                "copy": rng.random() < 0.6, "shapes": ",".join(shapes)}
    experts = _log_int(rng, 2, 160)
    topk = rng.randint(1, min(8, experts))
    if op in ("rows", "wgrad"):
        fmt = rng.choice(["e4m3", "e4m3", "e2m1", "e5m2"])
        align = {"e2m1": 64}.get(fmt, 32) if op == "wgrad" else rng.choice([1, 32])
        out = rng.choice(["bf16", "f32"])
        mult = 8 if out == "bf16" else 4
        n = (_log_int(rng, 40, 6144) + mult - 1) // mult * mult
        k = _log_int(rng, 40, 6144)
        k = (k + 31) // 32 * 32 if op == "rows" else k
        n = max(mult, min(n, (1 << 29) // (experts * k) // mult * mult))
        tokens = _log_int(rng, 1, max(1, min(32768, (1 << 38) // (n * k * topk))))
        if op == "wgrad":
            return {"op": op, "tokens": tokens, "topk": topk, "experts": experts, "m": k, "n": n,
                    "fmt": fmt, "out": out, "align": align}
        layout = "rowmajor"
        if k % (256 if fmt == "e2m1" else 128) == 0 and rng.random() < 0.7:
            layout = "tc"
        return {"op": op, "tokens": tokens, "topk": topk, "experts": experts, "n": n, "k": k,
                "fmt": fmt, "out": out, "layout": layout, "align": align}
    cols = _log_int(rng, 33, 8192)
    if rng.random() < 0.6:
        cols = (cols + 7) // 8 * 8
    tokens = _log_int(rng, 1, max(1, min(32768, (1 << 28) // (cols * topk))))
    return {"op": op, "tokens": tokens, "topk": topk, "experts": experts, "cols": cols,
            "dtype": rng.choice(["bf16", "bf16", "f32"]), "align": rng.choice([1, 32, 64])}


# ---- inputs ---------------------------------------------------------------------

def _up(n, m):
    return (n + m - 1) // m * m


def _capacity(case):
    """Rows that any choices of the case's experts fit in."""
    n, a = case["tokens"] * case["topk"], case["align"]
    return _up(n + min(case["experts"], n) * (a - 1), a)


def _choices(case, g):
    """(ids, weights): distinct experts of uneven popularity for each token, and the
    softmax of their scores."""
    scores = torch.randn(case["tokens"], case["experts"], device="cuda", generator=g)
    scores += torch.randn(case["experts"], device="cuda", generator=g).mul_(0.5)
    top, ids = scores.topk(case["topk"], dim=1)
    return ids.to(torch.int32), torch.softmax(top, 1)


def _offsets(case, ids):
    """First row of every expert, and the end of the last one's rows, on the host."""
    counts = torch.bincount(ids.flatten().long(), minlength=case["experts"]).tolist()
    at = [0]
    for c in counts:
        at.append(at[-1] + _up(c, case["align"]))
    return at


def _student(rows, cols, g):
    """Student-t(3) times a per-channel LogNormal(0, 1): heavy tails, outlier channels."""
    z = torch.randn(rows, cols, device="cuda", generator=g)
    v = torch.randn(rows, cols, device="cuda", generator=g).square_()
    v += torch.randn(rows, cols, device="cuda", generator=g).square_()
    v += torch.randn(rows, cols, device="cuda", generator=g).square_()
    col = torch.randn(1, cols, device="cuda", generator=g).exp_()
    return z.div_(v.div_(3.0).sqrt_().clamp_min_(1e-6)).mul_(col)


def _mx(x, fmt):
    """MX codes and row-major E8M0 scales of x [lines][blocked]."""
    lines, k = x.shape
    v = x.view(lines, k // 32, 32)
    _, e = torch.frexp(v.abs().amax(2))
    s = (e - 1 - EMAX[fmt] + 127).clamp_(0, 254)
    q = (v * torch.exp2((127 - s).float())[:, :, None]).clamp_(-VMAX[fmt], VMAX[fmt])
    q = q.view(lines, k)
    s = s.to(torch.uint8)
    if fmt != "e2m1":
        return q.to(FP8[fmt]).view(torch.uint8), s
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    c = torch.bucketize(q.abs(), mid, out_int32=True).to(torch.uint8)
    c += (q < 0).to(torch.uint8) * 8
    return c[:, 0::2] | (c[:, 1::2] << 4), s


def _chunks(s):
    """Row-major scales [lines][blocks] in the tensor cores' chunk layout: one chunk of
    512 bytes for 128 lines and 4 blocks."""
    lines, kb = s.shape
    full = torch.zeros(_up(lines, 128), kb, dtype=torch.uint8, device=s.device)
    full[:lines] = s
    t = full.view(-1, 4, 32, kb // 4, 4)              # tile, quarter, line, chunk, block
    return t.permute(0, 3, 2, 1, 4).reshape(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "adamw":
        return _prepare_adamw(s, g)
    ids, weights = _choices(case, g)
    rows = _capacity(case)
    s["rows"] = rows
    if case["op"] in ("rows", "wgrad"):
        at = _offsets(case, ids)
        s["at"] = at                                   # the same offsets on the host
        s["offsets"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        out = FLOATS[case["out"]]
    if case["op"] == "rows":
        n, k, fmt = case["n"], case["k"], case["fmt"]
        s["A"], s["sA"] = _mx(_student(rows, k, g), fmt)
        eb = k // 2 if fmt == "e2m1" else k
        s["B"] = torch.empty(case["experts"], n, eb, dtype=torch.uint8, device="cuda")
        s["sB_rows"] = torch.empty(case["experts"], n, k // 32, dtype=torch.uint8, device="cuda")
        for e in range(case["experts"]):
            w = torch.randn(n, k, device="cuda", generator=g).mul_(0.02)
            s["B"][e], s["sB_rows"][e] = _mx(w, fmt)
        s["sB"] = s["sB_rows"]
        if case["layout"] == "tc":
            s["sB"] = torch.stack([_chunks(t) for t in s["sB_rows"]])
        s["out_buffer"] = torch.zeros(rows, n, dtype=out, device="cuda")
    elif case["op"] == "wgrad":
        m, n, fmt = case["m"], case["n"], case["fmt"]
        live = torch.zeros(rows, device="cuda")        # rows of padding hold zeros
        counts = torch.bincount(ids.flatten().long(), minlength=case["experts"]).tolist()
        for e, c in enumerate(counts):
            live[at[e]:at[e] + c] = 1.0
        dy = torch.randn(m, rows, device="cuda", generator=g).mul_(1e-3)
        dy.mul_(torch.randn(m, 1, device="cuda", generator=g).exp_()).mul_(live)
        s["A"], s["sA"] = _mx(dy, fmt)
        x = torch.randn(n, rows, device="cuda", generator=g)
        x.mul_(torch.randn(n, 1, device="cuda", generator=g).exp_()).mul_(live)
        s["B"], s["sB"] = _mx(x, fmt)
    else:
        dt, t, c = FLOATS[case["dtype"]], case["tokens"], case["cols"]
        s["ids"], s["weights"] = ids, weights
        if case["op"] == "dispatch":
            s["x"] = torch.randn(t, c, device="cuda", generator=g).to(dt)
            s["out_buffer"] = torch.zeros(rows, c, dtype=dt, device="cuda")
        else:
            # what the dispatch left in the program's hands
            s["row_of"], s["offsets"], s["counts"] = _order(ids, case["experts"], case["align"])
            s["y"] = torch.randn(rows, c, device="cuda", generator=g).to(dt)
        if case["op"] == "combine_backward":
            s["dout"] = torch.randn(t, c, device="cuda", generator=g).to(dt)
            s["out_buffer"] = torch.zeros(rows, c, dtype=dt, device="cuda")
    return s


def _numels(case):
    return [math.prod(int(d) for d in t.split("x")) for t in case["shapes"].split(",")]


def _prepare_adamw(s, g):
    """The tensors as pieces of flat buffers, each from a multiple of 128 elements on;
    zeros between them."""
    at, total = [], 0
    for n in _numels(s):
        at.append((total, n))
        total += _up(n, BLOCK)
    live = torch.zeros(total, device="cuda")
    for a, n in at:
        live[a:a + n] = 1.0
    flat = {"param": torch.randn(total, device="cuda", generator=g).mul_(0.02).mul_(live)}
    width = torch.randn(total // BLOCK, 1, device="cuda", generator=g).exp_()
    grad = torch.randn(total // BLOCK, BLOCK, device="cuda", generator=g).mul_(1e-3).mul_(width)
    flat["grad"] = grad.view(-1).mul_(live).to(FLOATS[s["grad"]])
    m = torch.randn(total // BLOCK, BLOCK, device="cuda", generator=g).mul_(3e-4).mul_(width)
    r = torch.randn(total // BLOCK, BLOCK, device="cuda", generator=g).mul_(0.3).exp_()
    r.mul_(1e-3).mul_(width)
    m, r = m.view(-1).mul_(live), r.view(-1).mul_(live)
    if s["bits"] == 32:
        flat["m"], flat["v"] = m, r * r
    else:
        flat["m"], flat["m_scale"] = _moment_codes(m, False)
        flat["r"], flat["r_scale"] = _moment_codes(r, True)
    if s["copy"]:
        flat["copy"] = flat["param"].to(torch.bfloat16)
    s["flat"], s["step"] = flat, 1000
    cut = lambda name: [flat[name][a:a + n] for a, n in at]
    scales = lambda name: [flat[name][a // BLOCK:(a + _up(n, BLOCK)) // BLOCK] for a, n in at]
    s["params"], s["grads"] = cut("param"), cut("grad")
    if s["bits"] == 32:
        s["states"] = list(zip(cut("m"), cut("v")))
    else:
        s["states"] = list(zip(zip(cut("m"), scales("m_scale")), zip(cut("r"), scales("r_scale"))))
    s["copies"] = cut("copy") if s["copy"] else None
    return s


# ---- the plain forms ------------------------------------------------------------

def _order(ids, experts, align):
    """Row of every choice, by expert and then in the order of the choices; first row of
    every expert and the end; choices of every expert."""
    flat = ids.flatten().long()
    hot = flat[:, None] == torch.arange(experts, device=ids.device)
    before = hot.to(torch.int32).cumsum(0, dtype=torch.int32)
    counts = before[-1]
    padded = (counts + (align - 1)) // align * align
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = padded.cumsum(0)
    row = offsets[flat] + before.gather(1, flat[:, None])[:, 0] - 1
    return row.view(ids.shape).to(torch.int32), offsets, counts


def _gather(x, row_of, offsets, counts, out, scale=None):
    """x's rows at their choices' rows of `out`, zeros in the experts' padding."""
    experts = counts.shape[0]
    r = torch.arange(out.shape[0], device=out.device)
    e = (r[:, None] >= offsets[None, 1:]).sum(1)
    inside = (e < experts) & (r < offsets[-1])
    e = e.clamp_max(experts - 1)
    out[inside & (r >= (offsets[:-1] + counts)[e])] = 0
    for j in range(row_of.shape[1]):
        v = x.float() if scale is None else x.float() * scale[:, j:j + 1]
        out[row_of[:, j].long()] = v.to(out.dtype)
    return out


def _values(codes, scales, fmt):
    """fp32 values of MX codes [lines][blocked]."""
    if fmt == "e2m1":
        grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
        v = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], 2).flatten(1)
    else:
        v = codes.view(FP8[fmt]).float()
    e = torch.exp2(scales.float() - 127.0)
    return (v.view(v.shape[0], -1, 32) * e[:, :, None]).view(v.shape)


def _rows_product(s):
    a = _values(s["A"], s["sA"], s["fmt"])
    out = s["out_buffer"]
    for e in range(s["experts"]):
        lo, hi = s["at"][e], s["at"][e + 1]
        if hi > lo:
            b = _values(s["B"][e], s["sB_rows"][e], s["fmt"])
            out[lo:hi] = (a[lo:hi] @ b.t()).to(out.dtype)
    return out


def _wgrad_product(s):
    a = _values(s["A"], s["sA"], s["fmt"])
    b = _values(s["B"], s["sB"], s["fmt"])
    out = torch.empty(s["experts"], s["m"], s["n"], dtype=FLOATS[s["out"]], device=a.device)
    for e in range(s["experts"]):
        lo, hi = s["at"][e], s["at"][e + 1]
        out[e] = (a[:, lo:hi] @ b[:, lo:hi].t()).to(out.dtype)
    return out


def _combine(y, row_of, weights):
    total = 0.0
    for j in range(row_of.shape[1]):
        total = total + y[row_of[:, j].long()].float() * weights[:, j:j + 1]
    return total.to(y.dtype)


def _combine_backward(s):
    out = _gather(s["dout"], s["row_of"], s["offsets"], s["counts"], s["out_buffer"],
                  s["weights"])
    d = s["dout"].float()
    dw = [(s["y"][s["row_of"][:, j].long()].float() * d).sum(1) for j in range(s["topk"])]
    return {"dy": out, "dweights": torch.stack(dw, 1)}


def _moment_codes(x, positive):
    """E4M3 codes of x with one scale per block of 128; a positive value keeps at least
    the smallest code where `positive` (it is divided by)."""
    v = x.view(-1, BLOCK)
    scale = (v.abs().amax(1) / 448.0).clamp_min(2.0 ** -126)
    q = v * (1.0 / scale)[:, None]
    if positive:
        q = torch.where(v > 0, q.clamp_min(2.0 ** -9), q)
    return q.clamp(-448.0, 448.0).to(FP8["e4m3"]).view(torch.uint8).view(-1), scale


def _moment(codes, scale):
    return (codes.view(FP8["e4m3"]).float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _adamw(s):
    f = s["flat"]
    g = f["grad"].float()
    if s["bits"] == 32:
        m, v = f["m"], f["v"]
    else:
        m = _moment(f["m"], f["m_scale"])
        v = _moment(f["r"], f["r_scale"]).square()
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g * g * (1.0 - BETA2)
    r = torch.sqrt(v)
    denom = r * (1.0 / math.sqrt(1.0 - BETA2 ** s["step"])) + EPS
    p = f["param"] * (1.0 - LR * DECAY) - m / denom * (LR / (1.0 - BETA1 ** s["step"]))
    f["param"].copy_(p)
    if s["copy"]:
        f["copy"].copy_(p)
    if s["bits"] == 32:
        f["m"].copy_(m)
        f["v"].copy_(v)
    else:
        for name, x, positive in (("m", m, False), ("r", r, True)):
            codes, scale = _moment_codes(x, positive)
            f[name].copy_(codes)
            f[name + "_scale"].copy_(scale)
    return _adamw_out(s)


def _adamw_out(s):
    """The updated buffers, 8-bit codes as the values they stand for."""
    out = {k: t for k, t in s["flat"].items() if k != "grad"}
    return {k: t.view(FP8["e4m3"]) if t.dtype == torch.uint8 else t for k, t in out.items()}


def _plain(s):
    op = s["op"]
    if op == "rows":
        return _rows_product(s)
    if op == "wgrad":
        return _wgrad_product(s)
    if op == "dispatch":
        row_of, offsets, counts = _order(s["ids"], s["experts"], s["align"])
        return {"row_of": row_of, "offsets": offsets, "counts": counts,
                "x": _gather(s["x"], row_of, offsets, counts, s["out_buffer"])}
    if op == "combine":
        return _combine(s["y"], s["row_of"], s["weights"])
    if op == "combine_backward":
        return _combine_backward(s)
    return _adamw(s)


# ---- the framework's operators --------------------------------------------------

def _own(s):
    from precision_mx_quantize_gb300 import mxq
    op = s["op"]
    if op == "rows":
        return mxq.mx_gemm_experts(s["A"], s["sA"], s["B"], s["sB"], s["offsets"], s["fmt"],
                                   s["rows"], s["n"], s["k"], out_dtype=FLOATS[s["out"]],
                                   out=s["out_buffer"], b_scale_layout=s["layout"])
    if op == "wgrad":
        return mxq.mx_gemm_experts_wgrad(s["A"], s["sA"], s["B"], s["sB"], s["offsets"], s["fmt"],
                                         s["m"], s["n"], s["rows"], out_dtype=FLOATS[s["out"]])
    if op == "dispatch":
        row_of, offsets, counts = mxq.expert_order(s["ids"], s["experts"], s["align"])
        x = mxq.expert_gather(s["x"], row_of, offsets, counts, s["rows"], out=s["out_buffer"])
        return {"row_of": row_of, "offsets": offsets, "counts": counts, "x": x}
    if op == "combine":
        return mxq.expert_combine(s["y"], row_of=s["row_of"], weights=s["weights"])
    if op == "combine_backward":
        dy, dw = mxq.expert_combine_backward(s["dout"], s["y"], s["row_of"], s["offsets"],
                                             s["counts"], s["weights"], out=s["out_buffer"])
        return {"dy": dy, "dweights": dw}
    if "plan" not in s:   # a program makes it once, for as long as it trains these tensors
        s["plan"] = mxq.adamw_plan(s["params"], s["states"], weights=s["copies"],
                                   weight_decay=DECAY)
    mxq.adamw_step(s["plan"], s["grads"], s["step"], LR, betas=(BETA1, BETA2), eps=EPS)
    return _adamw_out(s)


def run(state):
    return _own(state) if own else _plain(state)


# ---- bytes and operations -------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(_numels(case))
        state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        per = 8 + (4 if case["grad"] == "f32" else 2) + state + (2 if case["copy"] else 0)
        return {"bytes": n * per, "flops": 16 * n}
    t, k, e = case["tokens"], case["topk"], case["experts"]
    n = t * k
    if op in ("rows", "wgrad"):
        code = (0.5 if case["fmt"] == "e2m1" else 1.0) + 1 / 32      # with its scale
        out = 2 if case["out"] == "bf16" else 4
        if op == "wgrad":
            return {"bytes": n * (case["m"] + case["n"]) * code + e * case["m"] * case["n"] * out,
                    "flops": 2 * n * case["m"] * case["n"]}
        used = e * (1.0 - (1.0 - k / e) ** t)                        # experts with a row
        return {"bytes": n * case["k"] * code + used * case["n"] * case["k"] * code
                + n * case["n"] * out, "flops": 2 * n * case["n"] * case["k"]}
    b, c = (2 if case["dtype"] == "bf16" else 4), case["cols"]
    if op == "dispatch":
        return {"bytes": (t + n) * c * b + 8 * n + 8 * e, "flops": n}
    if op == "combine":
        return {"bytes": (t + n) * c * b + 8 * n, "flops": 2 * n * c}
    return {"bytes": (t + 2 * n) * c * b + 12 * n, "flops": 3 * n * c}


# ---- the definitions in 64 bits -------------------------------------------------

def _table(fmt, device):
    """The value of every code."""
    if fmt == "e2m1":
        return torch.tensor([(-1.0 if c & 8 else 1.0) * E2M1[c & 7] for c in range(16)],
                            dtype=torch.float64, device=device)
    return torch.arange(256, dtype=torch.uint8, device=device).view(FP8[fmt]).to(torch.float64)


def _exact_values(codes, scales, fmt):
    table = _table(fmt, codes.device)
    if fmt == "e2m1":
        wide = codes.new_empty(codes.shape[0], 2 * codes.shape[1])
        wide[:, 0::2], wide[:, 1::2] = codes.bitwise_and(15), codes.div(16, rounding_mode="floor")
        codes = wide
    two = torch.full((), 2.0, dtype=torch.float64, device=codes.device)
    return table[codes.int()] * torch.pow(two, scales.int() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits: an 8-bit code's place holds
    the value before its rounding."""
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "adamw":
        return _exact_adamw(s)
    if op == "rows":
        out = torch.zeros(s["rows"], s["n"], dtype=f64, device="cuda")
        for e, (lo, hi) in enumerate(zip(s["at"], s["at"][1:])):
            a = _exact_values(s["A"][lo:hi], s["sA"][lo:hi], s["fmt"])
            b = _exact_values(s["B"][e], s["sB_rows"][e], s["fmt"]) if hi > lo else None
            if hi > lo:
                torch.mm(a, b.t(), out=out[lo:hi])
        return out
    if op == "wgrad":
        a = _exact_values(s["A"], s["sA"], s["fmt"])
        b = _exact_values(s["B"], s["sB"], s["fmt"])
        parts = [torch.mm(a[:, lo:hi], b[:, lo:hi].t()) for lo, hi in zip(s["at"], s["at"][1:])]
        return torch.stack(parts)
    if op == "dispatch":
        flat = s["ids"].flatten()
        by_expert = torch.sort(flat, stable=True)[1]
        at = _offsets(case, s["ids"])
        counts = torch.bincount(flat.long(), minlength=case["experts"])
        start = torch.tensor(at[:-1], device="cuda")
        first = torch.cumsum(counts, 0) - counts
        row = torch.empty_like(by_expert)
        owner = flat[by_expert].long()
        row[by_expert] = start[owner] + torch.arange(row.numel(), device="cuda") - first[owner]
        x = torch.zeros(s["rows"], s["cols"], dtype=f64, device="cuda")
        x[row] = s["x"].to(f64).repeat_interleave(case["topk"], 0)
        return {"row_of": row.view(s["ids"].shape), "offsets": torch.tensor(at), "counts": counts,
                "x": x}
    rows, w = s["row_of"].long(), s["weights"].to(f64)
    if op == "combine":
        return torch.einsum("tjc,tj->tc", s["y"].to(f64)[rows], w)
    d = s["dout"].to(f64)
    dy = torch.zeros(s["rows"], s["cols"], dtype=f64, device="cuda")
    dy[rows.flatten()] = torch.einsum("tc,tj->tjc", d, w).flatten(0, 1)
    return {"dy": dy, "dweights": torch.einsum("tjc,tc->tj", s["y"].to(f64)[rows], d)}


def _exact_adamw(s):
    f, f64 = s["flat"], torch.float64
    g = f["grad"].to(f64)
    wide = lambda name: _table("e4m3", g.device)[f[name].int()] \
        * f[name + "_scale"].to(f64).repeat_interleave(BLOCK)
    m = f["m"].to(f64) if s["bits"] == 32 else wide("m")
    v = f["v"].to(f64) if s["bits"] == 32 else torch.pow(wide("r"), 2)
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g.square(), v, BETA2)
    first = m / -math.expm1(s["step"] * math.log(BETA1))
    second = v / -math.expm1(s["step"] * math.log(BETA2))
    p = f["param"].to(f64)
    p = p - LR * DECAY * p - LR * first / (second.sqrt() + EPS)
    out = {"param": p}
    if s["copy"]:
        out["copy"] = p
    if s["bits"] == 32:
        out["m"], out["v"] = m, v
        return out
    for name, x in (("m", m), ("r", v.sqrt())):
        t = x.view(-1, BLOCK)
        scale = torch.clamp(t.abs().amax(1) / 448.0, min=2.0 ** -126)
        q = t / scale[:, None]
        if name == "r":
            q = torch.where(t > 0, torch.clamp(q, min=2.0 ** -9), q)
        out[name], out[name + "_scale"] = q.view(-1), scale
    return out
