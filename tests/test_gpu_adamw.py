"""The AdamW step on the GPU against the definition in float64.

Tolerances, e = 2^-24 (half a step of fp32).  m and v: two rounded coefficients, products
and one addition, 5 e of the terms' magnitudes (v one more for g^2).  The hardware's
quotient is within two steps, 4 e.  p: one rounding of p, and the step: m's 6 e of its
terms, half of v's 7 e, one each for the root and its factor, two for the factor itself, one
for eps, the quotient's 4, and 3 for the rate, whose expm1 form is within that: 22 e of the
step that m's terms would give (U), and the product lr decay, 3 e of it.  8 bits: the state is what its codes stand for, rounded to fp32 once (e more, 2 e in
v); the new code is half a step of four bits, 2^-4 of the value, or 2^-10 of the scale
among the subnormal codes, and r's smallest code is 2^-9 of the scale; the scale is
amax / 448 within its value's error and two more roundings.  Below 2^-126 a rounding is
off by up to 2^-150, whatever the value: two of them in v leave 2^-149, and r, its root,
2^-74 (a gradient of 1e-25 has a square of 0)."""

import numpy as np
import pytest
import torch

from oracle import expert_oracle as E
from precision_mx_quantize_gb300 import mxq
from tests.libutil import ensure_built, to_np

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
BETAS = (0.9, 0.95)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def _f(t):
    return to_np(t.float()).astype(np.float64).reshape(-1)


def _params(sizes, seed, offset=0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in sizes:
        out.append((torch.randn(n + offset, generator=g) * 0.1).cuda()[offset:])
    return out


def _grads(sizes, seed, dtype=torch.float32, offset=0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n + offset, generator=g) * torch.randn(n + offset, generator=g).exp()
             * 1e-3).to(dtype).cuda()[offset:] for n in sizes]


def _values(state):
    """float64 (m, v) that a state stands for."""
    m, v = state
    if isinstance(m, torch.Tensor):
        return _f(m), _f(v)
    return (E.moment(to_np(m[0]).reshape(-1), to_np(m[1])),
            E.moment(to_np(v[0]).reshape(-1), to_np(v[1])) ** 2)


def _check_codes(pair, x, tol, least):
    codes, scales = to_np(pair[0]).reshape(-1), to_np(pair[1]).astype(np.float64)
    got = E.moment(codes, pair[1].cpu().numpy())
    n = x.size
    blocks = np.pad(np.abs(x), (0, -n % 128)).reshape(-1, 128).max(1)
    slack = np.pad(tol, (0, -n % 128)).reshape(-1, 128).max(1)
    want = np.maximum(blocks / 448.0, 2.0 ** -126)
    assert (np.abs(scales - want) <= slack / 448.0 + 2 * EPS * want).all()
    s = np.repeat(scales, 128)[:n]
    room = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) * (1 + 1e-5) + 2 * tol
    ref = np.where((x > 0) & (x < 2.0 ** -9 * s), 2.0 ** -9 * s, x) if least else x
    assert (np.abs(got - ref) <= room).all()


def _step_and_check(params, grads, states, step, copies=None, decay=0.1, lr=3e-4, eps=1e-8,
                    scale=None, plan=None, **kw):
    n = len(params)
    decays = decay if isinstance(decay, list) else [decay] * n
    before = [(_f(p), _f(g) * (1.0 if scale is None else float(scale)), *_values(s))
              for p, g, s in zip(params, grads, states)]
    plan = plan or mxq.adamw_plan(params, states, weights=copies, weight_decay=decay)
    mxq.adamw_step(plan, grads, kw.get("step_arg", step), kw.get("lr_arg", lr), betas=BETAS, eps=eps,
                   grad_scale=None if scale is None else torch.tensor([float(scale)], device="cuda"))
    mxq.check()
    b1, b2 = BETAS
    for i, ((p, g, m, v), new, state) in enumerate(zip(before, params, states)):
        bits8 = not isinstance(state[0], torch.Tensor)
        g = np.float32(g).astype(np.float64) if scale is not None else g
        wp, wm, wv, U = E.adamw(p, g, m, v, step, lr, b1, b2, eps, decays[i])
        tm = (7 if bits8 else 6) * EPS * (np.abs(b1 * m) + np.abs((1 - b1) * g)) + 1e-44
        tv = (9 if bits8 else 7) * EPS * wv + 1e-44
        tp = EPS * (np.abs(p) + np.abs(wp)) + (24 if bits8 else 22) * EPS * U \
            + 3 * EPS * lr * decays[i] * np.abs(p) + 1e-44
        assert (np.abs(_f(new) - wp) <= tp).all(), i
        if copies is not None and copies[i] is not None:
            assert torch.equal(copies[i], new.to(torch.bfloat16))
        if bits8:
            _check_codes(state[0], wm, tm, False)
            r = np.sqrt(wv)
            _check_codes(state[1], r, 7 * EPS * r + 2.0 ** -74, True)
        else:
            assert (np.abs(_f(state[0]) - wm) <= tm).all()
            assert (np.abs(_f(state[1]) - wv) <= tv).all()
    return plan


SIZES = [1, 3, 4, 127, 128, 129, 0, 1000, 8191, 8192, 8193, 20001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1, 2], ids=["aligned", "off1", "off2"])
def test_steps(bits, dtype, offset):
    params = _params(SIZES, 1, offset)
    states = [mxq.adamw_state(p, bits) for p in params]
    copies = [torch.empty(p.numel() + offset, dtype=torch.bfloat16, device="cuda")[offset:]
              if i % 3 else None for i, p in enumerate(params)]
    plan = None
    for step in (1, 2, 3, 50):
        plan = _step_and_check(params, _grads(SIZES, step, dtype, offset), states, step, copies,
                               plan=plan)


def test_codes_of_the_formula_step_by_step():
    # each operation rounded once: the same formula in numpy's fp32 gives the same codes,
    # scales and moments, bit for bit
    n, f = 5000, np.float32
    p, g = _params([n], 1), _grads([n], 2)
    other = p[0].clone()
    state, plain = mxq.adamw_state(p[0], 8), mxq.adamw_state(other, 32)
    plans = [mxq.adamw_plan(p, [state]), mxq.adamw_plan([other], [plain])]
    from oracle import mx_oracle as O
    table = O.decode_table("e4m3").astype(f)
    decode = lambda c, s: table[to_np(c)] * np.repeat(to_np(s), 128)[:n]
    b1, c1, b2, c2 = f(0.9), f(1 - 0.9), f(0.95), f(1 - 0.95)
    for step in (1, 2, 3):
        d = to_np(g[0])
        old = [decode(*state[0]), decode(*state[1]) ** 2, to_np(plain[0]), to_np(plain[1])]
        for plan in plans:
            mxq.adamw_step(plan, g, step, 1e-3, betas=BETAS)
        mxq.check()
        m, v = old[0] * b1 + d * c1, old[1] * b2 + d * d * c2
        for (codes, scales), x, least in ((state[0], m, f(0)), (state[1], np.sqrt(v), f(2.0 ** -9))):
            t = np.pad(x, (0, -n % 128)).reshape(-1, 128)
            s = np.maximum(np.abs(t).max(1) * (f(1) / f(448)), f(2.0 ** -126))
            q = t * (f(1) / s)[:, None]
            q = np.where(t > 0, np.maximum(q, least), q).reshape(-1)[:n]
            want = O.encode_element(O.round_to_element(q.astype(np.float64), "e4m3"), "e4m3")
            assert np.array_equal(to_np(scales), s) and np.array_equal(to_np(codes), want)
        assert np.array_equal(to_np(plain[0]), old[2] * b1 + d * c1)
        assert np.array_equal(to_np(plain[1]), old[3] * b2 + d * d * c2)


def test_matrices_decays_and_no_copies():
    params = [torch.randn(33, 65, device="cuda"), torch.randn(65, device="cuda")]
    grads = [torch.randn_like(p) for p in params]
    states = [mxq.adamw_state(p) for p in params]
    assert states[0][0].shape == (33, 65)
    _step_and_check(params, grads, states, 7, decay=[0.3, 0.0], lr=0.01, eps=1e-3)


def test_more_tensors_than_a_launch_takes():
    sizes = [5 + i % 7 for i in range(900)]
    params = _params(sizes, 3)
    states = [mxq.adamw_state(p) for p in params]
    _step_and_check(params, _grads(sizes, 4), states, 1)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_and_extremes(bits):
    # no gradient yet: v is 0 and p only decays; then gradients whose squares underflow,
    # and gradients of very unlike sizes in a block (r's smallest code bounds the step)
    params = _params([300], 5)
    states = [mxq.adamw_state(params[0], bits)]
    _step_and_check(params, [torch.zeros(300, device="cuda")], states, 1)
    _step_and_check(params, [torch.full((300,), 1e-25, device="cuda")], states, 2)
    g = torch.full((300,), 1e-9, device="cuda")
    g[5] = 10.0
    for step in (3, 4, 5):
        _step_and_check(params, [g], states, step)
    assert params[0].isfinite().all()


def test_device_scalars_and_a_captured_step():
    sizes = [1000, 129]
    params = _params(sizes, 6)
    states = [mxq.adamw_state(p, 8) for p in params]
    grads = _grads(sizes, 7)
    step, lr = torch.tensor([1], device="cuda"), torch.tensor([3e-4], device="cuda")
    plan = _step_and_check(params, grads, states, 1, lr=float(lr), step_arg=step, lr_arg=lr)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxq.adamw_step(plan, grads, step, lr, betas=BETAS)
    other = [p.clone() for p in params]
    ostate = [tuple((c.clone(), s.clone()) for c, s in st) for st in states]
    oplan = mxq.adamw_plan(other, ostate, weight_decay=0.1)
    for t in (2, 3, 1000):
        step.fill_(t)
        lr.fill_(1e-3 / t)
        for g, h in zip(grads, _grads(sizes, t)):
            g.copy_(h)
        graph.replay()
        mxq.adamw_step(oplan, grads, step, lr, betas=BETAS)
        mxq.check()
        for a, b in zip(params, other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
def test_grad_scale(bits):
    params = _params([700], 8)
    states = [mxq.adamw_state(params[0], bits)]
    grads = _grads([700], 9)
    plan = _step_and_check(params, grads, states, 1, scale=0.125)
    flat = [params[0]] + [t for s in states[0] for t in (s if bits == 8 else [s])]
    before = [t.clone() for t in flat]
    for bad in (float("nan"), float("inf"), -float("inf")):
        mxq.adamw_step(plan, grads, 2, 1e-3, grad_scale=torch.tensor([bad], device="cuda"))
    mxq.check()
    for a, b in zip(before, flat):
        assert torch.equal(a, b)


def test_nan_gradient_stays_in_its_block():
    params = _params([512], 10)
    states = [mxq.adamw_state(params[0], 8)]
    grads = _grads([512], 11)
    grads[0][200] = float("nan")
    plan = mxq.adamw_plan(params, states)
    mxq.adamw_step(plan, grads, 1, 1e-3)
    bad = torch.zeros(512, dtype=torch.bool, device="cuda")
    bad[200] = True
    assert torch.equal(params[0].isnan(), bad)
    for codes, scales in states[0]:
        assert scales.isnan().tolist() == [False, True, False, False]
        assert codes[128:256].eq(0).all()
    mxq.check()


def test_a_tensor_that_moved_is_looked_up_anew():
    params = [torch.ones(300, device="cuda")]
    states = [mxq.adamw_state(params[0])]
    plan = mxq.adamw_plan(params, states)
    g = [torch.ones(300, device="cuda")]
    mxq.adamw_step(plan, g, 1, 1e-2)
    old = params[0].data
    was = old.clone()
    params[0].data = torch.full((300,), 5.0, device="cuda")
    mxq.adamw_step(plan, g, 2, 1e-2)
    mxq.check()
    assert torch.equal(old, was) and params[0].lt(5.0).all() and params[0].gt(4.9).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_the_step_is_a_rounded_quotient(bits):
    # betas of 1/2 and 3/4 and a rate of 1/2 make every factor of the first step a power of
    # two, so that from p = 0 the step is m / (2 sqrt(v)) with one rounding: numpy's, bit for bit
    n, f = 6000, np.float32
    state = mxq.adamw_state(torch.zeros(n, device="cuda"), bits)
    start = mxq.adamw_plan([torch.zeros(n, device="cuda")], [state])
    for seed in (1, 2):        # moments of unlike gradients
        mxq.adamw_step(start, _grads([n], seed), seed, 1e-3)
    from oracle import mx_oracle as O
    table = O.decode_table("e4m3").astype(f)
    decode = lambda c, s: table[to_np(c)] * np.repeat(to_np(s), 128)[:n]
    m, v = (to_np(state[0]), to_np(state[1])) if bits == 32 else \
        (decode(*state[0]), decode(*state[1]) ** 2)
    p, g = torch.zeros(n, device="cuda"), _grads([n], 3)
    d = to_np(g[0])
    mxq.adamw_step(mxq.adamw_plan([p], [state]), g, 1, 0.5, betas=(0.5, 0.75), eps=0.0)
    mxq.check()
    m = m * f(0.5) + d * f(0.5)
    v = v * f(0.75) + d * d * f(0.25)
    assert np.array_equal(to_np(p), -(m / (np.sqrt(v) * f(2))))


@pytest.mark.parametrize("bits", [32, 8])
def test_moments_that_moved_are_looked_up_anew(bits):
    # replaced as a checkpoint's are, or given back and allocated anew: what a new plan does
    params, grads = _params([700, 129], 1), _grads([700, 129], 2)
    states = [mxq.adamw_state(p, bits) for p in params]
    flat = lambda st: [t for s in st for x in s for t in (x if bits == 8 else (x,))]
    plan = mxq.adamw_plan(params, states)
    mxq.adamw_step(plan, grads, 1, 1e-3)
    for step, how in ((2, "data"), (3, "storage")):
        saved = [t.clone() for t in flat(states)]
        for t, old in zip(flat(states), saved):
            if how == "data":
                t.data = old.clone()
            else:
                size = t.untyped_storage().nbytes()
                t.untyped_storage().resize_(0)
                with pytest.raises(ValueError, match="storage"):
                    plan.table()
                t.untyped_storage().resize_(size + 4096)
                t.copy_(old)
        other = [p.clone() for p in params]
        copy = [tuple(tuple(t.clone() for t in x) if bits == 8 else x.clone() for x in s) for s in states]
        mxq.adamw_step(plan, grads, step, 1e-3)
        mxq.adamw_step(mxq.adamw_plan(other, copy), grads, step, 1e-3)
        mxq.check()
        for a, b in zip(params + flat(states), other + flat(copy)):
            assert torch.equal(a, b)
