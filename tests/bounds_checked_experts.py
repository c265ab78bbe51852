"""Layers of experts and the AdamW step against the bounds-checked build.

Run as ``MXQ_BOUNDS_CHECKED=1 python -m tests.bounds_checked_experts`` (the GPU test
beside it does so in a subprocess): no case may record an index out of range.
Prints one JSON line with the number of cases and the errors found."""

import json

import torch

from precision_mx_quantize_gb300 import mxq, synth
from precision_mx_quantize_gb300.expert_layer import MxExpertLinear
from tests.libutil import ensure_built


def main():
    assert mxq.BOUNDS_CHECKED and mxq.LIB_PATH.endswith("libmxq_debug.so"), mxq.LIB_PATH
    ensure_built()
    errors, n = [], 0

    def checked(tag):
        nonlocal n
        n += 1
        st = mxq.mxq_check(mxq._stream())
        if st != 0:
            errors.append((tag, mxq.STATUS.get(st, st)))

    for tokens, topk, experts, cols, align in ((1, 1, 1, 1, 1), (7, 3, 5, 33, 32), (300, 9, 64, 264, 1),
                                               (5000, 2, 1000, 64, 64)):
        g = torch.Generator().manual_seed(tokens)
        ids = torch.randint(-1, experts, (tokens, topk), generator=g).cuda()
        r = mxq.expert_order(ids, experts, align)
        rows = mxq.expert_rows(ids.numel(), experts, align)
        w = torch.rand(tokens, topk, device="cuda")
        for dt in (torch.bfloat16, torch.float32):
            x = synth.normal((tokens, cols), 1).cuda().to(dt)
            y = mxq.expert_gather(x, *r, rows, weights=w)
            mxq.expert_combine(y, r[0], w)
            mxq.expert_combine_backward(x, y, *r, w)
            checked(f"rows {tokens}x{topk} of {experts} x {cols} {dt}")
    for fmt in ("e4m3", "e5m2", "e2m1"):
        for wgrad in ("e4m3", "e2m1"):
            for tokens, experts, topk, out_f, in_f in ((1, 8, 2, 64, 96), (40, 3, 2, 288, 512),
                                                       (700, 2, 1, 128, 2208), (300, 2, 2, 96, 4512)):
                layer = MxExpertLinear(synth.weight(experts * out_f, in_f, 3).cuda()
                                       .view(experts, out_f, in_f), fmt, wgrad)
                ids = torch.randint(0, experts, (tokens, topk),
                                    generator=torch.Generator().manual_seed(1)).cuda()
                rows, (row_of, offsets, counts) = layer.dispatch(
                    synth.normal((tokens, in_f), 1).cuda(), ids)
                y, saved = layer.forward(rows, offsets)
                layer.backward(y, saved, offsets)
                layer.infer(rows, offsets)
                checked(f"layer {fmt} {wgrad} {tokens} of {experts} {out_f}x{in_f}")
    for bits in (8, 32):
        for dt in (torch.bfloat16, torch.float32):
            params = [torch.randn(m, device="cuda") for m in (1, 127, 8193, 30000)]
            plan = mxq.adamw_plan(params, [mxq.adamw_state(p, bits) for p in params])
            mxq.adamw_step(plan, [p.clone().to(dt) for p in params], 1, 1e-3)
            checked(f"adamw {bits} {dt}")
    print(json.dumps({"cases": n, "errors": errors}))


if __name__ == "__main__":
    main()
