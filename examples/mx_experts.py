"""Fits a linear layer of experts on MX operands to random targets, with AdamW moments in
8 bits, and then serves single tokens with it.

    python examples/mx_experts.py

Every dispatch, product, sum and optimizer step runs the CUDA operators; the router is a
fixed random projection, its top experts and their softmax.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from precision_mx_quantize_gb300 import mxq, synth                     # noqa: E402
from precision_mx_quantize_gb300.expert_layer import MxExpertLinear    # noqa: E402


def route(x, router, topk):
    """(ids [tokens, topk], weights [tokens, topk]) of the tokens' best experts."""
    top, ids = (x.float() @ router).topk(topk, dim=1)
    return ids, torch.softmax(top, 1)


def main(tokens=600, experts=6, topk=2, in_f=256, out_f=384, steps=40, lr=0.02, bits=8):
    x = synth.normal((tokens, in_f), 0).cuda()
    router = synth.normal((in_f, experts), 1, 0.1).cuda().float()
    target = synth.weight(experts * out_f, in_f, 2).cuda().view(experts, out_f, in_f) * 5.0
    master = synth.weight(experts * out_f, in_f, 3).cuda().view(experts, out_f, in_f).float()
    layer = MxExpertLinear(master.to(torch.bfloat16))
    plan = mxq.adamw_plan([master], [mxq.adamw_state(master, bits)], weights=[layer.weight])
    ids, weights = route(x, router, topk)
    rows, (row_of, offsets, counts) = layer.dispatch(x, ids)
    want = torch.zeros(tokens, out_f, device="cuda")
    for j in range(topk):
        want += weights[:, j, None] * torch.einsum("toi,ti->to", target[ids[:, j]].float(), x.float())
    losses = []
    for step in range(1, steps + 1):
        y, saved = layer.forward(rows, offsets)
        out = mxq.expert_combine(y, row_of, weights)
        diff = out.float() - want
        losses.append(diff.square().mean().item())
        dout = (diff * (2.0 / tokens)).to(torch.bfloat16)
        dy, _ = mxq.expert_combine_backward(dout, y, row_of, offsets, counts, weights)
        drows, dweight = layer.backward(dy, saved, offsets)
        mxq.adamw_step(plan, [dweight], step, lr, eps=1e-10)
        layer.requantize()
    # one token: its rows alone, without padding
    one, w1 = route(x[:1], router, topk)
    rows1, (r1, o1, _) = layer.dispatch(x[:1], one, padded=False)
    served = mxq.expert_combine(layer.infer(rows1, o1), r1, w1)
    trained = mxq.expert_combine(layer.forward(rows, offsets)[0], row_of, weights)[:1]
    gap = (served.float() - trained.float()).norm() / trained.float().norm()
    mxq.check()
    print(f"mean squared error {losses[0]:.4g} -> {losses[-1]:.4g} in {steps} steps; "
          f"one token served, {gap.item():.2%} off the training path")
    return losses, gap.item()


if __name__ == "__main__":
    main()
