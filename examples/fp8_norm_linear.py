"""Fits a pre-norm linear layer on block-128 FP8 operands to a random target
and then serves single tokens with it.

    python examples/fp8_norm_linear.py

Every forward, backward and token step runs the CUDA operators; torch holds
the master weights and takes the optimizer steps.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from precision_mx_quantize_gb300 import mxq, synth                     # noqa: E402
from precision_mx_quantize_gb300.fp8_layer import Fp8NormLinear        # noqa: E402


def main(tokens=1000, in_f=512, out_f=768, steps=40, lr=0.2):
    x = synth.normal((tokens, in_f), 0).cuda()
    target = synth.weight(out_f, in_f, 1).cuda() * 5.0
    master = synth.weight(out_f, in_f, 2).cuda().float()
    norm_weight = torch.ones(in_f, device="cuda")
    layer = Fp8NormLinear(master.to(torch.bfloat16), norm_weight, kind="rms")
    want = (mxq.rms_norm(x, norm_weight)[0].float() @ target.float().t())
    losses = []
    for _ in range(steps):
        y, saved = layer.forward(x)
        diff = y.float() - want
        losses.append(diff.square().mean().item())
        dx, dw, dnw, _ = layer.backward((diff * (2.0 / tokens)).to(torch.bfloat16), saved)
        master -= lr * dw
        norm_weight -= 0.01 * lr * dnw
        layer.weight.copy_(master)
        layer.requantize()
    token = x[:1].contiguous()
    served, trained = layer.infer(token), layer.forward(token)[0]
    gap = (served.float() - trained.float()).norm() / trained.float().norm()
    mxq.check()
    print(f"mean squared error {losses[0]:.4g} -> {losses[-1]:.4g} in {steps} steps; "
          f"one token served, {gap.item():.2%} off the training path")
    return losses, gap.item()


if __name__ == "__main__":
    main()
