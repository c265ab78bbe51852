"""A pre-norm linear layer on block-128 FP8 operands: y = norm(x) W^T.

It strings the operators together as a training step and a server use them:

* requantize() after an optimizer step: W in 128x128 tiles, W and W^T codes
  from one read;
* forward(): norm, both layouts of its output from one read (the rows feed the
  forward product, the columns wait for the weight gradient), product;
* backward(): both layouts of dy, the input gradient against W^T's codes, the
  weight gradient in fp32, the norm's backward pass (an fp32 residual stream gets
  its gradient from an fp32 input-gradient product);
* infer(): the norm writes the product's operand directly.

Host code only: every operation is one of mxq's calls on the current stream, but
for the rounding of an fp32 norm output to the quantizer's bf16.
"""

from __future__ import annotations

import torch

from . import mxq


class Fp8NormLinear:
    """weight [out, in] bf16; norm_weight [in] (and norm_bias, kind "layer")
    bf16 or fp32; grad_fmt: element format of dy ("e4m3", or "e5m2" for a
    wider range at two mantissa bits)."""

    def __init__(self, weight, norm_weight, norm_bias=None, kind="rms", eps=1e-5, grad_fmt="e4m3"):
        if kind not in ("rms", "layer"):
            raise ValueError(f'kind must be "rms" or "layer", got {kind!r}')
        if kind == "rms" and norm_bias is not None:
            raise ValueError("an RMS norm has no bias")
        self.weight, self.norm_weight, self.norm_bias = weight, norm_weight, norm_bias
        self.kind, self.eps, self.grad_fmt = kind, eps, grad_fmt
        self.out_features, self.in_features = weight.shape
        self.operands = None
        self.requantize()

    def requantize(self):
        """The FP8 operands of the present weight (call it after every update)."""
        self.operands = mxq.fp8_quantize_tiles(self.weight, out=self.operands)

    def forward(self, x):
        """x [tokens, in] bf16 or fp32 -> (y [tokens, out] bf16, what backward() needs)."""
        if self.kind == "layer":
            h, mean, rstd = mxq.layer_norm(x, self.norm_weight, self.norm_bias, self.eps)
        else:
            h, rstd = mxq.rms_norm(x, self.norm_weight, self.eps)
            mean = None
        hr, hrs, hc, hcs = mxq.fp8_quantize_dual(h.to(torch.bfloat16))
        w, ws = self.operands[:2]
        y = mxq.fp8_gemm(hr, hrs, w, ws, x.shape[0], self.out_features, self.in_features)
        return y, (x, mean, rstd, hc, hcs)

    def backward(self, dy, saved):
        """dy [tokens, out] bf16 -> (dx, dweight, dnorm_weight, dnorm_bias): dx in
        x's dtype, the others fp32, dnorm_bias None for an RMS norm."""
        x, mean, rstd, hc, hcs = saved
        T, N, K, g = x.shape[0], self.out_features, self.in_features, self.grad_fmt
        dr, drs, dc, dcs = mxq.fp8_quantize_dual(dy, g, g)
        wt, wts = self.operands[2:]
        dh = mxq.fp8_gemm(dr, drs, wt, wts, T, K, N, fmt_a=g, out_dtype=x.dtype)
        dweight = mxq.fp8_gemm(dc, dcs, hc, hcs, N, K, T, fmt_a=g, b_scales="line",
                               out_dtype=torch.float32)
        if self.kind == "layer":
            dx, dnw, dnb = mxq.layer_norm_backward(dh, x, self.norm_weight, mean, rstd)
        else:
            dx, dnw = mxq.rms_norm_backward(dh, x, self.norm_weight, rstd)
            dnb = None
        return dx, dweight, dnw, dnb

    def infer(self, x):
        """y of forward() for a server's tokens: nothing is kept, and the norm's
        output is quantized from fp32 without a bf16 rounding."""
        if self.kind == "layer":
            h, hs, _, _ = mxq.layer_norm_quantize(x, self.norm_weight, self.norm_bias, self.eps)
        else:
            h, hs, _ = mxq.rms_norm_quantize(x, self.norm_weight, self.eps)
        w, ws = self.operands[:2]
        return mxq.fp8_gemm(h, hs, w, ws, x.shape[0], self.out_features, self.in_features)
