"""A linear layer of experts on MX operands: y[r] = x[r] W_e^T for the rows r of expert e.

It strings the operators together as a mixture-of-experts training step and a server
use them:

* requantize() after an optimizer step: the codes of every expert's weight along its
  rows (forward) and along its columns, stored transposed (input gradient);
* dispatch(): the rows that the router's choices get, and the tokens gathered into them;
* forward(): both layouts of the rows from one read (the rows feed the forward product,
  the columns wait for the weight gradient), the product grouped by expert;
* backward(): both layouts of dy, the input gradient against the transposed codes, and
  one weight gradient per expert in fp32;
* infer(): the rows alone, for a server's tokens, dispatched without padding.

The offsets of the experts' rows stay on the device.  Host code only: every operation is
one of mxq's calls on the current stream.
"""

from __future__ import annotations

import torch

from . import mxq


class MxExpertLinear:
    """weight [experts, out, in] bf16, out and in multiples of 32.  fmt: element format of
    the forward product and the input gradient ("e4m3", "e5m2" or "e2m1"); wgrad_fmt: of
    the weight gradient, whose operands are rotated (the fixed 32-point Hadamard) where
    it is "e2m1"."""

    def __init__(self, weight, fmt="e4m3", wgrad_fmt="e4m3"):
        if not isinstance(weight, torch.Tensor) or weight.dim() != 3:
            raise ValueError("weight must be a 3-D torch.Tensor [experts, out, in]")
        self.experts, self.out_features, self.in_features = weight.shape
        if self.out_features % 32 or self.in_features % 32:
            raise ValueError(f"out and in must be multiples of 32, got {self.out_features} and "
                             f"{self.in_features}")
        self.weight, self.fmt, self.wgrad_fmt = weight, fmt, wgrad_fmt
        # rows of an expert start where a block of the weight gradient may
        self.align = 64 if wgrad_fmt == "e2m1" else 32
        # the weights' scales straight in the tensor cores' layout where there is one
        stage = 256 if fmt == "e2m1" else 128
        self.layout = "tc" if self.in_features % stage == 0 and self.out_features % stage == 0 \
            else "rowmajor"
        self.operands = None
        self.requantize()

    def requantize(self):
        """The MX operands of the present weights (call it after every update)."""
        if self.operands is None:
            e, n, k = self.weight.shape
            dev, half = self.weight.device, 2 if self.fmt == "e2m1" else 1
            byte = lambda *s: torch.empty(s, dtype=torch.uint8, device=dev)
            scales = lambda lines, blocked: byte(
                e, mxq.mxq_scales_tc_bytes(lines, blocked) if self.layout == "tc"
                else lines * (blocked // 32))
            self.operands = (byte(e, n, k // half), scales(n, k), byte(e, k, n // half),
                             scales(k, n))
        for i in range(self.experts):
            mxq.mx_quantize_dual(self.weight[i], self.fmt, False, self.fmt, False,
                                 out=tuple(t[i] for t in self.operands), scale_layout=self.layout)

    def dispatch(self, x, ids, padded=True):
        """x [tokens, in] bf16, ids [tokens, topk] -> (rows [capacity, in], routing): what
        forward() and backward() take, and the places to gather from and combine into.
        padded False: the choices' rows alone, for infer() (backward() needs the padding;
        a token of eight experts has 8 rows then, and 256 with it)."""
        align = self.align if padded else 1
        routing = mxq.expert_order(ids, self.experts, align)
        rows = mxq.expert_rows(ids.numel(), self.experts, align)
        return mxq.expert_gather(x, *routing, rows), routing

    def forward(self, rows, offsets):
        """rows [capacity, in] bf16 -> (y [capacity, out] bf16, what backward() needs).  Rows
        that no expert holds are not written."""
        c = rows.shape[0]
        r, rs, k, ks = mxq.mx_quantize_dual(rows, self.fmt, False, self.wgrad_fmt,
                                            self.wgrad_fmt == "e2m1")
        w, ws = self.operands[:2]
        y = mxq.mx_gemm_experts(r, rs, w, ws, offsets, self.fmt, c, self.out_features,
                                self.in_features, out_dtype=torch.bfloat16,
                                b_scale_layout=self.layout)
        return y, (k, ks)

    def backward(self, dy, saved, offsets):
        """dy [capacity, out] bf16 -> (drows [capacity, in] bf16, dweight [experts, out, in]
        fp32)."""
        c, n, k = dy.shape[0], self.out_features, self.in_features
        r, rs, d, ds = mxq.mx_quantize_dual(dy, self.fmt, False, self.wgrad_fmt,
                                            self.wgrad_fmt == "e2m1")
        wt, wts = self.operands[2:]
        drows = mxq.mx_gemm_experts(r, rs, wt, wts, offsets, self.fmt, c, k, n,
                                    out_dtype=torch.bfloat16, b_scale_layout=self.layout)
        dweight = mxq.mx_gemm_experts_wgrad(d, ds, *saved, offsets, self.wgrad_fmt, n, k, c)
        return drows, dweight

    def infer(self, rows, offsets):
        """y of forward() for a server's tokens: nothing is kept, any number of rows."""
        r, rs = mxq.mx_quantize(rows, "row", self.fmt)
        w, ws = self.operands[:2]
        return mxq.mx_gemm_experts(r, rs, w, ws, offsets, self.fmt, rows.shape[0],
                                   self.out_features, self.in_features, out_dtype=torch.bfloat16,
                                   b_scale_layout=self.layout)
