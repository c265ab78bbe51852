"""The block-128 FP8 operators and the norms against the bounds-checked build.

Run as ``MXQ_BOUNDS_CHECKED=1 python -m tests.bounds_checked_fp8`` (the GPU test
beside it does so in a subprocess): no case may record an index out of range.
Prints one JSON line with the number of cases and the errors found."""

import json

import torch

from precision_mx_quantize_gb300 import mxq, synth
from precision_mx_quantize_gb300.fp8_layer import Fp8NormLinear
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

    for r, c in ((1, 1), (1, 4096), (3, 130), (127, 129), (128, 128), (300, 1001), (257, 136)):
        x = synth.normal((r, c), r).cuda()
        for fmt in ("e4m3", "e5m2"):
            a = mxq.fp8_quantize(x, "row", fmt)
            mxq.fp8_quantize(x, "col", fmt)
            mxq.fp8_quantize_dual(x, fmt, fmt)
            w = mxq.fp8_quantize_tiles(x, fmt)
            checked(f"quantize {r}x{c} {fmt}")
            for dt in (torch.bfloat16, torch.float32):
                mxq.fp8_gemm(*a, *w[:2], r, r, c, fmt, fmt, out_dtype=dt)
                mxq.fp8_gemm(*a, *a, r, r, c, fmt, fmt, "line", out_dtype=dt)
                checked(f"gemm {r}x{r}x{c} {fmt} {dt}")
    for m, nn, k in ((1500, 1296, 200), (2000, 1001, 130), (1792, 1028, 300), (5, 700, 4096)):
        a = mxq.fp8_quantize(synth.normal((m, k), 1).cuda())
        w = synth.weight(nn, k, 2).cuda()
        for kind, b in (("tile", mxq.fp8_quantize_tiles(w)[:2]), ("line", mxq.fp8_quantize(w))):
            for dt in (torch.bfloat16, torch.float32):
                mxq.fp8_gemm(*a, *b, m, nn, k, b_scales=kind, out_dtype=dt)
                checked(f"gemm {m}x{nn}x{k} {kind} {dt}")
    for r, c in ((1, 1), (5, 129), (7, 1000), (4, 1001), (9, 4096), (3, 8200), (2, 16384), (2, 20001)):
        for dt in (torch.bfloat16, torch.float32):
            x, v = synth.normal((r, c), r).cuda().to(dt), torch.ones(c, device="cuda")
            y, mean, rstd = mxq.layer_norm(x, v, v)
            mxq.layer_norm_quantize(x, v, v)
            mxq.rms_norm_quantize(x, v)
            mxq.layer_norm_backward(y, x, v, mean, rstd)
            mxq.rms_norm_backward(y, x, v, rstd)
            checked(f"norm {r}x{c} {dt}")
    layer = Fp8NormLinear(synth.weight(640, 512, 3).cuda(), torch.ones(512, device="cuda"))
    x = synth.normal((333, 512), 1).cuda()
    layer.backward(synth.out_grad(333, 640, 2).cuda(), layer.forward(x)[1])
    layer.infer(x[:1].contiguous())
    checked("layer")
    print(json.dumps({"cases": n, "errors": errors}))


if __name__ == "__main__":
    main()
