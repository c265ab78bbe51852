"""Every kernel of the block-128 FP8 product, by name, and the norms of rows that
one CTA cannot hold, against the bounds-checked build.

Run as ``MXQ_BOUNDS_CHECKED=1 python -m tests.bounds_checked_fp8_forms`` (the GPU
test beside it does so in a subprocess).  Prints one JSON line with the number of
cases and the errors found."""

import json

import torch

from precision_mx_quantize_gb300 import mxq, synth
from tests.libutil import ensure_built


def main():
    assert mxq.BOUNDS_CHECKED and mxq.LIB_PATH.endswith("libmxq_debug.so"), mxq.LIB_PATH
    ensure_built()
    from tests.test_gpu_fp8_forms import call
    errors, n = [], 0

    def checked(tag):
        nonlocal n
        n += 1
        st = mxq.mxq_check(mxq._stream())
        if st != 0:
            errors.append((tag, mxq.STATUS.get(st, st)))

    for m, nn, k in ((512, 1025, 520), (257, 593, 1100), (130, 383, 512), (385, 516, 520),
                     (256, 520, 1111), (129, 770, 1000), (2300, 2305, 520)):
        a = mxq.fp8_quantize(synth.normal((m, k), 1).cuda())
        w = synth.weight(nn, k, 2).cuda()
        for kind, b in (("tile", mxq.fp8_quantize_tiles(w)[:2]), ("line", mxq.fp8_quantize(w))):
            for dt in (torch.bfloat16, torch.float32):
                c = torch.empty(m, nn, dtype=dt, device="cuda")
                for pairs in range(5):
                    st = call([*a, *b], m, nn, k, "e4m3", "e4m3", kind, c, pairs)
                    assert st == 0, st
                    checked(f"product {m}x{nn}x{k} {kind} {dt} pairs {pairs}")
    # the rings, aligned and not; rows past every register plan
    for r, c in ((1000, 4097), (2000, 2048), (700, 8190), (5, 16385), (3, 16392), (40, 20001),
                 (17, 9000), (1300, 1003)):
        for dt in (torch.bfloat16, torch.float32):
            x, v = synth.normal((r, c), r).cuda().to(dt), torch.ones(c, device="cuda")
            y, mean, rstd = mxq.layer_norm(x, v, v)
            mxq.layer_norm_quantize(x, v, v)
            y2, rs = mxq.rms_norm(x, v)
            mxq.rms_norm_quantize(x, v)
            mxq.layer_norm_backward(y, x, v, mean, rstd)
            mxq.rms_norm_backward(y2, x, v, rs)
            checked(f"norm {r}x{c} {dt}")
    print(json.dumps({"cases": n, "errors": errors}))


if __name__ == "__main__":
    main()
