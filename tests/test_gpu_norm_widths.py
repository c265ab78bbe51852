"""Norms of many widths, called from two threads.

The rings' shared memory depends on the width, so a process that meets many
widths asks for many sizes of one kernel.  However many came before, a call must
not take back the size that another thread has just asked for."""

import threading

import pytest
import torch

from precision_mx_quantize_gb300 import mxq
from tests.libutil import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()


def test_two_threads_after_many_widths():
    rows = 4864   # enough for a ring at every width
    long = torch.randn(rows * 6400, device="cuda").to(torch.bfloat16)
    w = torch.ones(16384, device="cuda")
    for cols in range(520, 6400, 8):
        mxq.rms_norm(long[:rows * cols].view(rows, cols), w[:cols])
    mxq.check()
    del long
    failures = []

    def work(cols):
        # the C entry point in a tight loop: most of the time is spent inside it,
        # where the other thread runs too
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            x = torch.randn(400, cols, device="cuda").to(torch.bfloat16)
            want, rstd = mxq.rms_norm(x, w[:cols])
            y = torch.empty_like(x)
            a = mxq._NORM_ARGS.pack(x.data_ptr(), w.data_ptr(), 0, y.data_ptr(), 0, rstd.data_ptr(),
                                    0, 0, 400, cols, 1e-5, mxq.NORM_RMS, mxq.OUT_BF16, mxq.OUT_F32, 0)
            call, s = mxq.lib().mxq_norm_forward, stream.cuda_stream
            failures.extend((cols, st) for st in {call(a, s) for _ in range(20000)} if st)
            stream.synchronize()
            if not torch.equal(y, want):
                failures.append((cols, "other values"))

    threads = [threading.Thread(target=work, args=(c,)) for c in (9224, 12000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    mxq.check()
    assert not failures, failures
