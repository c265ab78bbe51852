"""Norms of rows without elements: their statistics are 0 / 0, not whatever lay in
the memory (CPU; recorders in place of the library)."""

import pytest
import torch

from precision_mx_quantize_gb300 import mxq
from tests.test_fp8_checks import fake, lib   # noqa: F401  (fixtures)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_statistics_of_no_columns_are_nan(fake, monkeypatch, dtype):
    x, v = torch.zeros(3, 0, dtype=dtype), torch.zeros(0)
    sevens = lambda f: lambda *a, **kw: f(*a, **kw).fill_(7)
    monkeypatch.setattr(torch, "empty", sevens(torch.empty))
    monkeypatch.setattr(torch, "empty_like", sevens(torch.empty_like))
    y, mean, rstd = mxq.layer_norm(x, v, v)
    assert y.shape == (3, 0) and mean.shape == rstd.shape == (3,)
    codes, scales, qmean, qrstd = mxq.layer_norm_quantize(x, v)
    assert codes.numel() == scales.numel() == 0
    for stat in (mean, rstd, qmean, qrstd, mxq.rms_norm(x, v)[1], mxq.rms_norm_quantize(x, v)[2]):
        assert stat.isnan().all()
