"""The norms' C entry points refuse fp32 vectors that no float load or store can
address (CPU: every call fails its checks before any device work)."""

import pytest

from tests.test_fp8_checks import P, _grad_args, _norm_args, lib   # noqa: F401

MISPLACED = P.value + 2


@pytest.mark.parametrize("field", ["mean", "rstd"])
def test_forward(field):
    assert _norm_args(**{field: MISPLACED}) == 2


@pytest.mark.parametrize("field", ["mean", "rstd", "dweight", "dbias"])
def test_backward(field):
    assert _grad_args(**{field: MISPLACED}) == 2
    if field.startswith("d"):
        assert _grad_args(**{field: MISPLACED}, rows=0) == 2   # no rows: zeros are written
