"""Layers of experts and the AdamW step against the bounds-checked build of the
library: no kernel computes an index outside the extent its arguments imply
(tests/bounds_checked_experts.py, in a subprocess)."""

import json
import os
import subprocess
import sys

import pytest
import torch

from precision_mx_quantize_gb300 import build as _build
from tests.libutil import ensure_built

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_bounds_error():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ensure_built()
    assert os.path.exists(_build.LIB_DEBUG), "the bounds-checked library was not built"
    env = dict(os.environ, MXQ_BOUNDS_CHECKED="1")
    p = subprocess.run([sys.executable, "-m", "tests.bounds_checked_experts"], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=900)
    assert p.returncode == 0, p.stdout[-3000:] + p.stderr[-3000:]
    res = json.loads(p.stdout.strip().splitlines()[-1])
    assert res["errors"] == [] and res["cases"] == 36, res
