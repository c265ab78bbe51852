"""The norm backward's workspace belongs to the device it is made for (CPU: fakes
of the library's size query and of the current device)."""

import contextlib

import pytest
import torch

from precision_mx_quantize_gb300 import mxq


@pytest.fixture
def devices(monkeypatch):
    """Two devices, of 100 and of 152 SMs; the library asks the current one."""
    state = {"now": 0, "asked": []}

    @contextlib.contextmanager
    def use(index):
        before, state["now"] = state["now"], index
        yield
        state["now"] = before

    def size(rows, cols):
        state["asked"].append((state["now"], rows, cols))
        return (100, 152)[state["now"]] * cols * 8

    monkeypatch.setattr(torch.cuda, "device", use)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["now"])
    monkeypatch.setattr(mxq, "mxq_norm_backward_workspace_size", size)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: (n, str(device)))
    mxq._norm_backward_workspace.cache_clear()
    yield state
    mxq._norm_backward_workspace.cache_clear()


def test_each_device_has_its_own_size(devices):
    ws = lambda d: mxq.norm_backward_workspace(4096, 64, d)
    assert ws("cuda:0") == (100 * 64 * 8, "cuda:0")
    assert ws("cuda:1") == (152 * 64 * 8, "cuda:1")     # a cached size of device 0 is too small
    assert ws(torch.device("cuda", 0)) == (100 * 64 * 8, "cuda:0")
    assert ws("cuda") == (100 * 64 * 8, "cuda")
    devices["now"] = 1
    assert ws("cuda") == (152 * 64 * 8, "cuda")
    assert devices["now"] == 1 and len(devices["asked"]) == 2   # once per device


def test_small_sizes_have_a_workspace(devices):
    assert mxq.norm_backward_workspace(0, 0, "cuda:0")[0] == 256
