"""Tensors on a GPU that is not the current one are refused before any launch (CPU:
recorders in place of the library, and a current device that the test names).  Stream
handle 0 is the default stream of the current device, so such a launch would run there
on the other device's memory."""

import pytest
import torch

from precision_mx_quantize_gb300 import mxq

U8, I32, F32, BF = torch.uint8, torch.int32, torch.float32, torch.bfloat16
HERE = torch.zeros(1).get_device()      # what host tensors answer


@pytest.fixture
def machine(monkeypatch):
    """Host tensors stand for tensors on device HERE; state["now"] is the current device."""
    state = {"now": HERE, "calls": [], "streams": []}
    for name in [n for n, _, _ in mxq.SIGNATURES if not n.endswith(("_size", "_bytes"))]:
        if hasattr(mxq, name):
            monkeypatch.setattr(mxq, name, lambda *a, _n=name: state["calls"].append(_n) or 0)
    monkeypatch.setattr(mxq, "_on_gpu", lambda t: True)
    monkeypatch.setattr(mxq, "_current_device", lambda: state["now"])
    monkeypatch.setattr(mxq, "_raw_stream", lambda i: state["streams"].append(i) or 0)
    return state


def _calls():
    x, q = torch.zeros(64, 128, dtype=BF), torch.zeros(64, 128, dtype=U8)
    s, f = torch.zeros(64, 4, dtype=U8), torch.zeros(64, 128)
    one, stat = torch.zeros(128), torch.zeros(64)
    ids, row_of = torch.zeros(64, 2, dtype=I32), torch.zeros(64, 2, dtype=I32)
    off, counts = torch.zeros(3, dtype=I32), torch.zeros(2, dtype=I32)
    plan = mxq.adamw_plan([f], [mxq.adamw_state(f)])
    ws, tc = torch.zeros(1 << 20, dtype=U8), torch.zeros(512, dtype=U8)
    return {
        "mx_quantize": lambda: mxq.mx_quantize(x),
        "mx_quantize_dual": lambda: mxq.mx_quantize_dual(x),
        "hadamard": lambda: mxq.hadamard_mx_quantize(x),
        "ablation": lambda: mxq.mx_quantize_ablation(x),
        "dequantize": lambda: mxq.mx_dequantize(q, s, 64, 128),
        "gemm": lambda: mxq.mx_gemm(q, s, q, s, "e4m3", 64, 64, 128),
        "gemm_quantize": lambda: mxq.mx_gemm_quantize(q, s, q, s, "e4m3", 64, 64, 128),
        "gemm_grouped": lambda: mxq.mx_gemm_grouped([(q, tc, q, tc, 64, 64, 128)], "e4m3"),
        "fp8_quantize": lambda: mxq.fp8_quantize(x),
        "fp8_gemm": lambda: mxq.fp8_gemm(q, torch.zeros(1, 64), q, torch.zeros(1, 1), 64, 64, 128),
        "rms_norm": lambda: mxq.rms_norm(f, one),
        "rms_norm_backward": lambda: mxq.rms_norm_backward(f, f, one, stat, workspace=ws),
        "order": lambda: mxq.expert_order(ids, 2),
        "gather": lambda: mxq.expert_gather(x, row_of, off, counts, 128),
        "combine": lambda: mxq.expert_combine(x, row_of),
        "combine_backward": lambda: mxq.expert_combine_backward(x, q.to(BF), row_of, off, counts),
        "gemm_experts": lambda: mxq.mx_gemm_experts(q, s, torch.zeros(2, 8, 128, dtype=U8),
                                                    torch.zeros(2, 8, 4, dtype=U8), off, "e4m3", 64,
                                                    8, 128),
        "wgrad": lambda: mxq.mx_gemm_experts_wgrad(q, s, q, s, off, "e4m3", 64, 64, 128),
        "adamw": lambda: mxq.adamw_step(plan, [torch.zeros(64, 128)], 1, 1e-3)}


@pytest.mark.parametrize("name", ["mx_quantize", "mx_quantize_dual", "hadamard", "ablation",
                                  "dequantize", "gemm", "gemm_quantize", "gemm_grouped",
                                  "fp8_quantize", "fp8_gemm", "rms_norm", "rms_norm_backward",
                                  "order", "gather", "combine", "combine_backward", "gemm_experts",
                                  "wgrad", "adamw"])
def test_another_device_is_refused(machine, name):
    call = _calls()[name]
    call()
    assert len(machine["calls"]) == 1 and machine["streams"] == [HERE]
    machine["now"] = HERE + 2
    with pytest.raises(ValueError, match="current device"):
        call()
    assert len(machine["calls"]) == 1 and machine["streams"] == [HERE]


def test_stream_of_a_device(machine, monkeypatch):
    machine["now"] = 1
    monkeypatch.setattr(torch.cuda, "current_device", lambda: machine["now"])
    for device in (None, 1, torch.device("cuda", 1), torch.device("cuda"), "cuda:1"):
        assert mxq._stream(device) == 0
    assert machine["streams"] == [1] * 5
    for device in (0, torch.device("cuda", 0), "cuda:2"):
        with pytest.raises(ValueError, match="current device is 1"):
            mxq._stream(device)
