"""The sequence operators' launches go to their tensors' device (host: the device calls are stood in for)."""
from __future__ import annotations

import pytest

from grouped_convolution_amd import binding as B

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("current", [0, 1])
def test_tensors_of_another_device_than_the_current_one(monkeypatch, current):
    state = {"device": current, "calls": []}

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, state["device"] = state["device"], self.index

        def __exit__(self, *_):
            state["device"] = self.before

    class Library:
        @staticmethod
        def gconv_orthogonalize(*args):
            state["calls"].append((state["device"], args))
            return 0

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["device"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    monkeypatch.setattr(B, "load", lambda: Library)
    B._launch("gconv_orthogonalize", torch.device("cuda", 1), "d", 2)
    assert state["calls"] == [(1, ("d", 2, 101))] and state["device"] == current
