"""The library works on the current device: the ctypes binding makes that the tensors' device for the call, on
that device's current stream, and refuses a stream of another.  With a stand-in for CUDA, so on the CPU."""

import contextlib

import pytest
import torch

import lm_head_linear_gb300 as flce
from lm_head_linear_gb300 import binding


class Stream:
    def __init__(self, index, handle):
        self.device, self.cuda_stream = torch.device("cuda", index), handle


class Buffer:
    """A workspace on cuda:1."""
    device = torch.device("cuda", 1)

    def data_ptr(self):
        return 4096


@pytest.fixture
def cuda(monkeypatch):
    """Two devices, cuda:0 current, and a library that records (current device, stream handle)."""
    state = {"device": 0, "calls": []}

    @contextlib.contextmanager
    def device(d):
        was, state["device"] = state["device"], d.index
        try:
            yield
        finally:
            state["device"] = was

    class Library:
        status = 0

        def flce_read_device_status(self, ws, stream, out):
            state["calls"].append((state["device"], stream.value))
            return self.status

        def flce_last_error(self):
            return b"text"

    state["library"] = Library()
    monkeypatch.setattr(binding, "_LIB", state["library"])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["device"])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(d.index, 100 + d.index) if d else Stream(0, 100))
    monkeypatch.setattr(torch.cuda, "device", device)
    return state


def test_a_call_runs_on_its_tensors_device_and_stream(cuda):
    flce.flce_read_device_status(Buffer())
    assert cuda["calls"] == [(1, 101)] and cuda["device"] == 0
    flce.flce_read_device_status(Buffer(), Stream(1, 7))
    assert cuda["calls"][-1] == (1, 7) and cuda["device"] == 0
    cuda["library"].status = 5
    with pytest.raises(flce.FlceError):
        flce.flce_read_device_status(Buffer())
    assert cuda["device"] == 0


def test_a_stream_of_another_device_is_refused(cuda):
    with pytest.raises(ValueError, match="cuda:0"):
        flce.flce_read_device_status(Buffer(), Stream(0, 7))
    assert cuda["calls"] == []
