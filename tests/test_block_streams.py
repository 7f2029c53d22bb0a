"""The stream a block operator is called on, without a GPU: a pointer is a stream of the
tensors' device, a torch stream of another device is refused."""
from __future__ import annotations

import contextlib
from types import SimpleNamespace

import pytest
import torch

from quantized_swiglu_mlp_gb300 import ops


class FakeStream:
    def __init__(self, pointer=0, device=None):
        self.pointer, self.device = pointer, device


@pytest.fixture
def current(monkeypatch):
    """(device, pointer) of the stream made current, by device, as torch keeps them."""
    now = {}

    @contextlib.contextmanager
    def use(stream):
        saved = dict(now)
        now[stream.device] = stream.pointer
        yield
        now.clear()
        now.update(saved)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    # as torch's: without a device, one of the current device
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda pointer, device=None: FakeStream(pointer, device or torch.device("cuda", 0)))
    monkeypatch.setattr(torch.cuda, "stream", use)
    return now


@pytest.mark.parametrize("index", [0, 1])
def test_a_pointer_is_a_stream_of_the_tensors_device(current, index):
    x = SimpleNamespace(is_cuda=True, device=torch.device("cuda", index))
    assert ops._call(lambda t, k: (k, current.get(t.device)), 4711, x, 5) == (5, 4711)
    assert not current


def test_a_stream_of_another_device_is_refused(current):
    x = SimpleNamespace(is_cuda=True, device=torch.device("cuda", 1))
    there, elsewhere = FakeStream(7, torch.device("cuda", 1)), FakeStream(9, torch.device("cuda", 0))
    assert ops._call(lambda t: current.get(t.device), there, x) == 7
    with pytest.raises(ValueError, match="stream"):
        ops._call(lambda t: current.get(t.device), elsewhere, x)


def test_without_a_stream_or_a_cuda_tensor(current):
    x = SimpleNamespace(is_cuda=True, device=torch.device("cuda", 1))
    assert ops._call(lambda t: dict(current), None, x) == {}
    assert ops._call(lambda t: "refused by the binding", 4711, torch.zeros(2)) == "refused by the binding"
    assert ops._call(lambda t: "refused by the binding", 4711, None) == "refused by the binding"
