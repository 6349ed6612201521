"""A call's stream argument belongs to its tensors' device, whichever device is
current (host logic alone, with stand-ins for streams and tensors)."""

import contextlib

import pytest
import torch

from mxfp8_block_scaled_quantize_amd import _tensors


class Tensor:
    is_cuda = True

    def __init__(self, index):
        self.device = torch.device("cuda", index)
        self.recorded = []

    def record_stream(self, stream):
        self.recorded.append(stream)


class Stream:
    def __init__(self, handle, device=None):
        self.handle = handle
        self.device = torch.device("cuda", 0) if device is None else device


@pytest.fixture
def current(monkeypatch):
    entered = []

    @contextlib.contextmanager
    def stream(s):
        entered.append(s)
        yield
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    return entered


def test_raw_handle_of_another_device(current):
    t = Tensor(1)
    assert _tensors.on_stream(1234, (None, t), lambda: "result") == "result"
    s, = current
    assert s.handle == 1234 and s.device == torch.device("cuda", 1) and t.recorded == [s]


def test_stream_of_another_device(current):
    called = []
    with pytest.raises(ValueError, match="cuda:0"):
        _tensors.on_stream(Stream(1), (Tensor(1),), lambda: called.append(1))
    assert not called and not current
    s = Stream(1, torch.device("cuda", 1))
    _tensors.on_stream(s, (Tensor(1), None), lambda: called.append(1))
    assert called and current == [s]
