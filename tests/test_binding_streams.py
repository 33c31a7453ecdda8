"""Which stream's memory the binding allocates from, on the CPU: torch's
stream calls are replaced by recorders."""
from __future__ import annotations

import contextlib
from types import SimpleNamespace

import pytest

import shared_prefix_kv_deft_gb300 as deft


class Streams:
    """torch.cuda's stream calls; like torch's own, ExternalStream takes a
    handle of 0 for no handle and gives out one of its pool's streams."""

    def __init__(self):
        self.entered = []

    def ExternalStream(self, handle):
        return SimpleNamespace(cuda_stream=handle or 0x900)

    def default_stream(self):
        return SimpleNamespace(cuda_stream=0)

    @contextlib.contextmanager
    def stream(self, s):
        self.entered.append(s.cuda_stream)
        yield


@pytest.mark.parametrize("handle", [0, 0x77])
@pytest.mark.parametrize("raw", [False, True])
def test_memory_is_the_launch_streams(monkeypatch, handle, raw):
    cuda = Streams()
    monkeypatch.setattr(deft, "_torch", SimpleNamespace(cuda=cuda))
    stream = handle if raw else SimpleNamespace(cuda_stream=handle)
    with deft._allocating_for(stream):
        pass
    assert cuda.entered == [handle] == [deft._stream(stream)]


def test_current_stream_is_left_alone(monkeypatch):
    cuda = Streams()
    monkeypatch.setattr(deft, "_torch", SimpleNamespace(cuda=cuda))
    with deft._allocating_for(None):
        pass
    assert cuda.entered == []
