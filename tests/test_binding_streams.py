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


@pytest.mark.parametrize("call", ["deft_tree_attn", "deft_naive_attn", "deft_prompt_attn"])
def test_steps_allocate_in_the_launch_streams_memory(monkeypatch, call):
    """Every step that allocates its own buffers does so inside
    _allocating_for(its stream)."""
    import torch

    class Allocated(Exception):
        pass

    inside = []

    @contextlib.contextmanager
    def allocating_for(stream):
        inside.append(stream)
        yield
        inside.pop()

    def alloc_buffers(*a):
        raise Allocated(list(inside))

    monkeypatch.setattr(deft, "_allocating_for", allocating_for)
    monkeypatch.setattr(deft, "alloc_buffers", alloc_buffers)
    q, pages = torch.zeros((1, 1, 64), dtype=torch.bfloat16), torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16)
    index = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(Allocated) as e:
        getattr(deft, call)(q, pages, pages, index, index, None, stream=0x77)
    assert e.value.args[0] == [0x77]
