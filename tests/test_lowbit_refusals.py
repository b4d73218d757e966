"""The Python side of the 4-bit and SwiGLU calls without a GPU: which stream a
handle names, and what is refused before anything reaches the library.  Tensors
on a GPU are stood in for; no call here launches anything."""
import contextlib

import pytest
import torch

import fp8_hybrid_granularity_gb300 as fp8hg
from fp8_hybrid_granularity_gb300 import lowbit


def test_stream_handles(monkeypatch):
    """A torch stream as it is, a raw handle wrapped, and handle 0 as the
    default stream (a wrapper around 0 would be a new stream)."""
    entered = []

    class Stream:
        pass

    @contextlib.contextmanager
    def enter(s):
        entered.append(s)
        yield

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    call = lowbit._streamed(lambda v, w=0: v + w)
    own = Stream()
    assert call(1, w=2) == 3 and entered == []
    assert call(1, w=2, stream=own) == 3 and call(2, stream=0x5000) == 2 and call(3, stream=0) == 3
    assert entered == [own, ("external", 0x5000), "default"]
