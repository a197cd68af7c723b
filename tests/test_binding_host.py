"""What the Python binding takes for pointers and streams (no GPU)."""

import enum

import pytest

from quantized_rank_fine_amd import qlora as q


class Address(int):
    """A device address with a type of its own."""


class Place(enum.IntEnum):
    START = 4096


@pytest.mark.parametrize("p", [4096, Address(4096), Place.START])
def test_pointers_as_integers(p):
    """Any int is an address, of a subclass too."""
    assert q._ptr(p) == 4096
    assert q._ptr(None) is None
    with pytest.raises(q.QloraError) as e:               # refused by the library itself
        q.qlora_dropout(p, 64, None, 0, 4, 64, q.BF16, 1.0, 0, 0, p, 64, stream=0)
    assert e.value.status == 7


@pytest.mark.parametrize("gone", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_current_stream_without_the_short_getters(monkeypatch, gone):
    """A torch without one of the two: the public call, each time."""
    import torch
    stream = type("Stream", (), {"cuda_stream": 0})()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.delattr(torch._C, gone)
    monkeypatch.setattr(q, "_current_raw", None)
    for handle in (4660, 22136):
        stream.cuda_stream = handle
        assert q._stream(None) == handle
    assert q._stream(7) == 7 and q._stream(stream) == 22136
