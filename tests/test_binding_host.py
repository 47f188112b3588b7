"""The binding's way to the current stream and its checks of devices.  No GPU."""
import types

import torch

import kv_shared_b200 as hs


class Stream:
    cuda_stream = 0x7fff12345670


def test_current_stream_without_torchs_private_calls(monkeypatch):
    """A torch without the two calls below torch.cuda.current_stream(): that is asked."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    for c in (types.SimpleNamespace(), types.SimpleNamespace(_cuda_getDevice=lambda: 3),
              types.SimpleNamespace(_cuda_getCurrentRawStream=lambda d: 5)):
        assert hs._current_stream_getter(c)() == Stream.cuda_stream
    c = types.SimpleNamespace(_cuda_getDevice=lambda: 3, _cuda_getCurrentRawStream=lambda d: 100 + d)
    assert hs._current_stream_getter(c)() == 103


def test_streams_given_and_current(monkeypatch):
    monkeypatch.setattr(hs, "_current_stream", lambda: 77)
    assert hs._stream() == 77 and hs._stream(Stream) == Stream.cuda_stream
