"""The binding's way to the current stream and its checks of devices.  No GPU."""
import types

import pytest
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
    assert hs._current_stream_getter(c)() == 103 and hs._current_stream_getter(c)(2) == 102


def test_streams_given_and_current(monkeypatch):
    monkeypatch.setattr(hs, "_current_stream", lambda d=None: 77)
    assert hs._stream() == 77 and hs._stream(Stream) == Stream.cuda_stream


class Tensor:
    """An address on a device (-1: the host's memory)."""
    def __init__(self, device):
        self.device = device

    def data_ptr(self):
        return 0x1000

    def get_device(self):
        return self.device

    def numel(self):
        return 1 << 40

    def element_size(self):
        return 1


CALLS = {  # arguments before the stream, with the tensor that is looked at in its place
    "hs2_qk_norm_rope": lambda t: (hs.make_rope_desc(1, 1, 1, 64), *[None] * 6, t, *[None] * 7),
    "hs2_window_attn": lambda t: (hs.make_desc(1, 1, 1, 64, max_ctx=8), 0, *[None] * 5, t, *[None] * 3, Tensor(1)),
    "hs2_weight_accum": lambda t: (hs.make_desc(1, 1, 1, 64, max_ctx=8), *[None] * 4, t, None, 1.0, None, None, Tensor(1)),
    "hs2_kv_evict": lambda t: (hs.make_evict_desc(1, 64, kv_capacity=8), t, *[None] * 12),
}


@pytest.mark.parametrize("name", CALLS)
def test_calls_refuse_tensors_of_another_device(name, monkeypatch):
    """On device 1: tensors of device 0 and of the host, and a stream of device 0, are refused before the
    library is called; what passes is refused there for its missing arguments (status 1 without a reason)."""
    monkeypatch.setattr(hs, "_device", lambda: 1)
    monkeypatch.setattr(hs, "_current_stream", lambda d=None: 77)
    on1, on0 = (types.SimpleNamespace(cuda_stream=5, device_index=i) for i in (1, 0))
    for device, stream, refused in ((0, None, True), (-1, None, True), (1, None, False), (0, on1, True), (1, on0, True),
                                    (1, on1, False), (-1, on1, False), (1, Stream, False), (0, Stream, True)):
        with pytest.raises(hs.HS2Error) as e:
            getattr(hs, name)(*CALLS[name](Tensor(device)), stream=stream)
        assert e.value.status == hs.HS2_ERR_INVALID_ARG
        assert ("current device" in str(e.value)) == refused, (device, stream)
    with pytest.raises(hs.HS2Error):                              # a missing tensor is the library's to refuse
        getattr(hs, name)(*CALLS[name](None), stream=on1)


@pytest.mark.parametrize("name", CALLS)
def test_calls_take_what_has_only_an_address(name, monkeypatch):
    """An object that cannot tell its device passes, with a stream and without."""
    class Address:
        def data_ptr(self):
            return 0x1000

    monkeypatch.setattr(hs, "_device", lambda: 1)
    monkeypatch.setattr(hs, "_current_stream", lambda d=None: 77)
    for stream in (None, Stream):
        with pytest.raises(hs.HS2Error) as e:                      # the library's refusal of the rest
            getattr(hs, name)(*CALLS[name](Address()), stream=stream)
        assert e.value.status == hs.HS2_ERR_INVALID_ARG and "current device" not in str(e.value)
