"""The binding's fast calls (csrc/calls.c) against functions that note what arrives: every argument in
its place, None as NULL, what is refused before the library is called.  No GPU."""
import ctypes
import os

import pytest
import torch

import kv_shared_b200 as hs

P, I32, F32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {"rope": [P] * 16, "window": [P, I32] + [P] * 10 + [SZ, P], "accum": [P] * 7 + [F32] + [P] * 3 + [SZ, P],
              "evict": [P] * 15}


class Tensor:
    """What the calls need of a tensor, at an address of our own."""
    def __init__(self, at, n=0):
        self.at, self.n = at, n

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n

    def element_size(self):
        return 1


class Stream:
    cuda_stream = 0x7fff12345670


@pytest.fixture
def seen():
    if not os.path.exists(hs.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    m, notes = hs._fast(), []
    fakes = [ctypes.CFUNCTYPE(ctypes.c_int, *SIGNATURES[n])(lambda *a, n=n: notes.append((n, a)) or 0)
             for n in ("rope", "window", "accum", "evict")]
    m.bind(*(ctypes.cast(f, P).value for f in fakes))
    yield notes
    L = hs.lib()
    m.bind(*(ctypes.cast(f, P).value for f in (L.hs2_qk_norm_rope, L.hs2_window_attn, L.hs2_weight_accum, L.hs2_kv_evict)))


def _tensors(n, holes):
    at = [0xffff800000000000 + 4096 * i if i % 2 else 0x7000 + 16 * i for i in range(n)]
    return [None if i in holes else Tensor(x) for i, x in enumerate(at)], tuple(None if i in holes else x for i, x in enumerate(at))


def _called(seen, name, desc):
    (got, a), = seen
    assert got == name and a[0] == ctypes.addressof(desc)
    seen.clear()
    return a[1:]


@pytest.mark.parametrize("holes", [(), (0,), (3, 7, 8), tuple(range(14))])
def test_rope_arguments(seen, holes):
    d = hs.make_rope_desc(2, 3, 16, 128)
    t, at = _tensors(14, holes)
    hs.hs2_qk_norm_rope(d, *t, stream=Stream)
    assert _called(seen, "rope", d) == at + (Stream.cuda_stream,)


@pytest.mark.parametrize("sinks", [0, 4, -1, (1 << 31) - 1])
def test_window_arguments(seen, sinks):
    d = hs.make_desc(2, 3, 16, 128, max_ctx=100)
    t, at = _tensors(9, (3, 4))
    hs.hs2_window_attn(d, sinks, *t, Tensor(4096, 3 << 32), stream=Stream)
    assert _called(seen, "window", d) == (sinks,) + at + (4096, 3 << 32, Stream.cuda_stream)


def test_accum_arguments(seen):
    d = hs.make_desc(2, 3, 16, 128, max_ctx=100)
    t, at = _tensors(8, (2, 6))
    hs.hs2_weight_accum(d, *t[:6], 0.5, *t[6:], Tensor(4096, 77), stream=Stream)
    assert _called(seen, "accum", d) == at[:6] + (0.5,) + at[6:] + (4096, 77, Stream.cuda_stream)


@pytest.mark.parametrize("holes", [(), (4, 5, 8, 9, 10)])
def test_evict_arguments(seen, holes):
    d = hs.make_evict_desc(2, 128, kv_capacity=4096)
    t, at = _tensors(13, holes)
    hs.hs2_kv_evict(d, *t, stream=Stream)
    assert _called(seen, "evict", d) == at + (Stream.cuda_stream,)


def test_a_status_is_raised(seen):
    with pytest.raises(hs.HS2Error) as e:                          # the library's own refusal
        L, m = hs.lib(), hs._fast()
        m.bind(*(ctypes.cast(f, P).value for f in (L.hs2_qk_norm_rope, L.hs2_window_attn, L.hs2_weight_accum, L.hs2_kv_evict)))
        hs.hs2_qk_norm_rope(hs.make_rope_desc(0, 1, 16, 128), *_tensors(14, ())[0], stream=Stream)
    assert e.value.status == 1


def test_wrong_arguments(seen):
    d, t = hs.make_desc(2, 3, 16, 128, max_ctx=100), _tensors(14, ())[0]
    m = hs._fast()
    for bad, err in (((d, *t), TypeError),                                        # another call's description
                     ((None, *t), TypeError), ((hs.make_rope_desc(1, 1, 1, 64), 5, *t[1:]), AttributeError)):
        with pytest.raises(err):
            hs.hs2_qk_norm_rope(*bad, stream=Stream)
    with pytest.raises(OverflowError):
        hs.hs2_window_attn(d, 1 << 31, *t[:9], Tensor(0, 5), stream=Stream)
    with pytest.raises(TypeError):
        hs.hs2_weight_accum(d, *t[:6], "much", *t[6:8], Tensor(0, 5), stream=Stream)
    with pytest.raises(TypeError):
        m.kv_evict(d, *t)
    with pytest.raises(ValueError):
        m.bind(1, 2, 3, 0)
    assert not seen


def test_tensors_give_their_addresses(seen):
    d, x = hs.make_evict_desc(1, 64, kv_capacity=8), torch.arange(40)
    hs.hs2_kv_evict(d, *(x[i:] for i in range(13)), stream=Stream)
    assert _called(seen, "evict", d)[:13] == tuple(x.data_ptr() + 8 * i for i in range(13))
