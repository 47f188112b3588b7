"""Host-side checks of the calls around the block where arguments meet: buffers that overlap.  An
accepted call ends with the missing device's status; where there is a device these do not run."""
import ctypes
import os

import pytest
import torch

import kv_shared_b200 as hs

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")

EVICT = ("len", "acc", "k", "v", "ks", "vs", "ko", "vo", "kso", "vso", "acco", "idx", "new_len")
WHERE = {n: (i + 1) << 32 for i, n in enumerate(EVICT)}
BATCH, CAP, OUT = 2, 4096, 2000
KEEP = 4 + 128 + 1024


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(hs.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return hs.lib()


def _evict(L, kv=hs.HS2_BF16, **at):
    d = hs.make_evict_desc(BATCH, 128, kv, 4, 128, 1024, CAP, OUT)
    return L.hs2_kv_evict(ctypes.byref(d), *[ctypes.c_void_p(at.get(n, WHERE[n])) for n in EVICT], None)


OUTPUTS = ("ko", "vo", "kso", "vso", "acco", "idx", "new_len")


@pytest.mark.parametrize("kv", [hs.HS2_BF16, hs.HS2_E4M3])
def test_evict_refuses_outputs_over_the_lengths(L, kv):
    """Every output that starts at the lengths, reaches into them or starts at their second entry; the new
    lengths may be the lengths themselves, but not one off."""
    for out in OUTPUTS:
        if kv != hs.HS2_E4M3 and out in ("kso", "vso"):
            continue
        for off in (0, 16, -16) if out in ("ko", "vo") else (0, 4, -4):
            at = WHERE["len"] + off
            met = off == 0 or (off > 0 and off < BATCH * 4) or (off < 0 and (out != "new_len" or -off < BATCH * 4))
            status = _evict(L, kv, **{out: at})
            assert (status == hs.HS2_ERR_INVALID_ARG) == (met and (out, off) != ("new_len", 0)), (out, off)


@pytest.mark.parametrize("kv", [hs.HS2_BF16, hs.HS2_E4M3])
def test_evict_refuses_new_lengths_inside_an_input(L, kv):
    for name in ("acc", "k", "v") + (("ks", "vs") if kv == hs.HS2_E4M3 else ()):
        for off in (0, 64, BATCH * CAP * 4 - 4, -4):
            assert _evict(L, kv, new_len=WHERE[name] + off) == hs.HS2_ERR_INVALID_ARG, (name, off)
        assert _evict(L, kv, new_len=WHERE[name] - BATCH * 4) != hs.HS2_ERR_INVALID_ARG
    # the lengths' own place is theirs only where nothing else lies there
    assert _evict(L, kv, len=WHERE["acc"], new_len=WHERE["acc"]) == hs.HS2_ERR_INVALID_ARG


def test_evict_takes_buffers_that_touch(L):
    """The first byte after an input is free."""
    assert _evict(L, new_len=WHERE["len"] + BATCH * 4) != hs.HS2_ERR_INVALID_ARG
    assert _evict(L, idx=WHERE["len"] + BATCH * 4) != hs.HS2_ERR_INVALID_ARG
    assert _evict(L, idx=WHERE["len"] - BATCH * KEEP * 4) != hs.HS2_ERR_INVALID_ARG


@pytest.mark.parametrize("kv", [hs.HS2_BF16, hs.HS2_E4M3])
def test_evict_refuses_outputs_over_one_another(L, kv):
    """k_out holds the selection's counts before its rows: an index or a length written there, or any
    output twice in one place, would be the call's own undoing."""
    names = [n for n in OUTPUTS if kv == hs.HS2_E4M3 or n not in ("kso", "vso")]
    for a in names:
        for b in names:
            if a != b:
                for off in (0,) if b == "new_len" else (0, 16):
                    assert _evict(L, kv, **{a: WHERE[b] + off}) == hs.HS2_ERR_INVALID_ARG, (a, b, off)
    assert _evict(L, kv, idx=WHERE["ko"] + BATCH * OUT * 128 * (1 if kv == hs.HS2_E4M3 else 2)) != hs.HS2_ERR_INVALID_ARG
    assert _evict(L, kv, new_len=WHERE["idx"] + BATCH * KEEP * 4) != hs.HS2_ERR_INVALID_ARG


def test_rope_reads_its_rows_with_plain_loads():
    """q_out may be q, so the rows' loads may not take the path for memory that the kernel does not write."""
    src = os.path.join(os.path.dirname(os.path.abspath(hs.__file__)), "csrc", "rope_cache.cu")
    loads = [body.split("\n}")[0] for body in open(src).read().split("void load8(")[1:]]
    assert len(loads) == 2
    assert all("__ldg" not in body and "reinterpret_cast<const" in body for body in loads)
