"""Host-side checks of the calls around the block: refusals (nothing is launched), workspace
sizes, and the fp64 forms that the GPU tests compare with, against independent identities."""
import ctypes
import math
import os

import pytest
import torch

import cache_ops_ref as ref
import kv_shared_b200 as hs

FAKE, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(hs.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return hs.lib()


def _desc(**kw):
    base = dict(batch=2, n_q=3, heads=16, head_dim=128, max_ctx=4096)
    base.update(kw)
    return hs.make_desc(**base)


# ---------------------------------------------------------------- refusals
def _rope(L, d, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qw=FAKE, kw=FAKE, freq=FAKE, row0=FAKE, pos=FAKE, n_rows=None, q_out=FAKE,
             kc=FAKE, vc=FAKE, ks=None, vs=None)
    a.update(kw)
    return L.hs2_qk_norm_rope(ctypes.byref(d), a["q"], a["k"], a["v"], a["qw"], a["kw"], a["freq"], a["row0"],
                              a["pos"], a["n_rows"], a["q_out"], a["kc"], a["vc"], a["ks"], a["vs"], None)


@pytest.mark.parametrize("desc, args, status", [
    (dict(batch=0), {}, 1), (dict(n=0), {}, 1), (dict(heads=0), {}, 1), (dict(eps=-1.0), {}, 1),
    (dict(eps=math.nan), {}, 1), (dict(eps=math.inf), {}, 1), (dict(rot_dim=144), {}, 1), (dict(rot_dim=-16), {}, 1),
    (dict(rot_dim=24), {}, 2), (dict(head_dim=96), {}, 2), (dict(heads=129), {}, 2), (dict(in_dtype=2), {}, 2),
    (dict(kv_dtype=0), {}, 2), (dict(kv_dtype=7), {}, 2), (dict(q_row=2047), {}, 1), (dict(q_row=2052), {}, 1),
    (dict(k_row=64), {}, 1), (dict(v_row=130), {}, 1), (dict(kv_capacity=0), {}, 1),
    (dict(kv_capacity=1 << 31), {}, 2), (dict(kv_capacity=1 << 62), {}, 2), (dict(q_row=1 << 40), {}, 2),
    ({}, dict(q=None, k=None, v=None), 1), ({}, dict(row0=None), 1), ({}, dict(q_out=None), 1),
    ({}, dict(kc=None), 1), ({}, dict(vc=None), 1), ({}, dict(freq=None), 1), ({}, dict(q=ODD), 1),
    ({}, dict(qw=ODD), 1), ({}, dict(freq=ODD), 1), ({}, dict(kc=ODD), 1),
    (dict(q_row=2304), dict(q_out=FAKE), 1),                       # in place needs contiguous rows
    (dict(kv_dtype=2), {}, 1),                                     # e4m3 needs scales
])
def test_rope_refuses(L, desc, args, status):
    base = dict(batch=2, n=5, heads=16, head_dim=128)
    base.update(desc)
    d = hs.make_rope_desc(**base)
    if "q_row" not in desc and "q_out" not in args:
        args = dict(args, q_out=ctypes.c_void_p(0x2000))
    assert _rope(L, d, **args) == status


def _window(L, d, sinks=4, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ks=None, vs=None, pos=FAKE, n_rows=None, o=FAKE, lse=None, ws=FAKE, size=1 << 40)
    a.update(kw)
    return L.hs2_window_attn(ctypes.byref(d), sinks, a["q"], a["k"], a["v"], a["ks"], a["vs"], a["pos"], a["n_rows"],
                             a["o"], a["lse"], a["ws"], a["size"], None)


BAD_DESC = [
    (dict(batch=0), 1), (dict(n_q=0), 1), (dict(heads=0), 1), (dict(max_ctx=2, kv_capacity=4096), 1),
    (dict(kv_capacity=100), 1), (dict(softmax_scale=-1.0), 1), (dict(softmax_scale=math.nan), 1),
    (dict(softmax_scale=math.inf), 1), (dict(head_dim=96), 2), (dict(heads=129), 2), (dict(q_dtype=0), 2),
    (dict(kv_dtype=0), 2), (dict(q_dtype=2), 2), (dict(kv_dtype=9), 2),
    (dict(kv_capacity=1 << 31), 2), (dict(kv_capacity=1 << 62), 2),
    (dict(n_q=1 << 24, heads=128, max_ctx=1 << 24), 2),
]


@pytest.mark.parametrize("desc, status", BAD_DESC + [(dict(window=0), 1), (dict(window=-5), 1)])
def test_window_refuses_descriptions(L, desc, status):
    d = _desc(**desc)
    assert _window(L, d) == status
    assert hs.hs2_window_workspace_size(d, 4) == 0


@pytest.mark.parametrize("args, status", [
    (dict(sinks=-1), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(pos=None), 1),
    (dict(o=None), 1), (dict(ws=None), 1), (dict(q=ODD), 1), (dict(lse=ODD), 1), (dict(ws=ODD), 1),
    (dict(n_rows=ctypes.c_void_p(0x1001)), 1), (dict(size=0), 3), (dict(size=4095), 3),
])
def test_window_refuses_arguments(L, args, status):
    assert _window(L, _desc(), **args) == status
    if "ks" not in args and args.get("sinks", 0) >= 0 and status == 1:
        assert _window(L, _desc(kv_dtype=hs.HS2_E4M3)) == 1        # e4m3 needs scales


def test_window_workspace_covers_the_split(L):
    # one token over a long window is cut over the SMs and needs its parts' room; a short window is not
    assert hs.hs2_window_workspace_size(_desc(n_q=1, window=128), 4) == 4096
    d = _desc(batch=1, n_q=1, window=1 << 20, max_ctx=1 << 20)
    n = hs.hs2_window_workspace_size(d, 4)
    assert n > 4096 and (n - 4096) % (16 * (128 * 4 + 8)) == 0
    assert _window(L, d, size=n - 1) == 3


def _accum(L, d, **kw):
    a = dict(q=FAKE, k=FAKE, ks=None, lse=FAKE, pos=FAKE, n_rows=None, decay=1.0, acc_in=FAKE, acc_out=FAKE, ws=FAKE,
             size=1 << 40)
    a.update(kw)
    return L.hs2_weight_accum(ctypes.byref(d), a["q"], a["k"], a["ks"], a["lse"], a["pos"], a["n_rows"], a["decay"],
                              a["acc_in"], a["acc_out"], a["ws"], a["size"], None)


@pytest.mark.parametrize("desc, status", BAD_DESC)
def test_accum_refuses_descriptions(L, desc, status):
    d = _desc(**desc)
    assert _accum(L, d) == status
    assert hs.hs2_weight_accum_workspace_size(d) == 0


@pytest.mark.parametrize("args, status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(lse=None), 1), (dict(pos=None), 1), (dict(acc_out=None), 1),
    (dict(ws=None), 1), (dict(decay=-0.5), 1), (dict(decay=math.nan), 1), (dict(decay=math.inf), 1), (dict(k=ODD), 1),
    (dict(lse=ODD), 1), (dict(acc_out=ctypes.c_void_p(0x1002)), 1), (dict(size=0), 3),
])
def test_accum_refuses_arguments(L, args, status):
    assert _accum(L, _desc(), **args) == status


def _evict(L, d, **kw):
    names = ("len", "acc", "k", "v", "ks", "vs", "ko", "vo", "kso", "vso", "acco", "idx", "new_len")
    a = {n: FAKE for n in names}
    a.update(kw)
    return L.hs2_kv_evict(ctypes.byref(d), *[a[n] for n in names], None)


@pytest.mark.parametrize("desc, args, status", [
    (dict(batch=0), {}, 1), (dict(sinks=-1), {}, 1), (dict(window=-1), {}, 1), (dict(budget=-1), {}, 1),
    (dict(sinks=0, window=0, budget=0, out_capacity=8), {}, 1), (dict(out_capacity=1155), {}, 1),
    (dict(kv_capacity=0), {}, 1), (dict(head_dim=96), {}, 2), (dict(kv_dtype=5), {}, 2),
    (dict(kv_capacity=1 << 31), {}, 2), (dict(out_capacity=1 << 31), {}, 2), (dict(kv_capacity=1 << 62), {}, 2),
    (dict(sinks=(1 << 31) - 1, window=(1 << 31) - 1, budget=(1 << 31) - 1), {}, 2),
    ({}, dict(len=None), 1), ({}, dict(acc=None), 1), ({}, dict(idx=None), 1), ({}, dict(new_len=None), 1),
    ({}, dict(ko=None), 1), ({}, dict(k=ODD), 1), ({}, dict(vo=ODD), 1), ({}, dict(acc=ctypes.c_void_p(0x1002)), 1),
    (dict(kv_dtype=2), dict(ks=None), 1), (dict(kv_dtype=2), dict(vso=None), 1),
])
def test_evict_refuses(L, desc, args, status):
    base = dict(batch=2, head_dim=128, sinks=4, window=128, budget=1024, kv_capacity=4096)
    base.update(desc)
    assert _evict(L, hs.make_evict_desc(**base), **args) == status


@pytest.mark.parametrize("kv", [hs.HS2_BF16, hs.HS2_E4M3])
@pytest.mark.parametrize("out, at", [("ko", "k"), ("vo", "v"), ("acco", "acc"), ("idx", "acc"), ("ko", "acc"), ("vo", "k")])
def test_evict_refuses_a_cache_cut_in_place(L, kv, out, at):
    """Outputs that start at an input, inside it, or reach into it."""
    names = ("len", "acc", "k", "v", "ks", "vs", "ko", "vo", "kso", "vso", "acco", "idx", "new_len")
    where = {n: (i + 1) << 32 for i, n in enumerate(names)}
    d = hs.make_evict_desc(2, 128, kv, 4, 128, 1024, 4096, 2000)
    for off in (0, 64, 2 * 4096 * 4 - 16, -16):
        args = {n: ctypes.c_void_p(x) for n, x in where.items()}
        args[out] = ctypes.c_void_p(where[at] + off)
        assert _evict(L, d, **args) == 1
    if kv == hs.HS2_E4M3:
        args = {n: ctypes.c_void_p(x) for n, x in where.items()}
        assert _evict(L, d, **dict(args, kso=args["ks"])) == _evict(L, d, **dict(args, vso=args["vs"])) == 1


# ---------------------------------------------------------------- the fp64 forms
def test_rotation_keeps_lengths_and_relative_angles():
    g = torch.Generator().manual_seed(1)
    freq = 1e4 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    q, k = (torch.randn(64, generator=g, dtype=torch.float64) for _ in range(2))
    for inter in (False, True):
        a = ref.rotate(q, 900_005, freq, inter)
        assert abs(float(a.norm() - q.norm())) < 1e-12
        near = ref.rotate(q, 5, freq, inter) @ ref.rotate(k, 3, freq, inter)
        far = a @ ref.rotate(k, 900_003, freq, inter)
        assert abs(float(near - far)) < 1e-9


def test_window_form_meets_full_attention_and_its_own_mask():
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((3, 64), (40, 64), (40, 64)))
    o, lse, _, _ = ref.window_row(q, k, v, 39, 40, 0, 0.125)
    w = torch.softmax(q @ k.T * 0.125, -1)
    assert torch.allclose(o, w @ v, atol=1e-12)
    o2, _, _, _ = ref.window_row(q, k, v, 39, 1, 100, 0.125)       # sinks reach past the window: all rows again
    assert torch.allclose(o2, o, atol=1e-12)
    o3, _, _, _ = ref.window_row(q, k, v, 39, 1, 0, 0.125)         # only itself
    assert torch.allclose(o3, v[39].expand(3, 64), atol=1e-12)


def test_weight_totals_sum_to_the_rows_and_heads():
    g = torch.Generator().manual_seed(3)
    q, k = torch.randn(5, 4, 64, generator=g, dtype=torch.float64), torch.randn(30, 64, generator=g, dtype=torch.float64)
    lse = torch.stack([(q[r] @ k[:20 + r + 1].T * 0.125).logsumexp(-1) for r in range(5)])
    t, _ = ref.weight_total(q, lse, k, 20, 0.125)
    assert t.shape == (25,) and abs(float(t.sum()) - 20.0) < 1e-10


def test_evicted_rows_ties_and_nan():
    acc = [9.0, 1.0, 1.0, math.nan, 0.0, -0.0, 2.0, 1.0, 5.0, 5.0]
    assert ref.evict_rows(acc, 10, 1, 2, 3) == [0, 1, 2, 6, 8, 9]
    assert ref.evict_rows(acc, 10, 0, 0, 8) == [0, 1, 2, 4, 6, 7, 8, 9]
    assert ref.evict_rows(acc, 5, 1, 2, 3) == [0, 1, 2, 3, 4]
