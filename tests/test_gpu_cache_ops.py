"""GPU tests of the calls around the block against plain fp64 forms (cache_ops_ref.py).

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value, to e4m3 by 2^-4 (by half of
2^-9 scale units below its normal range).  fp32 arithmetic: a dot product of D terms is off by at
most D 2^-24 times the sum of the terms' magnitudes (`mag`), a tensor-core sum is allowed twice
that; a weight exp(s - lse) then moves by that much relative.
"""
import math

import pytest
import torch

import cache_ops_ref as ref
import kv_shared_b200 as hs

pytestmark = pytest.mark.gpu

KIND = {"f32": hs.HS2_F32, "bf16": hs.HS2_BF16, "e4m3": hs.HS2_E4M3}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_BF16, HALF_E4M3 = 2.0 ** -8, 2.0 ** -4


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _cache(g, b, cap, d, kv, std=1.0):
    """(k, v, ks, vs) CPU tensors as the library holds them."""
    x = [torch.randn(b, cap, d, generator=g) * std for _ in range(2)]
    if kv == "e4m3":
        (k, ks), (v, vs) = ref.quantize(x[0]), ref.quantize(x[1])
        return k, v, ks, vs
    return x[0].to(DT[kv]), x[1].to(DT[kv]), None, None


def _cu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _poison(t, mask):
    """Rows where mask holds become NaN (uint8: the NaN code)."""
    t = t.clone()
    t[mask] = 0x7f if t.dtype == torch.uint8 else math.nan
    return t


# ------------------------------------------------------------------ norm, rotation, cache rows
ROPE = [
    # b, n, h, d, rot, interleaved, in, cache
    (2, 1, 16, 128, 128, False, "bf16", "bf16"),
    (3, 7, 16, 128, 128, True, "bf16", "e4m3"),
    (2, 5, 5, 64, 64, False, "f32", "f32"),
    (1, 33, 8, 64, 48, False, "f32", "e4m3"),
    (2, 9, 3, 128, 96, False, "bf16", "bf16"),
    (2, 3, 1, 128, 16, True, "f32", "bf16"),
    (1, 2, 24, 64, 0, False, "bf16", "e4m3"),
    (1, 4, 128, 64, 32, True, "bf16", "bf16"),
    (5, 700, 2, 128, 128, False, "bf16", "bf16"),
]


@pytest.mark.parametrize("b, n, h, d, rot, inter, dt, kv", ROPE)
@pytest.mark.parametrize("far", [False, True])
def test_rope_rows(b, n, h, d, rot, inter, dt, kv, far):
    g = _gen(1000 * b + 10 * n + h)
    pad = 8                                                   # a fused projection's row is longer than the heads
    row = (h + 2) * d + pad
    qkv = torch.randn(b, n, row, generator=g).to(DT[dt])
    qkv[:, :, h * d:(h + 1) * d] *= 3
    qkv[0, n - 1, (h + 1) * d:(h + 2) * d] = 0                # a value row of zeros
    qw, kw = 1 + 0.2 * torch.randn(d, generator=g), 1 + 0.2 * torch.randn(d, generator=g)
    freq = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    cap = n + 5
    row0 = torch.randint(0, 6, (b,), generator=g, dtype=torch.int32)
    pos = None
    if far:
        pos = torch.randint(0, 1 << 20, (b, n), generator=g, dtype=torch.int32)
        pos[0, 0] = (1 << 31) - 1
    n_rows = torch.tensor([(n + i) % (n + 1) if far else n for i in range(b)], dtype=torch.int32)   # n, 0, 1, ..
    mark = 7
    cdt = torch.uint8 if kv == "e4m3" else DT[kv]
    kc, vc = torch.full((b, cap, d), mark, dtype=cdt), torch.full((b, cap, d), mark, dtype=cdt)
    ks, vs = (torch.full((b, cap), 5.0), torch.full((b, cap), 5.0)) if kv == "e4m3" else (None, None)
    q_out = torch.full((b, n, h, d), float(mark), dtype=DT[dt])
    dev = _cu(qkv, qw, kw, freq, row0, pos, n_rows if far else None, q_out, kc, vc, ks, vs)
    desc = hs.make_rope_desc(b, n, h, d, rot_dim=rot, interleaved=inter, in_dtype=KIND[dt], kv_dtype=KIND[kv],
                             q_row=row, k_row=row, v_row=row, kv_capacity=cap, eps=1e-5)
    x = dev[0]
    hs.hs2_qk_norm_rope(desc, x, x[..., h * d:], x[..., (h + 1) * d:], *dev[1:])
    torch.cuda.synchronize()
    q_got, kc_got, vc_got = dev[7].cpu(), dev[8].cpu(), dev[9].cpu()
    for s in range(b):
        m = int(n_rows[s]) if far else n
        rows = torch.arange(m)
        p = (pos[s, :m] if far else row0[s] + rows).tolist()
        src = qkv[s, :m, :(h + 2) * d].reshape(m, h + 2, d)
        q_ref = ref.norm_rope(src[:, :h], qw, 1e-5, p, freq, inter)
        k_ref = ref.norm_rope(src[:, h:h + 1], kw, 1e-5, p, freq, inter)[:, 0]
        v_ref = src[:, h + 1].double()
        # fp32 slack of a rotated pair: 2^-18 of the head's largest magnitude
        half = HALF_BF16 if dt == "bf16" else 0.0
        err = (q_got[s, :m].double() - q_ref).abs()
        assert (err <= half * q_ref.abs() + 2.0 ** -18 * q_ref.abs().amax(-1, keepdim=True)).all()
        assert (q_got[s, m:] == mark).all()
        at = int(row0[s]) + rows
        other = torch.ones(cap, dtype=torch.bool)
        other[at] = False
        for got, want, sc in ((kc_got, k_ref, dev[10]), (vc_got, v_ref, dev[11])):
            assert (got[s, other] == mark).all()
            slack = 2.0 ** -18 * want.abs().amax(-1, keepdim=True)
            if kv == "e4m3":
                scale = sc.cpu()[s]
                assert (scale[other] == 5.0).all()
                amax = want.abs().amax(-1)
                s_ref = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
                assert (scale[at].double() - s_ref).abs().le(2.0 ** -17 * s_ref).all()
                val = ref.wide(got[s, at], scale[at])
                lim = HALF_E4M3 * want.abs() + 2.0 ** -10 * s_ref[:, None] + 2 * slack
            else:
                val = got[s, at].double()
                lim = (HALF_BF16 if kv == "bf16" else 0.0) * want.abs() + slack
            assert ((val - want).abs() <= lim).all()


def test_rope_parts_in_place_and_without_norm():
    g = _gen(5)
    b, n, h, d = 2, 6, 4, 128
    q0, k0 = torch.randn(b, n, h, d, generator=g), torch.randn(b, n, d, generator=g)
    freq = 1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    row0 = torch.tensor([3, 0], dtype=torch.int32)
    q, k, fr, r0 = _cu(q0, k0, freq, row0)
    desc = hs.make_rope_desc(b, n, h, d, normalize=False, in_dtype=hs.HS2_F32, kv_dtype=hs.HS2_F32, kv_capacity=8)
    hs.hs2_qk_norm_rope(desc, q, None, None, None, None, fr, r0, None, None, q, None, None)     # queries alone, in place
    kc = torch.full((b, 8, d), 7.0, device="cuda")
    hs.hs2_qk_norm_rope(desc, None, k, None, None, None, fr, r0, None, None, None, kc, None)    # keys alone
    torch.cuda.synchronize()
    for s in range(b):
        p = [int(row0[s]) + t for t in range(n)]
        want = ref.norm_rope(q0[s], None, 0.0, p, freq, False, normalize=False)
        assert (q[s].cpu().double() - want).abs().le(2.0 ** -18 * want.abs().amax(-1, keepdim=True)).all()
        want = ref.norm_rope(k0[s][:, None], None, 0.0, p, freq, False, normalize=False)[:, 0]
        fit = min(n, 8 - int(row0[s]))                         # rows past the cache are not written
        got = kc[s, int(row0[s]):int(row0[s]) + fit].cpu().double()
        assert (got - want[:fit]).abs().le(2.0 ** -18 * want[:fit].abs().amax(-1, keepdim=True)).all()
    assert (kc[1, n:] == 7).all() and (kc[0, :3] == 7).all()


# ------------------------------------------------------------------ sliding window with sinks
def _check_window(q, k, v, ks, vs, pos0, n_rows, window, sinks, o, lse, kv, mark, rows=None):
    b, n, h, d = q.shape
    scale = d ** -0.5
    for s in range(b):
        m = n if n_rows is None else int(n_rows[s])
        kk, vv = ref.wide(k[s], None if ks is None else ks[s]), ref.wide(v[s], None if vs is None else vs[s])
        for r in (range(m) if rows is None else [x for x in rows if x < m]):
            o_ref, l_ref, mag, av = ref.window_row(q[s, r].double(), kk, vv, int(pos0[s]) + r, window, sinks, scale)
            ds = (2 * d * mag + 8 * (l_ref.abs() + mag)) * 2.0 ** -24 + 2.0 ** -21    # a weight's relative error
            if kv == "f32":
                lim = (2 * ds + 2.0 ** -16)[:, None] * av
            else:
                lim = (2 * ds + HALF_BF16)[:, None] * av + HALF_BF16 * o_ref.abs()
            got = o[s, r].double()
            assert ((got - o_ref).abs() <= lim).all(), (s, r, float(((got - o_ref).abs() / lim).max()))
            # lse: the logit's error, the sum's, and the fp32 rounding of a value of its size
            assert ((lse[s, r].double() - l_ref).abs() <= 2 * ds + 2.0 ** -16 + 2.0 ** -22 * l_ref.abs()).all()
        assert (o[s, m:] == mark).all() and (lse[s, m:] == mark).all()


def _run_window(g, b, n, h, d, window, sinks, ctx, kv, ragged=False, pos0=None, poison=True, rows=None):
    dt = "f32" if kv == "f32" else "bf16"
    q = torch.randn(b, n, h, d, generator=g).to(DT[dt])
    k, v, ks, vs = _cache(g, b, ctx, d, kv)
    if pos0 is None:
        pos0 = torch.tensor([(ctx - n) if i == 0 else int(torch.randint(0, ctx - n + 1, (1,), generator=g))
                             for i in range(b)], dtype=torch.int32)
    n_rows = torch.tensor([(n, 0, n // 2, 1)[i % 4] for i in range(b)], dtype=torch.int32) if ragged else None
    # rows that no query attends to hold NaN
    seen = torch.zeros(b, ctx, dtype=torch.bool)
    for s in range(b):
        m = n if n_rows is None else int(n_rows[s])
        if m:
            seen[s, max(0, int(pos0[s]) - window + 1):int(pos0[s]) + m] = True
            seen[s, :min(sinks, int(pos0[s]) + m)] = True
    kp, vp = (_poison(k, ~seen), _poison(v, ~seen)) if poison else (k, v)
    mark = 7.0
    dev = _cu(q, kp, vp, ks, vs, pos0, n_rows)
    o = torch.full((b, n, h, d), mark, dtype=DT[dt], device="cuda")
    lse = torch.full((b, n, h), mark, device="cuda")
    desc = hs.make_desc(b, n, h, d, window=window, budget=0, q_dtype=KIND[dt], kv_dtype=KIND[kv], max_ctx=ctx)
    ws = hs.alloc_window_workspace(desc, sinks)
    hs.hs2_window_attn(desc, sinks, *dev, o, lse, ws)
    assert hs.hs2_last_status(ws) == hs.HS2_OK
    _check_window(q, k, v, ks, vs, pos0, n_rows, window, sinks, o.cpu(), lse.cpu(), kv, mark, rows)
    o2 = torch.full_like(o, mark)                              # without lse; the same bits
    hs.hs2_window_attn(desc, sinks, *dev, o2, None, ws)
    assert torch.equal(o, o2)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("b, h, d, window, sinks, ctx", [
    (1, 16, 128, 1, 0, 1), (2, 16, 128, 128, 4, 1000), (3, 5, 64, 33, 0, 77), (2, 24, 128, 7, 17, 300),
    (1, 1, 64, 1 << 30, 3, 513), (2, 128, 64, 16, 1, 40), (1, 16, 128, 100, 100, 150), (2, 16, 128, 64, 5, 70),
])
def test_window_single_tokens(kv, b, h, d, window, sinks, ctx):
    _run_window(_gen(h + ctx), b, 1, h, d, window, sinks, ctx, kv)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("b, h, window, sinks, ctx", [(1, 16, 6000, 4, 7001), (3, 12, 3000, 20, 4099)])
def test_window_single_tokens_split_and_joined(kv, b, h, window, sinks, ctx):
    _run_window(_gen(ctx), b, 1, h, 128, window, sinks, ctx, kv)
    _run_window(_gen(ctx), b, 1, h, 128, window, sinks, ctx, kv, ragged=True)


CHUNKS = [
    # b, n, h, d, window, sinks, ctx
    (1, 2, 16, 128, 128, 4, 2), (2, 37, 16, 128, 16, 4, 150), (4, 21, 8, 64, 5, 2, 90), (2, 65, 3, 128, 40, 0, 65),
    (1, 130, 16, 128, 128, 4, 700), (4, 50, 12, 128, 200, 130, 400), (1, 40, 1, 64, 1, 1, 300), (2, 9, 128, 64, 30, 3, 50),
    (1, 300, 5, 128, 64, 16, 1300),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("b, n, h, d, window, sinks, ctx", CHUNKS)
def test_window_chunks(kv, b, n, h, d, window, sinks, ctx):
    _run_window(_gen(n + ctx), b, n, h, d, window, sinks, ctx, kv, ragged=b == 4)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_window_long_chunk(kv):
    _run_window(_gen(3), 1, 1030, 16, 128, 900, 4, 2500, kv, rows=[0, 1, 15, 16, 511, 777, 1023, 1024, 1029])


def test_window_large_logits_and_offsets():
    # logits of several hundred: the running maximum has to carry; and a value offset of 1e4
    g = _gen(9)
    b, n, h, d, ctx = 1, 48, 16, 128, 400
    q = (torch.randn(b, n, h, d, generator=g) * 16).to(torch.bfloat16)
    k = (torch.randn(b, ctx, d, generator=g) * 4).to(torch.bfloat16)
    k = k[:, torch.argsort(k[0].float() @ q[0, 0, 0].float())]             # the first head's logits rise along the keys
    v = (torch.randn(b, ctx, d, generator=g) + 1e4).to(torch.bfloat16)
    pos0 = torch.tensor([ctx - n], dtype=torch.int32)
    for rows in (n, 1):
        dq = q[:, :rows].contiguous()
        dev = _cu(dq, k, v, None, None, pos0, None)
        o, lse = torch.zeros_like(dev[0]), torch.zeros(b, rows, h, device="cuda")
        desc = hs.make_desc(b, rows, h, d, window=300, budget=0, max_ctx=ctx)
        ws = hs.alloc_window_workspace(desc, 2)
        hs.hs2_window_attn(desc, 2, *dev, o, lse, ws)
        _check_window(dq, k, v, None, None, pos0, None, 300, 2, o.cpu(), lse.cpu(), "bf16", 0)


def test_window_reports_positions_outside_the_context():
    for n in (1, 40):
        desc = hs.make_desc(2, n, 16, 128, window=8, budget=0, max_ctx=64)
        ws = hs.alloc_window_workspace(desc, 1)
        q = torch.randn(2, n, 16, 128, device="cuda").bfloat16()
        kv = torch.randn(2, 64, 128, device="cuda").bfloat16()
        o = torch.zeros_like(q)
        for bad in ([-1, 0], [0, 65 - n]):
            pos0 = torch.tensor(bad, dtype=torch.int32, device="cuda")
            hs.hs2_window_attn(desc, 1, q, kv, kv, None, None, pos0, None, o, None, ws)
            assert hs.hs2_last_status(ws) == hs.HS2_ERR_INDEX
        assert hs.hs2_last_status(ws) == hs.HS2_OK


# ------------------------------------------------------------------ accumulated weight
def _run_accum(g, b, n, h, d, ctx, kv, decay, ragged, in_place=False, none_in=False):
    dt = "f32" if kv == "f32" else "bf16"
    scale = d ** -0.5
    q = torch.randn(b, n, h, d, generator=g).to(DT[dt])
    k, _, ks, _ = _cache(g, b, ctx, d, kv)
    pos0 = torch.tensor([(ctx - n) if i == 0 else int(torch.randint(0, ctx - n + 1, (1,), generator=g))
                         for i in range(b)], dtype=torch.int32)
    n_rows = torch.tensor([(n, 0, n // 2, 1)[i % 4] for i in range(b)], dtype=torch.int32) if ragged else None
    lse = torch.full((b, n, h), math.nan)                      # rows out of use hold anything
    want, mags = [], []
    acc = torch.rand(b, ctx, generator=g) * 3
    kp = k.clone()
    for s in range(b):
        m = n if n_rows is None else int(n_rows[s])
        kk = ref.wide(k[s], None if ks is None else ks[s])
        for r in range(m):
            lse[s, r] = ((q[s, r].double() @ kk[:int(pos0[s]) + r + 1].T) * scale).logsumexp(-1).float()
        t, mag = ref.weight_total(q[s, :m].double(), lse[s, :m].double(), kk, int(pos0[s]), scale)
        want.append(t)
        mags.append(mag)
        past = torch.zeros(ctx, dtype=torch.bool)
        past[int(pos0[s]) + m:] = True
        kp[s] = _poison(k[s], past)
    dev = _cu(q, kp, ks, lse, pos0, n_rows)
    mark = -3.0
    a_in = None if none_in else acc.cuda()
    out = a_in if in_place else torch.full((b, ctx), mark, device="cuda")
    desc = hs.make_desc(b, n, h, d, q_dtype=KIND[dt], kv_dtype=KIND[kv], max_ctx=ctx)
    ws = hs.alloc_accum_workspace(desc)
    hs.hs2_weight_accum(desc, *dev, decay, a_in, out, ws)
    assert hs.hs2_last_status(ws) == hs.HS2_OK
    got = out.cpu().double()
    for s in range(b):
        end = want[s].numel()
        old = 0.0 if none_in else decay * acc[s, :end].double()
        # a weight's relative error, then n h additions of positive terms and the last rounding
        rel = (2 * d * mags[s] + 8 * (mags[s] + 12)) * 2.0 ** -24 + 2.0 ** -20 + n * h * 2.0 ** -24
        err = (got[s, :end] - (old + want[s])).abs()
        assert (err <= rel * want[s] + 2.0 ** -22 * (old + want[s])).all(), (s, float((err / (old + want[s])).max()), rel)
        assert (out.cpu()[s, end:] == (acc[s, end:] if in_place else mark)).all()
    if not in_place:
        again = torch.full_like(out, mark)
        hs.hs2_weight_accum(desc, *dev, decay, a_in, again, ws)
        assert torch.equal(out, again)


ACCUM = [
    # b, n, h, d, ctx
    (1, 1, 16, 128, 1), (2, 1, 16, 128, 777), (3, 5, 5, 64, 130), (2, 32, 16, 128, 500), (4, 20, 12, 128, 129),
    (1, 70, 1, 64, 70), (2, 3, 128, 64, 100), (1, 129, 8, 128, 400), (1, 16, 16, 128, 3000),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("b, n, h, d, ctx", ACCUM)
def test_accum(kv, b, n, h, d, ctx):
    _run_accum(_gen(n + ctx), b, n, h, d, ctx, kv, 0.75, ragged=b == 4)


def test_accum_in_place_and_from_nothing():
    _run_accum(_gen(1), 2, 9, 16, 128, 300, "bf16", 1.0, False, in_place=True)
    _run_accum(_gen(2), 4, 9, 16, 128, 300, "bf16", 0.5, True, in_place=True)
    _run_accum(_gen(3), 2, 9, 16, 128, 300, "e4m3", 1.0, False, none_in=True)


# ------------------------------------------------------------------ eviction
def _run_evict(acc, lens, sinks, window, budget, kv, d, out_extra=0, seed=0, with_acc=True):
    b, cap = acc.shape
    g = _gen(seed)
    keep = sinks + window + budget
    k, v, ks, vs = _cache(g, b, cap, d, kv)
    out_cap = keep + out_extra
    mark = 7
    ko, vo = torch.full((b, out_cap, d), mark, dtype=k.dtype), torch.full((b, out_cap, d), mark, dtype=k.dtype)
    sc = [torch.full((b, out_cap), 5.0) if ks is not None else None for _ in range(2)]
    ao = torch.full((b, out_cap), 5.0) if with_acc else None
    idx, new_len = torch.full((b, keep), 99, dtype=torch.int32), torch.full((b,), 99, dtype=torch.int32)
    dev = _cu(torch.tensor(lens, dtype=torch.int32), acc, k, v, ks, vs, ko, vo, *sc, ao, idx, new_len)
    desc = hs.make_evict_desc(b, d, KIND[kv], sinks=sinks, window=window, budget=budget, kv_capacity=cap,
                              out_capacity=out_cap)
    hs.hs2_kv_evict(desc, *dev)
    torch.cuda.synchronize()
    _, _, _, _, _, _, ko, vo, kso, vso, ao, idx, new_len = [None if t is None else t.cpu() for t in dev]
    for s in range(b):
        rows = ref.evict_rows(acc[s], lens[s], sinks, window, budget)
        m = len(rows)
        assert int(new_len[s]) == m
        assert idx[s, :m].tolist() == rows and (idx[s, m:] == -1).all()
        for got, src, fill in ((ko, k, mark), (vo, v, mark), (kso, ks, 5.0), (vso, vs, 5.0), (ao, acc, 5.0)):
            if got is not None:
                x, y = got[s, :m], src[s, rows]
                assert torch.equal(x.view(torch.uint8), y.contiguous().view(torch.uint8))
                assert (got[s, m:] == fill).all()


@pytest.mark.parametrize("kv, d", [("bf16", 128), ("e4m3", 128), ("f32", 64), ("f32", 128), ("bf16", 64), ("e4m3", 64)])
def test_evict_types(kv, d):
    acc = (torch.randn(3, 1000, generator=_gen(4)) * 2).exp()
    _run_evict(acc, [1000, 77, 501], 4, 60, 100, kv, d, out_extra=3)


@pytest.mark.parametrize("cap, lens, sinks, window, budget", [
    (1, [1, 0], 0, 0, 1), (5, [5, 3], 1, 1, 1), (5, [5, 4], 0, 0, 3), (5, [5, 5], 0, 3, 0), (5, [4, 5], 2, 0, 0),
    (100, [100, 99], 3, 5, 91), (100, [100, 0], 0, 0, 99), (33000, [33000, 32768], 16, 128, 8000),
    (70001, [70001, 40000], 0, 1, 1),
])
def test_evict_sizes(cap, lens, sinks, window, budget):
    acc = (torch.randn(2, cap, generator=_gen(cap)) * 2).exp()
    _run_evict(acc, lens, sinks, window, budget, "bf16", 64)


def test_evict_ties_signs_and_specials():
    g = _gen(8)
    few = torch.randint(0, 3, (2, 20000), generator=g).float()               # three values only
    few[1] = -few[1]
    _run_evict(few, [20000, 19999], 2, 10, 5000, "e4m3", 64)
    odd = torch.randn(1, 9000, generator=g)
    odd[0, ::7], odd[0, 1::7], odd[0, 2::7] = math.nan, math.inf, -math.inf
    odd[0, 3::7], odd[0, 4::7] = 0.0, -0.0
    for budget in (10, 1285, 1290, 3000, 4500, 6500, 8990):
        _run_evict(odd, [9000], 0, 3, budget, "bf16", 64, with_acc=budget != 10)
    close = 1.0 + torch.randint(0, 3000, (1, 30000), generator=g).float() * 2.0 ** -23     # the last bits decide
    _run_evict(close, [30000], 1, 1, 12345, "bf16", 64)


def test_evict_clamps_lengths():
    acc = torch.rand(2, 50, generator=_gen(1))
    b, cap, d = 2, 50, 64
    k = torch.randn(b, cap, d, device="cuda").bfloat16()
    ko, vo = torch.zeros(b, 20, d, device="cuda").bfloat16(), torch.zeros(b, 20, d, device="cuda").bfloat16()
    idx, nl = torch.zeros(b, 20, dtype=torch.int32, device="cuda"), torch.zeros(b, dtype=torch.int32, device="cuda")
    desc = hs.make_evict_desc(b, d, hs.HS2_BF16, sinks=1, window=4, budget=15, kv_capacity=cap)
    ln = torch.tensor([-3, 1000], dtype=torch.int32, device="cuda")
    hs.hs2_kv_evict(desc, ln, acc.cuda(), k, k, None, None, ko, vo, None, None, None, idx, nl)
    assert nl.tolist() == [0, 20] and (idx[0] == -1).all()
    assert idx[1].tolist() == ref.evict_rows(acc[1], 50, 1, 4, 15)


# ------------------------------------------------------------------ as they are used
def test_chunks_then_single_tokens_over_an_evicted_cache():
    """Rows written by the rope call, attended with a window, scored, evicted; then a single token on the
    cut cache through the window layer and through the block's full attention."""
    g = _gen(21)
    b, n, h, d, cap = 2, 300, 16, 128, 400
    qkv = torch.randn(b, n, (h + 2) * d, generator=g).bfloat16().cuda()
    freq = (1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    zero = torch.zeros(b, dtype=torch.int32, device="cuda")
    rd = hs.make_rope_desc(b, n, h, d, q_row=(h + 2) * d, k_row=(h + 2) * d, v_row=(h + 2) * d, kv_capacity=cap)
    q = torch.empty(b, n, h, d, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.zeros(b, cap, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    hs.hs2_qk_norm_rope(rd, qkv, qkv[..., h * d:], qkv[..., (h + 1) * d:], None, None, freq, zero, None, None, q, k, v)

    # every row attends to all before it: the log-sum-exp of a window as long as the context
    wd = hs.make_desc(b, n, h, d, window=n, budget=0, kv_capacity=cap, max_ctx=n)
    o, lse = torch.empty_like(q), torch.empty(b, n, h, device="cuda")
    ws = hs.alloc_window_workspace(wd, 0)
    hs.hs2_window_attn(wd, 0, q, k, v, None, None, zero, None, o, lse, ws)
    acc = torch.zeros(b, cap, device="cuda")
    aw = hs.alloc_accum_workspace(wd)
    hs.hs2_weight_accum(wd, q, k, None, lse, zero, None, 1.0, None, acc, aw)
    # each of the n h softmax rows sums to one; lse and weights in fp32
    assert (acc.double().sum(1) - n * h).abs().max().item() < 1e-4 * n * h

    ed = hs.make_evict_desc(b, d, sinks=4, window=64, budget=100, kv_capacity=cap, out_capacity=200)
    ko, vo = (torch.zeros(b, 200, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ao, idx = torch.zeros(b, 200, device="cuda"), torch.zeros(b, 168, dtype=torch.int32, device="cuda")
    ln, nl = torch.full((b,), n, dtype=torch.int32, device="cuda"), torch.zeros(b, dtype=torch.int32, device="cuda")
    hs.hs2_kv_evict(ed, ln, acc, k, v, None, None, ko, vo, None, None, ao, idx, nl)
    assert nl.tolist() == [168, 168]
    for s in range(b):
        assert idx[s].tolist() == ref.evict_rows(acc[s].cpu(), n, 4, 64, 100)
        assert torch.equal(ko[s, :168], k[s, idx[s].long()]) and torch.equal(ao[s, :168], acc[s, idx[s].long()])

    # the next token: position 300, cache row 168
    one = torch.randn(b, 1, (h + 2) * d, generator=g).bfloat16().cuda()
    r1 = hs.make_rope_desc(b, 1, h, d, q_row=(h + 2) * d, k_row=(h + 2) * d, v_row=(h + 2) * d, kv_capacity=200)
    q1, pos = torch.empty(b, 1, h, d, device="cuda", dtype=torch.bfloat16), torch.full((b, 1), n, dtype=torch.int32, device="cuda")
    hs.hs2_qk_norm_rope(r1, one, one[..., h * d:], one[..., (h + 1) * d:], None, None, freq, nl, pos, None, q1, ko, vo)
    d1 = hs.make_desc(b, 1, h, d, window=200, budget=0, kv_capacity=200, max_ctx=200)
    o1, l1 = torch.empty_like(q1), torch.empty(b, 1, h, device="cuda")
    w1 = hs.alloc_window_workspace(d1, 0)
    hs.hs2_window_attn(d1, 0, q1, ko, vo, None, None, nl, None, o1, l1, w1)
    _check_window(q1.cpu(), ko.cpu(), vo.cpu(), None, None, nl.cpu(), None, 200, 0, o1.cpu(), l1.cpu(), "bf16", 0)
    fd = hs.make_desc(b, 1, h, d, window=16, budget=32, kv_capacity=200, max_ctx=200)
    fw = hs.alloc_workspace(fd)
    of, lf = torch.empty_like(q1), torch.empty(b, 1, h, device="cuda")
    si, sc = torch.zeros(b, 1, 48, dtype=torch.int32, device="cuda"), torch.zeros(b, 1, dtype=torch.int32, device="cuda")
    hs.hs2_full_attn_select(fd, q1, ko, vo, None, None, nl, of, lf, si, sc, None, fw)
    assert hs.hs2_last_status(fw) == hs.HS2_OK and hs.hs2_last_status(w1) == hs.HS2_OK
    # both layers saw the same 169 rows: two bf16 results, each within 2^-7 of the weights' sum of |v|
    assert (of.float() - o1.float()).abs().max().item() <= 2 * 2.0 ** -7 * vo.float().abs().max().item()
    assert (lf - l1).abs().max().item() < 1e-4


def test_calls_captured_in_a_graph_and_replayed():
    g = _gen(31)
    b, h, d, ctx = 2, 16, 128, 5000
    q, k, v = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((b, 1, h, d), (b, ctx, d), (b, ctx, d)))
    pos0 = torch.tensor([4999, 3000], dtype=torch.int32, device="cuda")
    desc = hs.make_desc(b, 1, h, d, window=4000, budget=0, max_ctx=ctx)
    ws, aws = hs.alloc_window_workspace(desc, 4), hs.alloc_accum_workspace(desc)
    o, lse, acc = torch.zeros_like(q), torch.zeros(b, 1, h, device="cuda"), torch.zeros(b, ctx, device="cuda")
    ko, vo = torch.zeros(b, 500, d, device="cuda").bfloat16(), torch.zeros(b, 500, d, device="cuda").bfloat16()
    ao, idx = torch.zeros(b, 500, device="cuda"), torch.zeros(b, 500, dtype=torch.int32, device="cuda")
    nl = torch.zeros(b, dtype=torch.int32, device="cuda")
    ln = torch.tensor([5000, 3001], dtype=torch.int32, device="cuda")
    ed = hs.make_evict_desc(b, d, sinks=4, window=96, budget=400, kv_capacity=ctx)

    def step():
        hs.hs2_window_attn(desc, 4, q, k, v, None, None, pos0, None, o, lse, ws)
        hs.hs2_weight_accum(desc, q, k, None, lse, pos0, None, 1.0, None, acc, aws)
        hs.hs2_kv_evict(ed, ln, acc, k, v, None, None, ko, vo, None, None, ao, idx, nl)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    q.copy_(torch.randn(b, 1, h, d, generator=g))
    for t in (o, lse, acc, ko, vo, ao, idx, nl):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (o, lse, acc, ko, vo, ao, idx, nl)]
    step()
    torch.cuda.synchronize()
    for x, y in zip(got, (o, lse, acc, ko, vo, ao, idx, nl)):
        assert torch.equal(x, y)
    _check_window(q.cpu(), k.cpu(), v.cpu(), None, None, pos0.cpu(), None, 4000, 4, o.cpu(), lse.cpu(), "bf16", 0)
