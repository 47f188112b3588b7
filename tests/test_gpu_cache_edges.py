"""GPU tests of the calls around the block where buffers, streams and values meet their limits: outputs
in an input's place, two calls at once, captured calls, NaN and infinities in rows that are in use.

The forms, the checks and their tolerances are those of test_gpu_cache_ops.py."""
import math
import threading

import pytest
import torch

import cache_ops_ref as ref
import kv_shared_b200 as hs
import test_gpu_cache_ops as base

pytestmark = pytest.mark.gpu


def _evict_set(acc, lens, sinks, window, budget, kv, d, seed=0):
    """(description, inputs and outputs of an eviction on the GPU in the call's order)."""
    b, cap = acc.shape
    k, v, ks, vs = base._cache(base._gen(seed), b, cap, d, kv)
    keep = sinks + window + budget
    ko, vo = torch.full((b, keep, d), 7, dtype=k.dtype), torch.full((b, keep, d), 7, dtype=k.dtype)
    sc = [torch.full((b, keep), 5.0) if ks is not None else None for _ in range(2)]
    out = [ko, vo, *sc, torch.full((b, keep), 5.0), torch.full((b, keep), 99, dtype=torch.int32),
           torch.full((b,), 99, dtype=torch.int32)]
    desc = hs.make_evict_desc(b, d, base.KIND[kv], sinks=sinks, window=window, budget=budget, kv_capacity=cap)
    return desc, base._cu(torch.tensor(lens, dtype=torch.int32), acc, k, v, ks, vs), base._cu(*out)


# ------------------------------------------------------------------ eviction: lengths in place
@pytest.mark.parametrize("lens, cap, sinks, window, budget, kv", [
    ([5000, 300, 4000], 5000, 4, 96, 400, "bf16"),                     # one CTA a sequence
    ([60000, 59000, 200, 45000], 60000, 2, 10, 9000, "e4m3"),          # clusters
    ([300000, 299999], 300000, 0, 64, 90000, "e4m3"),                  # teams of all SMs
    ([700000], 700000, 0, 2, 9, "e4m3"),                               # slices that are read again
])
def test_evict_lengths_in_place(lens, cap, sinks, window, budget, kv):
    """new_len in len's place: the rows and lengths of a call with new_len apart, and a second cut of the
    same lengths that finds nothing left to cut."""
    acc = torch.rand(len(lens), cap, generator=base._gen(cap))
    desc, ins, outs = _evict_set(acc, lens, sinks, window, budget, kv, 64)
    hs.hs2_kv_evict(desc, *ins, *outs)
    torch.cuda.synchronize()
    want = [None if t is None else t.clone() for t in outs]
    keep = sinks + window + budget
    assert want[-1].tolist() == [min(n, keep) for n in lens]
    for _ in range(20):
        for t in outs[:-1]:
            if t is not None:
                t.zero_()
        ins[0].copy_(torch.tensor(lens, dtype=torch.int32))
        hs.hs2_kv_evict(desc, *ins, *outs[:-1], ins[0])
        torch.cuda.synchronize()
        assert torch.equal(ins[0], want[-1]) and torch.equal(outs[-2], want[-2])
        for s, m in enumerate(want[-1].tolist()):
            for got, w in zip(outs[:-2], want[:-2]):
                assert got is None or torch.equal(got[s, :m], w[s, :m])
    hs.hs2_kv_evict(desc, *ins, *outs[:-1], ins[0])
    assert ins[0].tolist() == want[-1].tolist()
    for s, m in enumerate(want[-1].tolist()):
        assert outs[-2][s, :m].tolist() == list(range(m)) and (outs[-2][s, m:] == -1).all()


# ------------------------------------------------------------------ two host threads
def _threads(calls, times):
    """Each call `times` times in a thread and on a stream of its own, all at once: the errors."""
    errors, ready = [], threading.Barrier(len(calls))

    def go(call, stream):
        try:
            torch.zeros(1, device="cuda")                      # the device's context is the thread's, too
            ready.wait()
            for _ in range(times):
                call(stream)
        except Exception as e:                                 # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    workers = [threading.Thread(target=go, args=(c, torch.cuda.Stream())) for c in calls]
    for w in workers:
        w.start()
    for w in workers:
        w.join()
    torch.cuda.synchronize()
    return errors


@pytest.mark.parametrize("caps", [(1000, 16000), (20000, 140000)])
def test_evictions_of_two_threads(caps):
    """Selections whose shared memory differs, from two threads: each call is valid and is made."""
    sets = [_evict_set(torch.rand(1, cap, generator=base._gen(cap)), [cap], 1, 9, 100, "e4m3", 64) for cap in caps]
    for desc, ins, outs in sets:
        hs.hs2_kv_evict(desc, *ins, *outs)
    torch.cuda.synchronize()
    want = [[None if t is None else t.clone() for t in outs] for _, _, outs in sets]
    calls = [lambda st, s=s: hs.hs2_kv_evict(s[0], *s[1], *s[2], stream=st) for s in sets]
    assert _threads(calls, 2000) == []
    for (_, _, outs), ws in zip(sets, want):
        assert all(t is None or torch.equal(t, w) for t, w in zip(outs, ws))


def test_weight_calls_of_two_threads():
    """16 and 64 pairs a sequence take query slots of different size in the same kernel."""
    g = base._gen(12)
    d, ctx, sets = 128, 600, []
    k = torch.randn(1, ctx, d, generator=g).bfloat16().cuda()
    for n in (1, 4):
        q = torch.randn(1, n, 16, d, generator=g).bfloat16().cuda()
        desc = hs.make_desc(1, n, 16, d, max_ctx=ctx)
        sets.append((desc, q, k, None, torch.full((1, n, 16), 5.0, device="cuda"),
                     torch.tensor([ctx - n], dtype=torch.int32, device="cuda"), None, 1.0, None,
                     torch.zeros(1, ctx, device="cuda"), hs.alloc_accum_workspace(desc)))
    for s in sets:
        hs.hs2_weight_accum(*s)
    torch.cuda.synchronize()
    want = [s[-2].clone() for s in sets]
    calls = [lambda st, s=s: hs.hs2_weight_accum(*s, stream=st) for s in sets]
    assert _threads(calls, 3000) == []
    assert all(torch.equal(s[-2], w) for s, w in zip(sets, want))


def _fresh_thread(call):
    """A call made in a thread that has not used the device: its error, or None."""
    errors = []

    def go():
        try:
            call()
        except Exception as e:                                 # noqa: BLE001
            errors.append(e)

    stream = torch.cuda.current_stream()
    assert stream.cuda_stream is not None
    torch.cuda.synchronize()
    t = threading.Thread(target=go)
    t.start()
    t.join()
    torch.cuda.synchronize()
    return errors[0] if errors else None


@pytest.mark.parametrize("n", [1, 20, 600])
def test_calls_from_a_thread_that_has_not_used_the_device(n):
    """Every call that describes its tiles to the copy engine, as a thread's first: the bits of the main
    thread's call."""
    g = base._gen(n)
    b, h, d, ctx = 1, 16, 128, 2000
    q, k, v = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((b, n, h, d), (b, ctx, d), (b, ctx, d)))
    pos0 = torch.full((b,), ctx - n, dtype=torch.int32, device="cuda")
    st = torch.cuda.current_stream()
    desc = hs.make_desc(b, n, h, d, window=128, budget=256, max_ctx=ctx)
    ws = [hs.alloc_window_workspace(desc, 2), hs.alloc_accum_workspace(desc), hs.alloc_workspace(desc)]
    o, lse, acc = torch.empty_like(q), torch.empty(b, n, h, device="cuda"), torch.zeros(b, ctx, device="cuda")
    idx, cnt = torch.empty(b, n, 384, dtype=torch.int32, device="cuda"), torch.empty(b, n, dtype=torch.int32, device="cuda")
    x, w = torch.randn(b, n, 256, generator=g).bfloat16().cuda(), torch.randn(256, 256, generator=g).bfloat16().cuda()
    kb, vb = torch.zeros_like(k), torch.zeros_like(v)
    calls = {
        "window": (lambda: hs.hs2_window_attn(desc, 2, q, k, v, None, None, pos0, None, o, lse, ws[0], stream=st), (o, lse)),
        "accum": (lambda: hs.hs2_weight_accum(desc, q, k, None, lse, pos0, None, 1.0, None, acc, ws[1], stream=st), (acc,)),
        "full": (lambda: hs.hs2_full_attn_select(desc, q, k, v, None, None, pos0, o, lse, idx, cnt, None, ws[2], stream=st),
                 (o, lse, idx, cnt)),
        "sparse": (lambda: hs.hs2_sparse_attn(desc, q, k, v, None, None, idx, cnt, o, lse, ws[2], stream=st), (o, lse)),
        "bridge": (lambda: hs.hs2_kv_bridge_proj(x, w, b, n, 256, d, pos0, ctx, kb, vb, stream=st), (kb, vb)),
    }
    for name, (call, outs) in calls.items():
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        error = _fresh_thread(call)
        assert error is None, (name, error)
        assert all(torch.equal(t, x0) for t, x0 in zip(outs, want)), name


# ------------------------------------------------------------------ rotation in place
@pytest.mark.parametrize("b, n, h, d, rot, inter, dt", [
    (2, 3, 16, 128, 128, False, "bf16"), (1, 700, 16, 128, 128, False, "bf16"), (2, 400, 5, 64, 48, False, "f32"),
    (1, 650, 128, 64, 32, True, "bf16"), (3, 250, 7, 128, 96, False, "bf16"), (1, 5, 3, 64, 64, True, "f32"),
    (1, 601, 9, 128, 128, False, "f32"),
])
def test_rope_in_place_gives_the_bits_of_a_call_apart(b, n, h, d, rot, inter, dt):
    g = base._gen(n + h)
    q = torch.randn(b, n, h, d, generator=g).to(base.DT[dt]).cuda()
    w = (1 + 0.2 * torch.randn(d, generator=g)).cuda()
    freq = (1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).cuda()
    row0 = torch.arange(b, dtype=torch.int32, device="cuda")
    desc = hs.make_rope_desc(b, n, h, d, rot_dim=rot, interleaved=inter, in_dtype=base.KIND[dt], kv_dtype=base.KIND[dt],
                             kv_capacity=n)
    out = torch.empty_like(q)
    hs.hs2_qk_norm_rope(desc, q, None, None, w, None, freq, row0, None, None, out, None, None)
    for _ in range(3):
        x = q.clone()
        hs.hs2_qk_norm_rope(desc, x, None, None, w, None, freq, row0, None, None, x, None, None)
        assert torch.equal(x, out)


# ------------------------------------------------------------------ weights: NaN and infinities in use
ACCUM_FORMS = [  # rows, heads, kv: wide and narrow tiles of pairs, fp32
    (16, 16, "bf16"), (16, 16, "e4m3"), (4, 16, "bf16"), (4, 16, "e4m3"), (9, 8, "f32"), (2, 5, "f32"), (60, 5, "bf16"),
]


def _accum_case(n, h, kv, ctx=700, d=128):
    """(q, k, ks, lse, pos0, kk, logits): a prompt's last n rows, logits [n, h, ctx] in fp64, hidden ones -inf."""
    g = base._gen(n * h)
    q = torch.randn(1, n, h, d, generator=g).to(base.DT["f32" if kv == "f32" else "bf16"])
    k, _, ks, _ = base._cache(g, 1, ctx, d, kv)
    kk = ref.wide(k[0], None if ks is None else ks[0])
    x = torch.einsum("rhd,kd->rhk", q[0].double(), kk) * d ** -0.5
    hide = torch.arange(ctx) > ctx - n + torch.arange(n)[:, None]
    x = x.masked_fill(hide[:, None], -math.inf)
    return q, k, ks, x.logsumexp(-1).float()[None], torch.tensor([ctx - n], dtype=torch.int32), x


def _accum_of(q, k, ks, lse, pos0, kv):
    n, h, d = q.shape[1:]
    desc = hs.make_desc(1, n, h, d, q_dtype=base.KIND["f32" if kv == "f32" else "bf16"], kv_dtype=base.KIND[kv],
                        max_ctx=k.shape[1])
    ws, out = hs.alloc_accum_workspace(desc), torch.full((1, k.shape[1]), -3.0, device="cuda")
    hs.hs2_weight_accum(desc, *base._cu(q, k, ks, lse, pos0, None), 1.0, None, out, ws)
    assert hs.hs2_last_status(ws) == hs.HS2_OK
    return out[0].cpu()


@pytest.mark.parametrize("n, h, kv", ACCUM_FORMS)
@pytest.mark.parametrize("where", ["query", "lse"])
def test_accum_keeps_a_nan(n, h, kv, where):
    """A NaN in a pair's query or lse is in the total of every key that the pair sees, whichever pair it is."""
    q, k, ks, lse, pos0, _ = _accum_case(n, h, kv)
    base_out = _accum_of(q, k, ks, lse, pos0, kv)
    assert base_out.isfinite().all()
    for f in sorted({*range(min(n * h, 40)), n * h // 2, n * h - 1}):
        q2, l2 = q.clone(), lse.clone()
        if where == "query":
            q2[0, f // h, f % h, 3] = math.nan
        else:
            l2[0, f // h, f % h] = math.nan
        got, p = _accum_of(q2, k, ks, l2, pos0, kv), int(pos0[0]) + f // h
        assert got[:p + 1].isnan().all() and torch.equal(got[p + 1:], base_out[p + 1:]), f


@pytest.mark.parametrize("n, h, kv", ACCUM_FORMS)
def test_accum_of_an_lse_that_leaves_keys_out(n, h, kv):
    """An lse far below a pair's logits (of a layer whose rows leave keys out, say): weights up to 2^100
    are numbers, those past fp32's range infinite; an infinite lse makes them zero."""
    q, k, ks, lse, pos0, x = _accum_case(n, h, kv)
    ends = torch.arange(x.shape[2])
    for f in sorted({*range(min(n * h, 36)), n * h - 1}):
        r, p = f // h, int(pos0[0]) + f // h
        for shift, want in ((100.0, None), (140.0, math.inf), (400.0, math.inf)):
            l2 = lse.clone()
            l2[0, r, f % h] = x[r, f % h, :p + 1].min() - shift * math.log(2.0)
            if shift == 100.0:                              # weights of one pair from 2^100 up
                l2[0, r, f % h] = x[r, f % h, :p + 1].max() - shift * math.log(2.0)
            got = _accum_of(q, k, ks, l2, pos0, kv)[:p + 1].double()
            if want is not None:
                assert (got == want).all(), (f, shift)
                continue
            ref_w = (x[r, f % h, :p + 1] - l2[0, r, f % h].double()).exp()
            # the other pairs' weights, each at most one, are below 2^-60 of it; the exponent's own
            # rounding 2^-24 of |logit| + |lse| (below 2^8) in log2 units, the products' 2 d 2^-24 of 2^6
            rel = (2 * 128 * 64 + 8 * 256) * 2.0 ** -24
            assert ((got - ref_w).abs() <= rel * ref_w + n * h).all(), f
        l2 = torch.full_like(lse, math.inf)
        assert (_accum_of(q, k, ks, l2, pos0, kv)[ends < int(pos0[0]) + n] == 0).all()


@pytest.mark.parametrize("n", [4, 16])
@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_accum_of_an_infinite_query(n, bad):
    """Next to e4m3 keys a query goes in as finite codes: a row with an infinity gives NaN, not numbers."""
    q, k, ks, lse, pos0, _ = _accum_case(n, 16, "e4m3")
    clean = _accum_of(q, k, ks, lse, pos0, "e4m3")
    for f in (0, 5, 33, n * 16 - 1):
        q2 = q.clone()
        q2[0, f // 16, f % 16, 100] = bad
        got, p = _accum_of(q2, k, ks, lse, pos0, "e4m3"), int(pos0[0]) + f // 16
        assert got[:p + 1].isnan().all() and torch.equal(got[p + 1:], clean[p + 1:]), f


# ------------------------------------------------------------------ rotation: infinities
@pytest.mark.parametrize("rot, inter", [(0, False), (0, True), (32, False), (32, True), (96, False), (96, True), (128, False)])
@pytest.mark.parametrize("dt, kv", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("normalize", [False, True])
def test_rope_keeps_an_infinity_in_its_place(rot, inter, dt, kv, normalize):
    """An infinity or NaN in a dim that does not turn stays in that dim (without a norm); in a pair that
    turns it reaches the pair's other dim and no further."""
    g = base._gen(rot)
    n, h, d = 6, 3, 128
    q0, k0 = (torch.randn(1, n, x, d, generator=g).to(base.DT[dt]) for x in (h, 1))
    bad = [(0, 127, math.inf), (1, 100, -math.inf), (2, 5, math.inf), (3, 64, math.nan), (4, 31, math.inf)]
    for r, i, x in bad:
        q0[0, r, r % h, i] = x
        k0[0, r, 0, i] = x
    freq = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    row0 = torch.tensor([11], dtype=torch.int32)
    q, k, fr, r0 = base._cu(q0, k0, freq, row0)
    out, kc = torch.empty_like(q), torch.zeros(1, 32, d, dtype=base.DT[kv], device="cuda")
    desc = hs.make_rope_desc(1, n, h, d, rot_dim=rot, interleaved=inter, normalize=normalize, in_dtype=base.KIND[dt],
                             kv_dtype=base.KIND[kv], kv_capacity=32)
    hs.hs2_qk_norm_rope(desc, q, k, None, None, None, fr if rot else None, r0, None, None, out, kc, None)
    torch.cuda.synchronize()
    for got, src in ((out[0].cpu().double(), q0[0]), (kc[0, 11:11 + n, None].cpu().double(), k0[0])):
        want = ref.norm_rope(src, None, 1e-6, [11 + t for t in range(n)], freq, inter, normalize=normalize)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
        assert torch.equal(got[got.isinf()], want[want.isinf()])
        ok = want.isfinite()
        top = torch.where(ok, want.abs(), torch.zeros_like(want)).amax(-1, keepdim=True)
        half = base.HALF_BF16 if dt == "bf16" else 0.0
        assert ((got - want).abs() <= half * want.abs() + 2.0 ** -18 * top)[ok].all()


# ------------------------------------------------------------------ sliding window: NaN queries
@pytest.mark.parametrize("n, window, kv", [
    (1, 100, "bf16"), (1, 100, "e4m3"), (1, 2000, "bf16"), (1, 2000, "e4m3"), (20, 100, "bf16"), (20, 1800, "e4m3"),
    (600, 100, "bf16"), (300, 1800, "bf16"), (600, 100, "e4m3"), (300, 1800, "e4m3"), (1, 100, "f32"), (1, 2000, "f32"),
    (40, 300, "f32"), (700, 100, "f32"),
])
def test_window_keeps_a_nan_query(n, window, kv):
    """A NaN in a row's query is in that row's output and lse and in no other's."""
    g = base._gen(n + window)
    b, h, d, ctx = 2, 16, 128, 2500
    dt = base.DT["f32" if kv == "f32" else "bf16"]
    q = torch.randn(b, n, h, d, generator=g).to(dt)
    k, v, ks, vs = base._cache(g, b, ctx, d, kv)
    pos0 = torch.tensor([ctx - n, min(1900, ctx - n)], dtype=torch.int32)
    bad = n // 2
    q[0, bad, :, 7] = math.nan
    dev = base._cu(q, k, v, ks, vs, pos0, None)
    o, lse = torch.zeros_like(dev[0]), torch.zeros(b, n, h, device="cuda")
    desc = hs.make_desc(b, n, h, d, window=window, budget=0, q_dtype=base.KIND["f32" if kv == "f32" else "bf16"],
                        kv_dtype=base.KIND[kv], max_ctx=ctx)
    ws = hs.alloc_window_workspace(desc, 3)
    hs.hs2_window_attn(desc, 3, *dev, o, lse, ws)
    assert hs.hs2_last_status(ws) == hs.HS2_OK
    assert o[0, bad].isnan().all() and lse[0, bad].isnan().all()
    assert int(o.isnan().sum()) == h * d and int(lse.isnan().sum()) == h
    near = [r for r in (0, bad - 1, bad + 1, n - 1) if 0 <= r < n]
    for s in range(b):
        rows = [r for r in near if s or r != bad]
        base._check_window(q[s:s + 1], k[s:s + 1], v[s:s + 1], None if ks is None else ks[s:s + 1],
                           None if vs is None else vs[s:s + 1], pos0[s:s + 1], None, window, 3, o[s:s + 1].cpu(),
                           lse[s:s + 1].cpu(), kv, 0, rows=rows)


# ------------------------------------------------------------------ bounds of padded batches
@pytest.mark.parametrize("n, kv", [(1, "bf16"), (3, "e4m3"), (40, "bf16"), (700, "bf16"), (700, "e4m3"), (5, "f32"), (90, "f32")])
def test_row_counts_outside_the_batch_are_clamped(n, kv):
    """n_rows below 0 and above n: the bits of calls with 0 and n."""
    g = base._gen(n)
    b, h, d, ctx = 3, 16, 128, 1500
    dt = base.DT["f32" if kv == "f32" else "bf16"]
    qd = base.KIND["f32" if kv == "f32" else "bf16"]
    q, k0, v0 = (torch.randn(b, n, x, d, generator=g).to(dt).cuda() for x in (h, 1, 1))
    k, v, ks, vs = base._cu(*base._cache(g, b, ctx, d, kv))
    pos0 = torch.tensor([ctx - n, 100, 3], dtype=torch.int32, device="cuda")
    freq = (1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    lse0 = torch.full((b, n, h), 4.0, device="cuda")
    rd = hs.make_rope_desc(b, n, h, d, in_dtype=qd, kv_dtype=base.KIND[kv], kv_capacity=ctx)
    desc = hs.make_desc(b, n, h, d, window=200, budget=0, q_dtype=qd, kv_dtype=base.KIND[kv], max_ctx=ctx)
    ws, aws = hs.alloc_window_workspace(desc, 3), hs.alloc_accum_workspace(desc)

    def run(counts):
        rows = torch.tensor(counts, dtype=torch.int32, device="cuda")
        out = dict(q=torch.full_like(q, 7.0), kc=torch.zeros_like(k), vc=torch.zeros_like(v),
                   ks=None if ks is None else torch.zeros_like(ks), vs=None if vs is None else torch.zeros_like(vs),
                   o=torch.full_like(q, 7.0), lse=torch.full_like(lse0, 7.0), acc=torch.full((b, ctx), 7.0, device="cuda"))
        hs.hs2_qk_norm_rope(rd, q, k0, v0, None, None, freq, pos0, None, rows, out["q"], out["kc"], out["vc"], out["ks"],
                            out["vs"])
        hs.hs2_window_attn(desc, 3, q, k, v, ks, vs, pos0, rows, out["o"], out["lse"], ws)
        hs.hs2_weight_accum(desc, q, k, ks, lse0, pos0, rows, 1.0, None, out["acc"], aws)
        assert hs.hs2_last_status(ws) == hs.HS2_OK and hs.hs2_last_status(aws) == hs.HS2_OK
        return out

    for counts, clamped in (([-3, n + 5, n], [0, n, n]), ([-(1 << 31), (1 << 31) - 1, -1], [0, n, 0])):
        want, got = run(clamped), run(counts)
        for key, t in want.items():
            assert t is None or torch.equal(t, got[key]), (key, counts)


@pytest.mark.parametrize("n, window, ctx, ragged", [(1, 100, 900, False), (1, 3000, 5000, False), (20, 60, 900, True),
                                                    (600, 100, 1300, False), (300, 33, 800, True)])
def test_scales_of_rows_out_of_use_may_be_nan(n, window, ctx, ragged):
    """e4m3 rows that no query attends to: codes and scales hold NaN; results as with numbers there."""
    g = base._gen(n + ctx)
    b, h, d, sinks = 4, 16, 128, 5
    q = torch.randn(b, n, h, d, generator=g).to(torch.bfloat16)
    k, v, ks, vs = base._cache(g, b, ctx, d, "e4m3")
    pos0 = torch.tensor([ctx - n, 0, 300 % (ctx - n + 1), 57 % (ctx - n + 1)], dtype=torch.int32)
    counts = [n, 0, n // 2, 1] if ragged else [n] * b
    rows = torch.tensor(counts, dtype=torch.int32) if ragged else None
    seen, past = torch.zeros(b, ctx, dtype=torch.bool), torch.zeros(b, ctx, dtype=torch.bool)
    for s, m in enumerate(counts):
        past[s, int(pos0[s]) + m:] = True
        if m:
            seen[s, max(0, int(pos0[s]) - window + 1):int(pos0[s]) + m] = True
            seen[s, :min(sinks, int(pos0[s]) + m)] = True
    desc = hs.make_desc(b, n, h, d, window=window, budget=0, kv_dtype=hs.HS2_E4M3, max_ctx=ctx)
    ws, aws = hs.alloc_window_workspace(desc, sinks), hs.alloc_accum_workspace(desc)
    lse_in = torch.full((b, n, h), 5.0)
    got = []
    for mask_w, mask_a in ((~seen, past), (torch.zeros_like(seen), torch.zeros_like(past))):
        kw, vw, ka = (base._poison(t, m) for t, m in ((k, mask_w), (v, mask_w), (k, mask_a)))
        sw, tw, sa = (torch.where(m, torch.full_like(t, math.nan), t) for t, m in ((ks, mask_w), (vs, mask_w), (ks, mask_a)))
        o, lse = torch.full((b, n, h, d), 7.0, device="cuda").bfloat16(), torch.full((b, n, h), 7.0, device="cuda")
        acc = torch.full((b, ctx), 7.0, device="cuda")
        hs.hs2_window_attn(desc, sinks, *base._cu(q, kw, vw, sw, tw, pos0, rows), o, lse, ws)
        hs.hs2_weight_accum(desc, *base._cu(q, ka, sa, lse_in, pos0, rows), 1.0, None, acc, aws)
        assert hs.hs2_last_status(ws) == hs.HS2_OK and hs.hs2_last_status(aws) == hs.HS2_OK
        got.append((o, lse, acc))
    for x, y in zip(*got):
        assert x.isfinite().all() and torch.equal(x, y)


# ------------------------------------------------------------------ eviction by teams of all SMs
def test_evict_by_teams_in_a_graph_and_beside_another_stream():
    """The grid-wide selection captured and replayed on other lengths and totals, and run while another
    stream works: the bits of the call made alone."""
    g = base._gen(77)
    cap, lens = 300000, [300000, 150001]
    desc, ins, outs = _evict_set(torch.rand(2, cap, generator=g), lens, 3, 64, 60000, "e4m3", 64)

    def alone():
        hs.hs2_kv_evict(desc, *ins, *outs)
        torch.cuda.synchronize()
        return [t.clone() for t in outs]

    first = alone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hs2_kv_evict(desc, *ins, *outs)
    ins[1].copy_(torch.rand(2, cap, generator=g))
    ins[0].copy_(torch.tensor([299001, 60000], dtype=torch.int32))
    want = alone()
    assert not torch.equal(first[-2], want[-2])
    for _ in range(3):
        for t in outs:
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        for s, m in enumerate(want[-1].tolist()):
            assert all(torch.equal(t[s, :m], w[s, :m]) for t, w in zip(outs[:-1], want[:-1]))
        assert torch.equal(outs[-1], want[-1]) and torch.equal(outs[-2], want[-2])
    # beside weight calls and evictions of another form on a second stream
    q, kb = torch.randn(2, 8, 16, 128, generator=g).bfloat16().cuda(), torch.randn(2, 20000, 128, generator=g).bfloat16().cuda()
    ad = hs.make_desc(2, 8, 16, 128, max_ctx=20000)
    a_in = (q, kb, None, torch.full((2, 8, 16), 9.0, device="cuda"), torch.full((2,), 19992, dtype=torch.int32, device="cuda"), None)
    acc, aws = torch.zeros(2, 20000, device="cuda"), hs.alloc_accum_workspace(ad)
    small = _evict_set(torch.rand(3, 9000, generator=g), [9000, 8000, 7], 1, 5, 700, "bf16", 64)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for t in outs:
        t.fill_(9)
    torch.cuda.synchronize()
    for _ in range(20):
        hs.hs2_kv_evict(desc, *ins, *outs, stream=streams[0])
        hs.hs2_weight_accum(ad, *a_in, 1.0, None, acc, aws, stream=streams[1])
        hs.hs2_kv_evict(small[0], *small[1], *small[2], stream=streams[1])
    torch.cuda.synchronize()
    for s, m in enumerate(want[-1].tolist()):
        assert all(torch.equal(t[s, :m], w[s, :m]) for t, w in zip(outs[:-1], want[:-1]))
    beside = [acc.clone(), *[None if t is None else t.clone() for t in small[2]]]
    hs.hs2_weight_accum(ad, *a_in, 1.0, None, acc, aws)
    hs.hs2_kv_evict(small[0], *small[1], *small[2])
    for x, y in zip(beside, [acc, *small[2]]):
        assert x is None or torch.equal(x, y)
