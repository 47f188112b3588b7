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
