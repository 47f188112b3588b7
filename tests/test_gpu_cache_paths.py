"""GPU tests of the kernels behind the calls around the block at the sizes where one gives way to
another: key lists cut over CTAs, narrow and wide weight items, clusters and teams of the
eviction, rows shared by warps; values of very different magnitude; other streams.

The forms, the checks and their tolerances are those of test_gpu_cache_ops.py."""
import math

import pytest
import torch

import cache_ops_ref as ref
import kv_shared_b200 as hs
import test_gpu_cache_ops as base

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rows for the cache
@pytest.mark.parametrize("b, n, h, d, rot, inter, dt, kv", [
    (2, 330, 5, 128, 96, False, "bf16", "e4m3"), (1, 700, 3, 64, 32, True, "f32", "f32"),
    (3, 250, 7, 64, 64, False, "bf16", "bf16"), (1, 640, 1, 128, 0, False, "f32", "e4m3"),
    (2, 301, 24, 64, 48, False, "f32", "bf16"), (1, 601, 2, 128, 128, True, "bf16", "bf16"),
])
def test_rope_a_warp_to_a_row(b, n, h, d, rot, inter, dt, kv):
    """Enough rows that each has one warp (fewer share a row between warps, as in the base tests)."""
    base.test_rope_rows(b, n, h, d, rot, inter, dt, kv, True)


def test_rope_positions_follow_rows_past_32_bits():
    """Without positions the position is the cache row, also where the rows lie behind any cache: the
    queries turn by it, the key is not written."""
    n, h, d = 6, 3, 64
    g = base._gen(31)
    q0, k0 = torch.randn(1, n, h, d, generator=g), torch.randn(1, n, d, generator=g)
    freq = 1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    row0 = torch.tensor([(1 << 31) - 3], dtype=torch.int32)
    q, k, fr, r0 = base._cu(q0, k0, freq, row0)
    out, kc = torch.empty_like(q), torch.full((1, 8, d), 7.0, device="cuda")
    desc = hs.make_rope_desc(1, n, h, d, normalize=False, in_dtype=hs.HS2_F32, kv_dtype=hs.HS2_F32, kv_capacity=8)
    hs.hs2_qk_norm_rope(desc, q, k, None, None, None, fr, r0, None, None, out, kc, None)
    torch.cuda.synchronize()
    want = ref.norm_rope(q0[0], None, 0.0, [int(row0[0]) + t for t in range(n)], freq, False, normalize=False)
    assert (out[0].cpu().double() - want).abs().le(2.0 ** -18 * want.abs().amax(-1, keepdim=True)).all()
    assert (kc == 7).all()


# ------------------------------------------------------------------ sliding window
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("b, n, h, d, window, sinks, ctx", [
    (1, 20, 16, 128, 3000, 4, 4000),       # few pairs, many keys: the keys are cut
    (4, 33, 8, 64, 1500, 200, 2000),       # with a padded batch: parts without keys, sinks of over a tile
    (1, 16, 16, 128, 128, 16, 300), (2, 17, 16, 128, 112, 15, 300),
    (1, 24, 16, 64, 50, 120, 500),         # sinks longer than the window
    (3, 26, 5, 128, 7, 1, 200),
    (1, 9, 128, 128, 1, 0, 40),            # a window of the row itself
])
def test_window_small_calls(kv, b, n, h, d, window, sinks, ctx):
    base._run_window(base._gen(n + ctx), b, n, h, d, window, sinks, ctx, kv, ragged=b == 4)


# calls large enough for the tcgen05 kernel
LARGE = [
    # b, n, h, d, window, sinks, ctx
    (1, 512, 16, 128, 128, 4, 900), (3, 340, 8, 64, 33, 130, 700), (2, 8200, 1, 64, 1, 0, 8300),
    (2, 900, 5, 128, 64, 16, 1300), (1, 90, 128, 128, 30, 3, 200), (1, 520, 16, 64, 50, 120, 600),
    (1, 257, 16, 128, 3000, 4, 4000),      # keys cut
    (4, 80, 16, 128, 2500, 20, 4000),      # keys cut, a padded batch: sequences of no rows, parts of no keys
    (4, 300, 16, 64, 100, 15, 1000), (1, 600, 16, 128, 1 << 30, 7, 600), (2, 400, 12, 128, 112, 16, 500),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("b, n, h, d, window, sinks, ctx", LARGE)
def test_window_large_calls(kv, b, n, h, d, window, sinks, ctx):
    rows = sorted({0, 1, 2, 7, 8, 15, 16, 17, 31, 32, 50, 51, 52, n // 2 - 1, n // 2, n - 17, n - 2, n - 1})
    base._run_window(base._gen(n + ctx), b, n, h, d, window, sinks, ctx, kv, ragged=b == 4, rows=rows)


@pytest.mark.parametrize("b, n, h, d, window, sinks, ctx", [
    (2, 700, 8, 64, 100, 4, 900), (1, 340, 16, 128, 2000, 5, 3000),        # a CTA and more on every SM
    (1, 90, 16, 128, 1500, 40, 2000), (4, 30, 8, 64, 31, 33, 200),         # keys cut over the CTAs; a padded batch
    (1, 1, 3, 64, 4000, 0, 5000), (1, 7, 1, 128, 64, 1, 64),               # parts of a tile of keys each
])
def test_window_f32_calls(b, n, h, d, window, sinks, ctx):
    rows = sorted({0, 1, 2, 3, 4, 31, 32, n // 2, max(n - 2, 0), n - 1})
    base._run_window(base._gen(n + ctx), b, n, h, d, window, sinks, ctx, "f32", ragged=b == 4, rows=rows)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_window_large_call_with_rising_logits(kv):
    """Logits of several hundred that rise along the keys, so that the reference moves at every tile."""
    g = base._gen(9)
    b, n, h, d, ctx = 1, 600, 16, 128, 1400
    q = (torch.randn(b, n, h, d, generator=g) * 16).to(torch.bfloat16)
    k = torch.randn(b, ctx, d, generator=g) * 4
    k = k[:, torch.argsort(k[0] @ q[0, 0, 0].float())]
    v = torch.randn(b, ctx, d, generator=g) + 1e4
    (k, ks), (v, vs) = (ref.quantize(k), ref.quantize(v)) if kv == "e4m3" else ((k.bfloat16(), None), (v.bfloat16(), None))
    pos0 = torch.tensor([ctx - n], dtype=torch.int32)
    dev = base._cu(q, k, v, ks, vs, pos0, None)
    o, lse = torch.zeros_like(dev[0]), torch.zeros(b, n, h, device="cuda")
    desc = hs.make_desc(b, n, h, d, window=900, budget=0, kv_dtype=base.KIND[kv], max_ctx=ctx)
    ws = hs.alloc_window_workspace(desc, 2)
    hs.hs2_window_attn(desc, 2, *dev, o, lse, ws)
    assert hs.hs2_last_status(ws) == hs.HS2_OK
    base._check_window(q, k, v, ks, vs, pos0, None, 900, 2, o.cpu(), lse.cpu(), kv, 0, rows=[0, 1, 100, 333, 598, 599])


def test_window_large_call_reports_positions_outside_the_context():
    desc = hs.make_desc(2, 600, 16, 128, window=128, budget=0, max_ctx=700)
    ws = hs.alloc_window_workspace(desc, 1)
    q = torch.randn(2, 600, 16, 128, device="cuda").bfloat16()
    kv = torch.randn(2, 700, 128, device="cuda").bfloat16()
    o = torch.zeros_like(q)
    for bad in ([-1, 0], [0, 101]):
        pos0 = torch.tensor(bad, dtype=torch.int32, device="cuda")
        hs.hs2_window_attn(desc, 1, q, kv, kv, None, None, pos0, None, o, None, ws)
        assert hs.hs2_last_status(ws) == hs.HS2_ERR_INDEX
    assert hs.hs2_last_status(ws) == hs.HS2_OK


@pytest.mark.parametrize("n", [1, 20, 600])
@pytest.mark.parametrize("size", [1e-5, 1.0, 300.0])
def test_window_e4m3_scales_of_many_magnitudes(n, size):
    """Values whose rows differ by factors of thousands, queries far from one.  An output's error
    is within 2^-8 of its weights' sum of |v|, whatever the rows' magnitudes."""
    g = base._gen(n)
    b, h, d, ctx, window = 2, 16, 128, 1300, 600
    q = (torch.randn(b, n, h, d, generator=g) * size).to(torch.bfloat16)
    k = torch.randn(b, ctx, d, generator=g) / size
    v = torch.randn(b, ctx, d, generator=g) * torch.exp2(torch.randint(-14, 15, (b, ctx, 1), generator=g).float())
    (k, ks), (v, vs) = ref.quantize(k), ref.quantize(v)
    pos0 = torch.tensor([ctx - n, 650 - n], dtype=torch.int32)
    dev = base._cu(q, k, v, ks, vs, pos0, None)
    o, lse = torch.zeros_like(dev[0]), torch.zeros(b, n, h, device="cuda")
    desc = hs.make_desc(b, n, h, d, window=window, budget=0, kv_dtype=hs.HS2_E4M3, max_ctx=ctx)
    ws = hs.alloc_window_workspace(desc, 3)
    hs.hs2_window_attn(desc, 3, *dev, o, lse, ws)
    assert hs.hs2_last_status(ws) == hs.HS2_OK
    base._check_window(q, k, v, ks, vs, pos0, None, window, 3, o.cpu(), lse.cpu(), "e4m3", 0, rows=[0, 1, 19, 300, 599])


# ------------------------------------------------------------------ accumulated weight
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("b, n, h, d, ctx", [
    (1, 4, 16, 128, 600), (1, 5, 13, 128, 600),                # 64 and 65 pairs: one narrow tile, a wide one
    (2, 1, 128, 64, 300), (1, 90, 16, 64, 90),                 # a prompt that scores itself: keys seen by some rows only
    (4, 60, 16, 128, 200),                                     # pairs cut over CTAs, a padded batch
    (1, 3, 1, 128, 1300), (1, 200, 3, 64, 1100),
])
def test_accum_narrow_wide_and_cut(kv, b, n, h, d, ctx):
    base._run_accum(base._gen(n + ctx), b, n, h, d, ctx, kv, 0.5, ragged=b == 4)


def test_accum_many_items_per_cta():
    """More key blocks than SMs; totals against the plain form computed on the GPU in fp64."""
    g = base._gen(3)
    b, h, d = 2, 16, 128
    for n, kv in ((1, "e4m3"), (1, "bf16"), (12, "bf16"), (12, "e4m3")):
        ctx = 90001
        q = torch.randn(b, n, h, d, generator=g).to(torch.bfloat16).cuda()
        k, _, ks, _ = base._cache(g, b, ctx, d, kv)
        kk = ref.wide(k, ks).cuda()
        pos0 = torch.tensor([ctx - n, 70000], dtype=torch.int32, device="cuda")
        x = torch.einsum("brhd,bkd->brhk", q.double(), kk) * d ** -0.5
        hide = torch.arange(ctx, device="cuda") > (pos0[:, None] + torch.arange(n, device="cuda"))[..., None]
        x = x.masked_fill(hide[:, :, None], -math.inf)
        lse = x.logsumexp(-1).float()
        want = (x - lse.double()[..., None]).exp().sum((1, 2))
        acc = torch.full((b, ctx), 7.0, device="cuda")
        desc = hs.make_desc(b, n, h, d, kv_dtype=base.KIND[kv], max_ctx=ctx)
        ws = hs.alloc_accum_workspace(desc)
        hs.hs2_weight_accum(desc, q, k.cuda(), None if ks is None else ks.cuda(), lse, pos0, None, 1.0, None, acc, ws)
        assert hs.hs2_last_status(ws) == hs.HS2_OK
        for s in range(b):
            end = int(pos0[s]) + n
            # logits up to 7: 2 d 2^-24 of the products' magnitudes (below 2^5) and the exponent's rounding
            rel = (2 * d * 32 + 8 * 64) * 2.0 ** -24
            assert (acc[s, :end].double() - want[s, :end]).abs().le(rel * want[s, :end] + 1e-30).all()
            assert (acc[s, end:] == 7).all()


@pytest.mark.parametrize("size", [1e-4, 1.0, 1e3])
def test_accum_e4m3_queries_of_many_magnitudes(size):
    """The query goes in as two e4m3 numbers per element: dims that differ by 2^10 stay exact."""
    g = base._gen(17)
    b, n, h, d, ctx = 1, 6, 16, 128, 500
    q = (torch.randn(b, n, h, d, generator=g) * size * torch.exp2(-torch.randint(0, 9, (d,), generator=g).float())).to(torch.bfloat16)
    k = torch.randn(b, ctx, d, generator=g) / size
    k, ks = ref.quantize(k)
    pos0 = torch.tensor([ctx - n], dtype=torch.int32)
    kk = ref.wide(k[0], ks[0])
    lse = torch.stack([((q[0, r].double() @ kk[:ctx - n + r + 1].T) * d ** -0.5).logsumexp(-1) for r in range(n)]).float()[None]
    want, mag = ref.weight_total(q[0].double(), lse[0].double(), kk, ctx - n, d ** -0.5)
    out = torch.zeros(b, ctx, device="cuda")
    desc = hs.make_desc(b, n, h, d, kv_dtype=hs.HS2_E4M3, max_ctx=ctx)
    ws = hs.alloc_accum_workspace(desc)
    hs.hs2_weight_accum(desc, *base._cu(q, k, ks, lse, pos0, None), 1.0, None, out, ws)
    rel = (2 * d * mag + 8 * (mag + 12)) * 2.0 ** -24 + 2.0 ** -20 + n * h * 2.0 ** -24
    assert (out.cpu()[0].double() - want).abs().le(rel * want + 2.0 ** -22 * want).all()


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("lens", [[9000], [20000, 19000], [70000] * 3, [300000, 299999], [40000] * 16])
def test_evict_one_cta_clusters_and_teams(lens):
    """One CTA, clusters of 8 and 16, teams of all SMs: ties across slices, NaN, infinities and zeros of
    both signs, counts above, at and below the ties, a last-bit difference."""
    b, cap = len(lens), max(lens)
    g = base._gen(cap)
    few = torch.randint(0, 3, (b, cap), generator=g).float()
    few[::2] = -few[::2]
    base._run_evict(few, lens, 2, 10, cap // 3 + 5, "e4m3", 64)
    odd = torch.randn(b, cap, generator=g)
    odd[:, ::7], odd[:, 1::7], odd[:, 2::7] = math.nan, math.inf, -math.inf
    odd[:, 3::7], odd[:, 4::7] = 0.0, -0.0
    base._run_evict(odd, lens, 0, 3, cap * 3 // 7, "bf16", 64)
    close = 1.0 + torch.randint(0, 3000, (b, cap), generator=g).float() * 2.0 ** -23
    base._run_evict(close, [max(1, n - 3000 * i) for i, n in enumerate(lens)], 1, 1, cap // 5, "e4m3", 64, out_extra=2)


def test_evict_kept_rows_around_the_ties():
    odd = torch.randn(1, 30000, generator=base._gen(2))
    odd[0, ::7], odd[0, 1::7], odd[0, 2::7] = math.nan, math.inf, -math.inf
    odd[0, 3::7], odd[0, 4::7] = 0.0, -0.0
    for budget in (1, 4285, 4286, 8000, 12850, 17140, 21430, 29980):
        base._run_evict(odd, [30000], 0, 3, budget, "bf16", 64)


def test_evict_long_slices_are_read_again():
    """More rows a CTA than shared memory holds: few kept rows (no room for counts beside them) of a
    long cache, with more equal totals than the lists take, and with lists."""
    base._run_evict(torch.ones(1, 700000), [700000], 0, 2, 9, "e4m3", 64)
    base._run_evict(torch.randint(0, 2, (1, 700000), generator=base._gen(1)).float(), [699000], 3, 0, 60, "e4m3", 64)
    base._run_evict(torch.rand(1, 700001, generator=base._gen(5)), [700001], 0, 0, 90, "e4m3", 64)


@pytest.mark.parametrize("n, kv", [(1, "bf16"), (1, "e4m3"), (20, "bf16"), (600, "bf16"), (600, "e4m3"), (3, "f32")])
def test_calls_of_no_rows(n, kv):
    """A padded batch without a row in use: outputs stay, totals fade, and what follows is not overtaken."""
    g = base._gen(n)
    b, h, d, ctx = 2, 16, 128, 9000
    dt = base.DT["f32" if kv == "f32" else "bf16"]
    q = torch.full((b, n, h, d), math.nan, dtype=dt, device="cuda")
    k, v, ks, vs = base._cu(*base._cache(g, b, ctx, d, kv))
    pos0 = torch.tensor([ctx - n, 100], dtype=torch.int32, device="cuda")
    none = torch.zeros(b, dtype=torch.int32, device="cuda")
    desc = hs.make_desc(b, n, h, d, window=8000, budget=0, q_dtype=base.KIND["f32" if kv == "f32" else "bf16"],
                        kv_dtype=base.KIND[kv], max_ctx=ctx)
    ws, aws = hs.alloc_window_workspace(desc, 4), hs.alloc_accum_workspace(desc)
    o, lse = torch.full_like(q, 7.0), torch.full((b, n, h), math.nan, device="cuda")
    acc = torch.rand(b, ctx, generator=g).cuda()
    out = torch.full_like(acc, -3.0)
    for _ in range(3):
        hs.hs2_window_attn(desc, 4, q, k, v, ks, vs, pos0, none, o, lse, ws)
        hs.hs2_weight_accum(desc, q, k, ks, lse, pos0, none, 0.5, acc, out, aws)
    assert hs.hs2_last_status(ws) == hs.HS2_OK and hs.hs2_last_status(aws) == hs.HS2_OK
    assert (o == 7).all() and lse.isnan().all()
    for s in range(b):
        p = int(pos0[s])
        assert torch.equal(out[s, :p], 0.5 * acc[s, :p]) and (out[s, p:] == -3).all()


def test_evict_many_sequences():
    acc = torch.rand(150, 300, generator=base._gen(6))
    base._run_evict(acc, [300 - i for i in range(150)], 1, 5, 50, "bf16", 64)


# ------------------------------------------------------------------ streams
def test_calls_on_two_streams_at_once():
    """The same calls on two side streams, each with its own outputs and workspaces, give the bits of
    calls made alone."""
    g = base._gen(44)
    b, h, d, ctx = 2, 16, 128, 6000
    k, v = (torch.randn(b, ctx, d, generator=g).bfloat16().cuda() for _ in range(2))
    acc0 = torch.rand(b, ctx, generator=g).cuda()
    ln = torch.full((b,), ctx, dtype=torch.int32, device="cuda")
    sets = []
    for n in (1, 40, 1, 40):
        q = torch.randn(b, n, h, d, generator=g).bfloat16().cuda()
        pos0 = torch.full((b,), ctx - n, dtype=torch.int32, device="cuda")
        desc = hs.make_desc(b, n, h, d, window=5000, budget=0, max_ctx=ctx)
        ed = hs.make_evict_desc(b, d, sinks=4, window=96, budget=400, kv_capacity=ctx)
        out = dict(o=torch.zeros_like(q), lse=torch.zeros(b, n, h, device="cuda"), acc=torch.zeros(b, ctx, device="cuda"),
                   ko=torch.zeros(b, 500, d, device="cuda").bfloat16(), vo=torch.zeros(b, 500, d, device="cuda").bfloat16(),
                   idx=torch.zeros(b, 500, dtype=torch.int32, device="cuda"), nl=torch.zeros(b, dtype=torch.int32, device="cuda"))
        sets.append((q, pos0, desc, ed, hs.alloc_window_workspace(desc, 4), hs.alloc_accum_workspace(desc), out))

    def run(s, stream):
        q, pos0, desc, ed, ws, aws, out = s
        hs.hs2_window_attn(desc, 4, q, k, v, None, None, pos0, None, out["o"], out["lse"], ws, stream=stream)
        hs.hs2_weight_accum(desc, q, k, None, out["lse"], pos0, None, 0.5, acc0, out["acc"], aws, stream=stream)
        hs.hs2_kv_evict(ed, ln, out["acc"], k, v, None, None, out["ko"], out["vo"], None, None, None, out["idx"], out["nl"],
                        stream=stream)

    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in sets:
        run(s, side[0])
    torch.cuda.synchronize()
    alone = [{key: t.clone() for key, t in s[-1].items()} for s in sets]
    for s in sets:
        for t in s[-1].values():
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for i, s in enumerate(sets):
            run(s, side[i % 2])
    torch.cuda.synchronize()
    for want, s in zip(alone, sets):
        for key, t in s[-1].items():
            assert torch.equal(t, want[key]), key


def test_two_graphs_share_a_workspace():
    """Two captured calls of one workspace, replayed in turn on one stream."""
    g = base._gen(45)
    b, h, d, ctx = 1, 16, 128, 9000
    k, v = (torch.randn(b, ctx, d, generator=g).bfloat16().cuda() for _ in range(2))
    desc = hs.make_desc(b, 1, h, d, window=8000, budget=0, max_ctx=ctx)
    ws = hs.alloc_window_workspace(desc, 4)
    qs = [torch.randn(b, 1, h, d, generator=g).bfloat16().cuda() for _ in range(2)]
    pos0 = torch.tensor([ctx - 1], dtype=torch.int32, device="cuda")
    outs, graphs, want = [], [], []
    for q in qs:
        o = torch.zeros_like(q)
        hs.hs2_window_attn(desc, 4, q, k, v, None, None, pos0, None, o, None, ws)
        torch.cuda.synchronize()
        want.append(o.clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            hs.hs2_window_attn(desc, 4, q, k, v, None, None, pos0, None, o, None, ws)
        outs.append(o)
        graphs.append(graph)
    for _ in range(3):
        for o, graph in zip(outs, graphs):
            o.zero_()
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
