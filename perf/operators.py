"""Cases and plain forms of the operators around the hybrid block's cache.

Four operators, each computed either by the library (``own``) or in plain torch
operations in fp32 (angles in fp64), rounded once at the end:

  rope    per-head RMS norm and rotation of queries and keys; the keys and values go
          to their cache rows (bf16, or e4m3 codes with one scale per row, or fp32)
  window  attention over a sliding window and the first `sinks` tokens
  accum   attention weight of every cached key, summed over query rows and heads and
          added to a running total
  evict   the cache rows with the largest totals (with the first and the latest rows)
          moved into a smaller cache, in order

Sizes are those of the repository's workloads (16 heads of 128 over one shared K/V head,
contexts from 2K to 1M, agent rounds of 8192 new rows, 8 heads of 64 in fp32), with odd
sizes and other head counts between them.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
ROPE_THETA = 1.0e6


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token for each of 32 sequences: the call's latency counts
        dict(name="rope_decode_b32", op="rope", b=32, n=1, h=16, d=128, rot=128, inter=False, cache="bf16",
             dt="bf16", cap=2048, ctx=1700, ragged=False),
        # an agent round's 8192 new rows for 4 sequences, q/k/v out of one fused projection
        dict(name="rope_round_b4_n8192", op="rope", b=4, n=8192, h=16, d=128, rot=128, inter=False, cache="bf16",
             dt="bf16", cap=16384, ctx=8000, ragged=False),
        # a padded batch into an e4m3 cache, half of each head rotated in adjacent pairs
        dict(name="rope_padded_e4m3", op="rope", b=3, n=4097, h=16, d=128, rot=64, inter=True, cache="e4m3",
             dt="bf16", cap=8200, ctx=4000, ragged=True),
        # single tokens of 32 long sequences, the pages' window of 128
        dict(name="window_decode_b32_w128", op="window", b=32, n=1, h=16, d=128, w=128, sinks=4, ctx=16384,
             dt="bf16", kv="bf16", ragged=False),
        # a single token with a long window in an FP8 cache: split over the keys and joined
        dict(name="window_decode_b4_w32768_e4m3", op="window", b=4, n=1, h=16, d=128, w=32768, sinks=16, ctx=131072,
             dt="bf16", kv="e4m3", ragged=False),
        # an agent round through a layer with the pages' window
        dict(name="window_round_b4_n8192_w128", op="window", b=4, n=8192, h=16, d=128, w=128, sinks=4,
             ctx=65536 + 8192, dt="bf16", kv="bf16", ragged=False),
        # a prompt chunk through a layer with a long window
        dict(name="window_chunk_n8192_w4096", op="window", b=1, n=8192, h=16, d=128, w=4096, sinks=4, ctx=32768,
             dt="bf16", kv="bf16", ragged=False),
        # the fp32 block: 8 heads of 64, a padded batch of odd length
        dict(name="window_f32_h8_d64", op="window", b=2, n=1023, h=8, d=64, w=128, sinks=3, ctx=2048, dt="f32",
             kv="f32", ragged=True),
        # the last 32 rows of a round score a 128K cache
        dict(name="accum_b4_n32_ctx131072", op="accum", b=4, n=32, h=16, d=128, ctx=131072, dt="bf16", kv="bf16",
             decay=1.0, ragged=False),
        # one decode step's weights over an FP8 cache, older totals fading
        dict(name="accum_decode_b8_e4m3", op="accum", b=8, n=1, h=16, d=128, ctx=100001, dt="bf16", kv="e4m3",
             decay=0.96875, ragged=False),
        # 32 caches of 64K cut to 4096 rows and the window
        dict(name="evict_b32_65536_to_4228", op="evict", b=32, d=128, kv="bf16", ctx=65536, sinks=4, w=128,
             budget=4096, ragged=False),
        # a million-token FP8 cache halved
        dict(name="evict_1m_e4m3_half", op="evict", b=1, d=128, kv="e4m3", ctx=1 << 20, sinks=16, w=1024,
             budget=1 << 19, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "window", "window", "accum", "evict"])
    f32 = rng.random() < 0.2
    if f32:
        dt = kv = "f32"
    else:
        dt, kv = "bf16", rng.choice(["bf16", "bf16", "e4m3"])
    d = 64 if rng.random() < (0.7 if f32 else 0.25) else 128
    h = rng.choice([16, 16, 16, 8, 12, 5, 1, 24])
    ragged = rng.random() < 0.4
    if op == "rope":
        b = _log(rng, 1, 32)
        n = _log(rng, 1, max(1, 16384 // b))
        ctx = _log(rng, 1, 1 << 20)
        return dict(op=op, b=b, n=n, h=h, d=d, rot=rng.choice([d, d, d // 2, d // 4 * 3, 16]),
                    inter=rng.random() < 0.4, cache=kv, dt=dt, cap=n + rng.randrange(1, 64), ctx=ctx, ragged=ragged)
    if op == "window":
        sinks = rng.choice([0, 1, 4, 4, 16, 130])
        if rng.random() < 0.4:                                  # single tokens
            b = _log(rng, 1, 32)
            ctx = _log(rng, 1, (1 << 20) // b)
            n, w = 1, _log(rng, 1, (131072 if not f32 else 32768) // b)
        else:
            b = _log(rng, 1, 8)
            n = _log(rng, 2, (8192 if not f32 else 1024) // b)
            w = _log(rng, 1, 3960 if not f32 else 1024)
            ctx = n + _log(rng, 1, 32768 // b) - 1
        return dict(op=op, b=b, n=n, h=h if h <= 16 else 16, d=d, w=w, sinks=sinks, ctx=ctx, dt=dt, kv=kv,
                    ragged=ragged)
    if op == "accum":
        b = _log(rng, 1, 16)
        ctx = _log(rng, 1, (524288 if not f32 else 16384) // b)
        n = min(ctx, _log(rng, 1, max(1, min(2048, (1 << 24 if not f32 else 1 << 20) // (ctx * b)))))
        return dict(op=op, b=b, n=n, h=h if h <= 16 else 16, d=d, ctx=ctx, dt=dt, kv=kv,
                    decay=rng.choice([1.0, 1.0, 0.9]), ragged=ragged)
    b = _log(rng, 1, 64)
    ctx = _log(rng, 1, ((1 << 20) if kv == "e4m3" else (1 << 18)) // b)
    keep = _log(rng, 1, max(1, ctx // 2))
    return dict(op=op, b=b, d=d, kv=kv, ctx=ctx, sinks=rng.choice([0, 4, 16]), w=rng.choice([0, 1, 128]),
                budget=keep, ragged=ragged)


# ------------------------------------------------------------------------------- inputs
def _gen(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, shape, dt=torch.float32):
    return torch.randn(shape, generator=g, device=g.device).to(dt)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=g.device, dtype=torch.int32)


def _cache(g, b, rows, d, kv):
    """Cache rows as the library holds them: (k, v, k_scale, v_scale)."""
    if kv != "e4m3":
        return _normal(g, (b, rows, d), DTYPES[kv]), _normal(g, (b, rows, d), DTYPES[kv]), None, None
    out = []
    for _ in range(2):
        x = _normal(g, (b, rows, d))
        s = x.abs().amax(-1) / 448.0
        out.append(((x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), s))
        del x
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _empty_cache(b, rows, d, kv, dev):
    dt = torch.uint8 if kv == "e4m3" else DTYPES[kv]
    c = [torch.zeros(b, rows, d, dtype=dt, device=dev) for _ in range(2)]
    s = [torch.zeros(b, rows, device=dev) if kv == "e4m3" else None for _ in range(2)]
    return c[0], c[1], s[0], s[1]


def _rows_of(g, c):
    """Rows in use of each sequence of a padded batch (None: all of them)."""
    if not c["ragged"]:
        return None
    return _ints(g, max(0, c["n"] // 2), c["n"], c["b"])


def prepare(case, seed):
    dev = "cuda"
    g = _gen(seed, dev)
    c = dict(case)
    st = {"case": c}
    if c["op"] == "rope":
        b, n, h, d = c["b"], c["n"], c["h"], c["d"]
        # activations as a projection gives them, keys a little larger than queries
        qkv = torch.randn(b, n, h + 2, d, generator=g, device=dev)
        qkv[:, :, h] *= 1.5
        st["qkv"] = qkv.to(DTYPES[c["dt"]]).reshape(b, n, (h + 2) * d)
        st["qw"] = 1.0 + 0.1 * _normal(g, (d,))
        st["kw"] = 1.0 + 0.1 * _normal(g, (d,))
        st["freq"] = ROPE_THETA ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        # the cache row of a sequence's first row, and the positions (they differ after an eviction)
        st["row0"] = _ints(g, 0, c["cap"] - n, b)
        first = _ints(g, c["ctx"] // 2, c["ctx"], b)
        st["pos"] = (first[:, None] + torch.arange(n, device=dev, dtype=torch.int32)).contiguous()
        st["n_rows"] = _rows_of(g, c)
        st["q_out"] = torch.zeros(b, n, h, d, dtype=DTYPES[c["dt"]], device=dev)
        st["k"], st["v"], st["ks"], st["vs"] = _empty_cache(b, c["cap"], d, c["cache"], dev)
    elif c["op"] in ("window", "accum"):
        b, n, h, d, ctx = c["b"], c["n"], c["h"], c["d"], c["ctx"]
        st["q"] = _normal(g, (b, n, h, d), DTYPES[c["dt"]])
        st["k"], st["v"], st["ks"], st["vs"] = _cache(g, b, ctx, d, c["kv"])
        # contexts of unequal length where the batch is padded
        lo = ctx - n if not c["ragged"] else (ctx - n) // 2
        st["pos0"] = _ints(g, lo, ctx - n, b)
        st["n_rows"] = _rows_of(g, c)
        if c["op"] == "window":
            st["o"] = torch.zeros(b, n, h, d, dtype=DTYPES[c["dt"]], device=dev)
            st["lse"] = torch.zeros(b, n, h, device=dev)
        else:
            st["v"] = st["vs"] = None
            st["lse"] = _causal_lse(st)
            st["acc"] = _normal(g, (b, ctx)).exp()
            st["out"] = torch.zeros(b, ctx, device=dev)
    else:
        b, d, ctx = c["b"], c["d"], c["ctx"]
        st["k"], st["v"], st["ks"], st["vs"] = _cache(g, b, ctx, d, c["kv"])
        # totals spread over many octaves; some keys were hardly ever attended and tie
        acc = (2.0 * _normal(g, (b, ctx))).exp()
        coarse = torch.rand(b, ctx, generator=g, device=dev) < 0.25
        st["acc"] = torch.where(coarse, (acc * 4.0).floor() / 4.0, acc)
        st["len"] = _ints(g, ctx // 2 if c["ragged"] else ctx, ctx, b)
        keep = c["sinks"] + c["w"] + c["budget"]
        st["out"] = _empty_cache(b, keep, d, c["kv"], dev) + (torch.zeros(b, keep, device=dev),)
        st["idx"] = torch.zeros(b, keep, dtype=torch.int32, device=dev)
        st["new_len"] = torch.zeros(b, dtype=torch.int32, device=dev)
    return st


def _causal_lse(st):
    """Log-sum-exp of the scaled logits, as the attention layer returned it."""
    c = st["case"]
    out = torch.empty(c["b"], c["n"], c["h"], device=st["q"].device)
    for i in range(c["b"]):
        k = _wide(st["k"][i], None if st["ks"] is None else st["ks"][i], torch.float32)
        p = st["pos0"][i] + torch.arange(c["n"], device=k.device)
        for r in range(0, c["n"], 64):
            s = (st["q"][i, r:r + 64].float().reshape(-1, c["d"]) @ k.T) * c["d"] ** -0.5
            hide = torch.arange(c["ctx"], device=k.device) > p[r:r + 64].repeat_interleave(c["h"])[:, None]
            out[i, r:r + 64] = s.masked_fill_(hide, -math.inf).logsumexp(-1).reshape(-1, c["h"])
    return out


def _wide(x, scale, dt):
    """Cache rows as numbers."""
    if scale is None:
        return x.to(dt)
    return x.view(torch.float8_e4m3fn).to(dt) * scale.to(dt)[..., None]


# ------------------------------------------------------------------------------- plain forms
def _alive(st, n):
    """[b, n] truth: rows in use."""
    r = torch.arange(n, device=st["pos0" if "pos0" in st else "row0"].device).expand(st["case"]["b"], n)
    return r < (st["n_rows"][:, None] if st["n_rows"] is not None else n)


def _plain_rope(st):
    c = st["case"]
    b, n, h, d, rot = c["b"], c["n"], c["h"], c["d"], c["rot"]
    x = st["qkv"].float().reshape(b, n, h + 2, d)
    qk = x[:, :, :h + 1]
    w = torch.cat([st["qw"].expand(h, d), st["kw"][None]])
    qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + EPS) * w
    ang = st["pos"].double()[..., None] * st["freq"]
    cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    if c["inter"]:
        lo, hi = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([lo * cos - hi * sin, hi * cos + lo * sin], -1).flatten(-2)
    else:
        lo, hi = qk[..., :rot // 2], qk[..., rot // 2:rot]
        turned = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)
    qk = torch.cat([turned, qk[..., rot:]], -1)
    alive = _alive(st, n)
    st["q_out"].copy_(torch.where(alive[..., None, None], qk[:, :, :h].to(st["q_out"].dtype), st["q_out"]))
    bi, ti = alive.nonzero(as_tuple=True)
    at = st["row0"].long()[bi] + ti
    for src, dst, scale in ((qk[:, :, h], st["k"], st["ks"]), (x[:, :, h + 1], st["v"], st["vs"])):
        rows = src[bi, ti]
        if scale is None:
            dst[bi, at] = rows.to(dst.dtype)
        else:
            s = rows.abs().amax(-1) / 448.0
            s = torch.where(s > 0, s, torch.ones_like(s))
            dst[bi, at] = (rows / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            scale[bi, at] = s
    return _rope_out(st)


def _rope_out(st):
    f8 = st["case"]["cache"] == "e4m3"
    return {"q": st["q_out"], "k": st["k"].view(torch.float8_e4m3fn) if f8 else st["k"],
            "v": st["v"].view(torch.float8_e4m3fn) if f8 else st["v"], "ks": st["ks"], "vs": st["vs"]}


def _plain_window(st):
    """Blocks of query rows against the keys that any row of the block sees."""
    c = st["case"]
    b, n, h, d, w, sinks, ctx = c["b"], c["n"], c["h"], c["d"], c["w"], c["sinks"], c["ctx"]
    dev = st["q"].device
    bq = min(n, max(32, min(1024, w // 4)))
    nb = -(-n // bq)
    q = torch.zeros(b, nb * bq, h, d, device=dev)
    q[:, :n] = st["q"].float()
    first = st["pos0"].long()[:, None] + torch.arange(nb, device=dev) * bq                      # [b, nb]
    near = first[..., None] - w + 1 + torch.arange(bq + w - 1, device=dev)                      # [b, nb, keys]
    at = torch.cat([torch.arange(sinks, device=dev).expand(b, nb, sinks), near], -1)
    is_sink = torch.arange(at.shape[-1], device=dev) < sinks
    p = first[..., None] + torch.arange(bq, device=dev)                                         # [b, nb, bq]
    gap = p[..., None] - at[:, :, None]                                                         # [b, nb, bq, keys]
    see = torch.where(is_sink, gap >= w, (gap >= 0) & (gap < w)) & (at >= 0)[:, :, None]
    take = at.clamp(0, ctx - 1)
    seq = torch.arange(b, device=dev)[:, None, None]
    k = _wide(st["k"][seq, take], None if st["ks"] is None else st["ks"][seq, take], torch.float32)
    v = _wide(st["v"][seq, take], None if st["vs"] is None else st["vs"][seq, take], torch.float32)
    s = (q.reshape(b, nb, bq * h, d) @ k.transpose(-1, -2)) * d ** -0.5
    s = s.reshape(b, nb, bq, h, -1).masked_fill(~see[:, :, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    e = (s - m).exp()
    total = e.sum(-1, keepdim=True)
    o = (e.reshape(b, nb, bq * h, -1) @ v).reshape(b, nb * bq, h, d) / total.reshape(b, nb * bq, h, 1)
    lse = (m + total.log()).reshape(b, nb * bq, h)
    alive = _alive(st, n)
    st["o"].copy_(torch.where(alive[..., None, None], o[:, :n].to(st["o"].dtype), st["o"]))
    st["lse"].copy_(torch.where(alive[..., None], lse[:, :n], st["lse"]))
    return {"o": st["o"], "lse": st["lse"]}


def _plain_accum(st):
    c = st["case"]
    b, n, h, d, ctx = c["b"], c["n"], c["h"], c["d"], c["ctx"]
    dev = st["q"].device
    k = _wide(st["k"], st["ks"], torch.float32)
    s = (st["q"].float().reshape(b, n * h, d) @ k.transpose(-1, -2)) * d ** -0.5
    p = (s.reshape(b, n, h, ctx) - st["lse"][..., None]).exp()
    j = torch.arange(ctx, device=dev)
    see = (j <= (st["pos0"][:, None] + torch.arange(n, device=dev))[..., None]) & _alive(st, n)[..., None]
    total = torch.where(see[:, :, None], p, torch.zeros_like(p)).sum((1, 2))
    end = st["pos0"] + (st["n_rows"] if st["n_rows"] is not None else n)
    st["out"].copy_(torch.where(j < end[:, None], c["decay"] * st["acc"] + total, st["out"]))
    return st["out"]


def _plain_evict(st):
    c = st["case"]
    b, ctx = c["b"], c["ctx"]
    dev = st["acc"].device
    keep = c["sinks"] + c["w"] + c["budget"]
    n = st["len"].long()[:, None]
    j = torch.arange(ctx, device=dev)
    rank = torch.where((j < c["sinks"]) | (j >= n - c["w"]), torch.full_like(st["acc"], math.inf), st["acc"])
    rank = torch.where(j < n, rank, torch.full_like(rank, -math.inf))
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :keep]
    kept = torch.clamp(n, max=keep)
    slot = torch.arange(best.shape[1], device=dev)
    best = torch.where(slot < kept, best, torch.full_like(best, ctx)).sort(-1).values
    st["idx"].fill_(-1)
    st["idx"][:, :best.shape[1]] = torch.where(slot < kept, best, torch.full_like(best, -1)).int()
    st["new_len"].copy_(kept[:, 0])
    bi, si = (slot < kept).nonzero(as_tuple=True)
    src = best[bi, si]
    ko, vo, kso, vso, ao = st["out"]
    ko[bi, si] = st["k"][bi, src]
    vo[bi, si] = st["v"][bi, src]
    ao[bi, si] = st["acc"][bi, src]
    if kso is not None:
        kso[bi, si] = st["ks"][bi, src]
        vso[bi, si] = st["vs"][bi, src]
    return _evict_out(st)


def _evict_out(st):
    ko, vo, kso, vso, ao = st["out"]
    if st["case"]["kv"] == "e4m3":
        ko, vo = ko.view(torch.float8_e4m3fn), vo.view(torch.float8_e4m3fn)
    return {"k": ko, "v": vo, "ks": kso, "vs": vso, "acc": ao, "idx": st["idx"], "len": st["new_len"]}


# ------------------------------------------------------------------------------- the library's calls
def _plan(st):
    """Descriptions and workspaces, which a program makes once and keeps."""
    import kv_shared_b200 as hs

    kind = {"f32": hs.HS2_F32, "bf16": hs.HS2_BF16, "e4m3": hs.HS2_E4M3}
    c = st["case"]
    if c["op"] == "rope":
        row = (c["h"] + 2) * c["d"]
        desc = hs.make_rope_desc(c["b"], c["n"], c["h"], c["d"], rot_dim=c["rot"], interleaved=c["inter"],
                                 in_dtype=kind[c["dt"]], kv_dtype=kind[c["cache"]], eps=EPS, q_row=row, k_row=row,
                                 v_row=row, kv_capacity=c["cap"])
        qkv, h, d = st["qkv"], c["h"], c["d"]
        return hs, desc, (qkv[..., :h * d], qkv[..., h * d:(h + 1) * d], qkv[..., (h + 1) * d:])
    if c["op"] == "window":
        desc = hs.make_desc(c["b"], c["n"], c["h"], c["d"], window=c["w"], budget=0, q_dtype=kind[c["dt"]],
                            kv_dtype=kind[c["kv"]], max_ctx=c["ctx"])
        return hs, desc, hs.alloc_window_workspace(desc, c["sinks"])
    if c["op"] == "accum":
        desc = hs.make_desc(c["b"], c["n"], c["h"], c["d"], q_dtype=kind[c["dt"]], kv_dtype=kind[c["kv"]],
                            max_ctx=c["ctx"])
        return hs, desc, hs.alloc_accum_workspace(desc)
    desc = hs.make_evict_desc(c["b"], c["d"], kind[c["kv"]], sinks=c["sinks"], window=c["w"], budget=c["budget"],
                              kv_capacity=c["ctx"])
    return hs, desc, None


def _own(st):
    if "plan" not in st:
        st["plan"] = _plan(st)
    hs, desc, held = st["plan"]
    c = st["case"]
    if c["op"] == "rope":
        q, k, v = held
        hs.hs2_qk_norm_rope(desc, q, k, v, st["qw"], st["kw"], st["freq"], st["row0"], st["pos"], st["n_rows"],
                            st["q_out"], st["k"], st["v"], st["ks"], st["vs"])
        return _rope_out(st)
    if c["op"] == "window":
        hs.hs2_window_attn(desc, c["sinks"], st["q"], st["k"], st["v"], st["ks"], st["vs"], st["pos0"], st["n_rows"],
                           st["o"], st["lse"], held)
        return {"o": st["o"], "lse": st["lse"]}
    if c["op"] == "accum":
        hs.hs2_weight_accum(desc, st["q"], st["k"], st["ks"], st["lse"], st["pos0"], st["n_rows"], c["decay"],
                            st["acc"], st["out"], held)
        return st["out"]
    ko, vo, kso, vso, ao = st["out"]
    hs.hs2_kv_evict(desc, st["len"], st["acc"], st["k"], st["v"], st["ks"], st["vs"], ko, vo, kso, vso, ao, st["idx"],
                    st["new_len"])
    return _evict_out(st)


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "window": _plain_window, "accum": _plain_accum,
            "evict": _plain_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- floors
def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "e4m3": 1}
    if c["op"] == "rope":
        live = 0.75 if c["ragged"] else 1.0
        rows, d = c["b"] * c["n"] * live, c["d"]
        io = rows * ((c["h"] + 2) * d + c["h"] * d) * size[c["dt"]]
        cache = rows * 2 * (d * size[c["cache"]] + (4 if c["cache"] == "e4m3" else 0))
        return {"bytes": io + cache + rows * 4, "flops": rows * (c["h"] + 1) * (4 * d + 3 * c["rot"])}
    if c["op"] == "window":
        b, n, h, d, w, ctx = c["b"], c["n"], c["h"], c["d"], c["w"], c["ctx"]
        live = 0.75 if c["ragged"] and n > 1 else 1.0
        p0 = (ctx - n) * (0.75 if c["ragged"] else 1.0)
        keys = min(w + c["sinks"], p0 + n / 2 + 1)              # keys of a middle row
        union = min(w + c["sinks"] + n * live - 1, p0 + n * live)
        row = 2 * (d * size[c["kv"]] + (4 if c["kv"] == "e4m3" else 0))
        return {"bytes": b * (union * row + 2 * n * live * h * d * size[c["dt"]] + 4 * n * live * h),
                "flops": b * n * live * h * keys * 4 * d}
    if c["op"] == "accum":
        b, n, h, d, ctx = c["b"], c["n"], c["h"], c["d"], c["ctx"]
        p0 = (ctx - n) * (0.75 if c["ragged"] else 1.0)
        live = 0.75 if c["ragged"] and n > 1 else 1.0
        row = d * size[c["kv"]] + (4 if c["kv"] == "e4m3" else 0)
        return {"bytes": b * ((p0 + n * live) * (row + 8) + n * live * h * (d * size[c["dt"]] + 4)),
                "flops": b * n * live * h * (p0 + n / 2) * 2 * d}
    n = c["ctx"] * (0.75 if c["ragged"] else 1.0)
    kept = min(n, c["sinks"] + c["w"] + c["budget"])
    row = 2 * (c["d"] * size[c["kv"]] + (4 if c["kv"] == "e4m3" else 0)) + 4
    return {"bytes": c["b"] * (4 * n + 2 * kept * row + 4 * kept), "flops": 0}


# ------------------------------------------------------------------------------- 64 bits
def _live(st, i):
    return int(st["n_rows"][i]) if st["n_rows"] is not None else st["case"]["n"]


def _exact_rope(st):
    c = st["case"]
    b, n, h, d, rot = c["b"], c["n"], c["h"], c["d"], c["rot"]
    dev = st["qkv"].device
    half = rot // 2
    i = torch.arange(half, device=dev)
    first, second = (2 * i, 2 * i + 1) if c["inter"] else (i, i + half)
    q = torch.zeros(b, n, h, d, dtype=torch.float64, device=dev)
    cache = {m: torch.zeros(b, c["cap"], d, dtype=torch.float64, device=dev) for m in "kv"}
    scale = {m: torch.zeros(b, c["cap"], dtype=torch.float64, device=dev) for m in "kv"}
    for s in range(b):
        m = _live(st, s)
        x = st["qkv"][s, :m].double().reshape(m, h + 2, d)
        z = torch.polar(torch.ones((), dtype=torch.float64, device=dev), st["pos"][s, :m, None].double() * st["freq"])
        y = x[:, :h + 1] / (x[:, :h + 1].pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
        y[:, :h] *= st["qw"].double()
        y[:, h] *= st["kw"].double()
        t = torch.complex(y[..., first], y[..., second]) * z[:, None]
        y[..., first], y[..., second] = t.real, t.imag
        q[s, :m] = y[:, :h]
        r0 = int(st["row0"][s])
        for name, rows in (("k", y[:, h]), ("v", x[:, h + 1])):
            if c["cache"] == "e4m3":
                sc = rows.abs().amax(-1) / 448
                sc[sc == 0] = 1
                scale[name][s, r0:r0 + m] = sc
                rows = rows / sc[:, None]
            cache[name][s, r0:r0 + m] = rows
    f8 = c["cache"] == "e4m3"
    return {"q": q, "k": cache["k"], "v": cache["v"], "ks": scale["k"] if f8 else None,
            "vs": scale["v"] if f8 else None}


def _exact_window(st):
    c = st["case"]
    b, n, h, d = c["b"], c["n"], c["h"], c["d"]
    dev = st["q"].device
    out = torch.zeros(b, n, h, d, dtype=torch.float64, device=dev)
    lse = torch.zeros(b, n, h, dtype=torch.float64, device=dev)
    for s in range(b):
        m, p0 = _live(st, s), int(st["pos0"][s])
        for r in range(0, m, 128):
            e = min(m, r + 128)
            lo, hi = max(0, p0 + r - c["w"] + 1), p0 + e
            at = torch.arange(min(lo, hi), hi, device=dev)
            if lo > 0 and c["sinks"]:
                at = torch.cat([torch.arange(min(c["sinks"], lo), device=dev), at])
            k = _wide(st["k"][s, at], None if st["ks"] is None else st["ks"][s, at], torch.float64)
            v = _wide(st["v"][s, at], None if st["vs"] is None else st["vs"][s, at], torch.float64)
            p = p0 + torch.arange(r, e, device=dev)[:, None]
            see = (at <= p) & ((at > p - c["w"]) | (at < c["sinks"]))
            x = torch.einsum("rhd,kd->rhk", st["q"][s, r:e].double(), k) / math.sqrt(d)
            x[~see[:, None].expand_as(x)] = -math.inf
            lse[s, r:e] = x.logsumexp(-1)
            out[s, r:e] = torch.einsum("rhk,kd->rhd", x.softmax(-1), v)
    return {"o": out, "lse": lse}


def _exact_accum(st):
    c = st["case"]
    out = torch.zeros(c["b"], c["ctx"], dtype=torch.float64, device=st["q"].device)
    for s in range(c["b"]):
        m, p0 = _live(st, s), int(st["pos0"][s])
        out[s, :p0 + m] = c["decay"] * st["acc"][s, :p0 + m].double()
        k = _wide(st["k"][s, :p0 + m], None if st["ks"] is None else st["ks"][s, :p0 + m], torch.float64)
        for r in range(0, m, 16):
            e = min(m, r + 16)
            x = torch.einsum("kd,rhd->krh", k, st["q"][s, r:e].double()) / math.sqrt(c["d"])
            x = torch.exp(x - st["lse"][s, r:e].double())
            x *= (torch.arange(p0 + m, device=k.device)[:, None] <= p0 + torch.arange(r, e, device=k.device))[..., None]
            out[s, :p0 + m] += x.sum((1, 2))
    return out


def _exact_evict(st):
    c = st["case"]
    keep = c["sinks"] + c["w"] + c["budget"]
    outs = [None if t is None else torch.zeros(t.shape, dtype=torch.float64, device=t.device) for t in st["out"]]
    idx = torch.full_like(st["idx"], -1)
    new_len = torch.zeros_like(st["new_len"])
    for s in range(c["b"]):
        n = int(st["len"][s])
        if n <= keep:
            at = torch.arange(n)
        else:
            mid = st["acc"][s, c["sinks"]:n - c["w"]].cpu()
            # descending totals, the lower row first among equals
            best = torch.argsort(-mid.double(), stable=True)[:c["budget"]] + c["sinks"]
            at = torch.cat([torch.arange(c["sinks"]), best.sort().values, torch.arange(n - c["w"], n)])
        new_len[s] = at.numel()
        idx[s, :at.numel()] = at.int().to(idx.device)
        at = at.to(idx.device)
        for dst, src in zip(outs, (st["k"], st["v"], st["ks"], st["vs"], st["acc"])):
            if dst is not None:
                rows = src[s, at]
                rows = rows.view(torch.float8_e4m3fn) if rows.dtype == torch.uint8 else rows
                dst[s, :at.numel()] = rows.double()
    return {"k": outs[0], "v": outs[1], "ks": outs[2], "vs": outs[3], "acc": outs[4], "idx": idx, "len": new_len}


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "window": _exact_window, "accum": _exact_accum,
            "evict": _exact_evict}[case["op"]](st)
