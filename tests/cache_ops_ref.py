"""Plain fp64 forms of the calls around the block (query/key norm and rotation, sliding-window
attention, accumulated weight, eviction), row by row, for the tests.  CPU tensors in and out."""
import math

import torch


def wide(x, scale=None):
    """Cache rows as fp64 numbers (uint8: e4m3 codes)."""
    y = x.view(torch.float8_e4m3fn).double() if x.dtype == torch.uint8 else x.double()
    return y if scale is None else y * scale.double()[..., None]


def quantize(x):
    """fp32 rows -> (codes, scales) as hs2_kv_quantize_fp8 defines them."""
    s = x.abs().amax(-1) / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def rotate(head, pos, inv_freq, interleaved):
    """head [..., d] fp64 turned at one position."""
    y = head.clone()
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = float(pos) * float(inv_freq[i])
        c, s = math.cos(ang), math.sin(ang)
        y[..., a] = head[..., a] * c - head[..., b] * s
        y[..., b] = head[..., b] * c + head[..., a] * s
    return y


def norm_rope(x, weight, eps, pos, inv_freq, interleaved, normalize=True):
    """x [rows, heads, d] at pos [rows]."""
    x = x.double()
    out = torch.empty_like(x)
    for r in range(x.shape[0]):
        y = x[r]
        if normalize:
            y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt()
            if weight is not None:
                y = y * weight.double()
        out[r] = rotate(y, pos[r], inv_freq, interleaved)
    return out


def window_row(q, k, v, p, window, sinks, scale):
    """q [h, d] at position p over the rows k, v [ctx, d]: (o, lse, slack) with slack the sum of
    |q_d k_d| (times scale, largest over the visible rows) per head and sum of weight * |v|."""
    j = [i for i in range(p + 1) if i > p - window or i < sinks]
    x = (q @ k[j].T) * scale
    lse = x.logsumexp(-1)
    w = (x - lse[:, None]).exp()
    mag = (q.abs() @ k[j].abs().T).amax(-1) * scale
    return w @ v[j], lse, mag, w @ v[j].abs()


def weight_total(q, lse, k, p0, scale):
    """q [n, h, d], lse [n, h], k [ctx, d]: totals of keys 0 .. p0 + n - 1, and the largest
    sum of |q_d k_d| (times scale)."""
    n = q.shape[0]
    out = torch.zeros(p0 + n, dtype=torch.float64)
    mag = 0.0
    for r in range(n):
        kk = k[:p0 + r + 1]
        out[:p0 + r + 1] += ((q[r] @ kk.T) * scale - lse[r][:, None]).exp().sum(0)
        mag = max(mag, float((q[r].abs() @ kk.abs().T).max()) * scale)
    return out, mag


def evict_rows(acc, n, sinks, window, budget):
    """Kept rows of n, ascending."""
    if n <= sinks + window + budget:
        return list(range(n))
    mid = range(sinks, n - window)

    def key(j):
        x = float(acc[j])
        return (0, 0.0, j) if x != x else (-1, -x, j)           # NaN after every number; -0 == 0

    best = sorted(mid, key=key)[:budget]
    return list(range(sinks)) + sorted(best) + list(range(n - window, n))
