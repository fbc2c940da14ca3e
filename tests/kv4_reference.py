"""The 4-bit cache's format and the attention over it, from their definitions in 64 bits (torch float64, any device).

The format is written down here a second time: values by tables, rounding by
distances, bytes by explicit offsets.
"""
import math

import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def e4m3_values(device="cpu"):
    """The value of each e4m3 byte."""
    out = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if b & 127 == 127 else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        out.append(-v if b > 127 else v)
    return torch.tensor(out, dtype=torch.float64, device=device)


def nearest(x, values):
    """Index of the value nearest to x >= 0 among ascending `values`; a tie goes to the even index."""
    v = torch.tensor(values, dtype=torch.float64, device=x.device)
    i = torch.searchsorted(v, x.clamp(max=values[-1]), right=True) - 1
    j = (i + 1).clamp(max=len(values) - 1)
    low, high = x.clamp(max=values[-1]) - v[i], v[j] - x.clamp(max=values[-1])
    up = (high < low) | ((high == low) & (i % 2 == 1))
    return torch.where(up, j, i)


def stored(x, g=1.0):
    """What bf16 x [..., d] stands for once stored with tensor scale g."""
    b = x.double().unflatten(-1, (-1, 16))
    finite = torch.isfinite(b).all(-1, keepdim=True)
    b = torch.where(finite, b, 0.0)
    scales = [float(v) for v in e4m3_values()[:127]]
    s = e4m3_values(x.device)[nearest(b.abs().amax(-1, keepdim=True) / 6 / g, scales)]
    a = torch.where(s > 0, b.abs() / g / torch.where(s > 0, s, 1.0), 0.0)
    v = torch.tensor(E2M1, dtype=torch.float64, device=x.device)[nearest(a, E2M1)]
    out = torch.sign(b) * v * s * g
    return torch.where(finite, out, math.nan).flatten(-2)


def read(cache, d, page_size, pages, n, g_k=1.0, g_v=1.0):
    """K and V [n, heads, d] of the first n tokens of a sequence with these pages (a list), from the bytes."""
    heads = cache.shape[1]
    rb = d + d // 8
    tok = torch.arange(n, device=cache.device)
    page = torch.tensor(list(pages) + [0], device=cache.device)[tok // page_size]
    at = tok % page_size
    group, row = at // 16 * (16 * rb), at % 16
    values = e4m3_values(cache.device)
    e2m1 = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=cache.device)
    out = []
    for v, g in ((0, g_k), (1, g_v)):
        codes_at = group + v * 8 * rb + row * (d // 2)
        scales_at = group + v * 8 * rb + 8 * d + row * (d // 16)
        i = torch.arange(d, device=cache.device)
        byte = cache[page[:, None, None], torch.arange(heads, device=cache.device)[None, :, None],
                     (codes_at[:, None] + i // 2)[:, None, :]].long()
        code = torch.where(i % 2 == 0, byte & 15, byte >> 4)
        scale = cache[page[:, None, None], torch.arange(heads, device=cache.device)[None, :, None],
                      (scales_at[:, None] + i // 16)[:, None, :]].long()
        out.append(e2m1[code] * values[scale] * g)
    return out


def attend(q, k, v, scale):
    """q [n, Hq, d], the newest tokens of k, v [m, Hkv, d]: O [n, Hq, d], LSE [Hq, n] and w|V| + |O|.

    Keys a row does not see do not enter its sums, whatever they hold.
    """
    n, hq, d = q.shape
    m, group = k.shape[0], hq // k.shape[1]
    o = torch.zeros((n, hq, d), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    lse = torch.full((hq, n), -math.inf, dtype=torch.float64, device=q.device)
    most = 0.0
    for i in range(n):
        seen = m - n + 1 + i
        if seen <= 0:
            continue
        ks, vs = (t[:seen].double().repeat_interleave(group, 1) for t in (k, v))
        s = torch.einsum("hd,mhd->hm", q[i].double(), ks) * scale
        most = max(most, float(torch.nan_to_num(torch.einsum("hd,mhd->hm", q[i].double().abs(), ks.abs())).max()) * scale)
        lse[:, i] = torch.logsumexp(s, -1)
        w = torch.softmax(s, -1)
        o[i] = torch.einsum("hm,mhd->hd", w, vs)
        bound[i] = torch.einsum("hm,mhd->hd", w, vs.abs()) + o[i].abs()
    return o, lse, bound, most
