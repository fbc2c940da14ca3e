"""Trees of drafted tokens from their definitions in 64 bits (torch float64, any device)."""
import math

import torch


def lines(parents, first_position=0):
    """Each node's line from the context, itself included; [] for a place without a node."""
    out = []
    for i, p in enumerate(parents):
        if first_position + i < 0 or not (p == -1 or (0 <= p < i and out[p])):
            out.append([])
        else:
            out.append(([] if p == -1 else out[p]) + [i])
    return out


def depths(parents):
    return [max(0, len(x) - 1) for x in lines(parents)]


def tree(g, nodes, roots=1, absent=0):
    """Random parents: `roots` nodes at the context, the last `absent` places empty."""
    out = [-1] * min(roots, nodes)
    while len(out) < nodes:
        out.append(int(torch.randint(0, len(out), (1,), generator=g)))
    for i in range(absent):
        out[nodes - 1 - i] = -2
    return out


def attend(q, k, v, parents, scale):
    """q [n, Hq, d], the nodes at the last n of k, v [m, Hkv, d]: O, LSE [Hq, n], w|V| + |O|, the largest scale sum|q||k|, keys."""
    n, hq, d = q.shape
    m, group = k.shape[0], hq // k.shape[1]
    o = torch.zeros((n, hq, d), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    lse = torch.full((hq, n), -math.inf, dtype=torch.float64, device=q.device)
    most = 0.0
    for i, line in enumerate(lines(parents, m - n)):
        if not line:
            continue
        seen = torch.tensor(list(range(max(0, m - n))) + [m - n + j for j in line if m - n + j >= 0], device=q.device)
        ks, vs = (t[seen].double().repeat_interleave(group, 1) for t in (k, v))
        s = torch.einsum("hd,mhd->hm", q[i].double(), ks) * scale
        most = max(most, float(torch.nan_to_num(torch.einsum("hd,mhd->hm", q[i].double().abs(), ks.abs())).max()) * scale)
        lse[:, i] = torch.logsumexp(s, -1)
        w = torch.softmax(s, -1)
        o[i] = torch.einsum("hm,mhd->hd", w, vs)
        bound[i] = torch.einsum("hm,mhd->hd", w, vs.abs()) + o[i].abs()
    return o, lse, bound, most


def target(logits, temperature):
    x = torch.where(torch.isnan(logits), -math.inf, logits.double().clamp(max=3.4028234663852886e38))
    if bool((x == -math.inf).all()):
        return None
    if temperature == 0:
        return torch.zeros_like(x).index_fill_(0, torch.nonzero(x == x.max())[0], 1.0)
    return torch.softmax((x - x.max()) / temperature, -1)


def verify(logits, tokens, parents, u, probs, temperature):
    """One sequence: logits [n, V], lists of n: (path, next token)."""
    n, V = logits.shape
    if parents[0] != -1:
        return [], -1
    path = [0]
    while True:
        at = path[-1]
        r = target(logits[at], temperature)
        if r is None:
            return path, -1
        taken = None
        for j in range(at + 1, n):
            x = tokens[j]
            if parents[j] != at or not 0 <= x < V:
                continue
            q = probs[at].double() if probs is not None else torch.zeros_like(r).index_fill_(0, torch.tensor([x], device=r.device), 1.0)
            if u[j] * float(q[x]) < float(r[x]):
                taken = j
                break
            left = (r - q).clamp(min=0)
            if float(left.sum()) > 0:
                r = left / left.sum()
        if taken is None:
            c = torch.cumsum(r, 0)
            return path, int(torch.nonzero(c > u[0] * float(c[-1]))[0])
        path.append(taken)
