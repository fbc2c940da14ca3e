"""The serving operators: plain forms, inputs and cases for timing and comparing them.

Four operators are measured:

- ``prompt``: attention over packed prompts of different lengths with grouped heads;
- ``store``: quantising new keys and values into a paged 4-bit cache (the result is read
  back through ``load``, since 4-bit contents are compared by the values they stand for);
- ``load``: reading keys and values of cached sequences back as bf16;
- ``decode``: attention of the newest tokens of each sequence over the 4-bit cache.

The 4-bit format: 16 consecutive elements of a head share one e4m3 scale
s = e4m3(amax / 6), and each element is the e2m1 value nearest to x / s (ties to the even
code).  A page holds ``page`` tokens of every KV head, as groups of 16 tokens; a group is
[K codes 16 x d/2][K scales 16 x d/16][V codes 16 x d/2][V scales 16 x d/16] bytes, the
even element of a code byte in its low four bits.
"""
import math
import random

import torch

own = False

GROUP = 16   # tokens of one group of a page
BLOCK = 16   # elements that share a scale


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one short question to a model with grouped heads: latency
        {"name": "prompt-1x37", "kind": "prompt", "seqs": 1, "longest": 37, "ragged": False, "mix": 0,
         "hq": 32, "hkv": 8, "d": 128, "causal": True},
        # a batch of chat turns of very different lengths
        {"name": "prompt-24-ragged", "kind": "prompt", "seqs": 24, "longest": 1901, "ragged": True, "mix": 3,
         "hq": 32, "hkv": 8, "d": 128, "causal": True},
        # documents of one length through an encoder without grouped heads: no mask
        {"name": "prompt-8x1024-full", "kind": "prompt", "seqs": 8, "longest": 1024, "ragged": False, "mix": 0,
         "hq": 16, "hkv": 16, "d": 64, "causal": False},
        # one long document
        {"name": "prompt-1x16384", "kind": "prompt", "seqs": 1, "longest": 16384, "ragged": False, "mix": 0,
         "hq": 16, "hkv": 2, "d": 128, "causal": True},
        # a decoding step's new tokens: latency
        {"name": "store-step-64", "kind": "store", "seqs": 64, "longest": 1, "ragged": False, "mix": 0,
         "before": 700, "page": 64, "hkv": 8, "d": 128},
        # the keys and values of packed prompts
        {"name": "store-prompts", "kind": "store", "seqs": 40, "longest": 8191, "ragged": True, "mix": 5,
         "before": 0, "page": 64, "hkv": 8, "d": 128},
        # a shared prefix for a dense call
        {"name": "load-prefix", "kind": "load", "seqs": 3, "longest": 1000, "ragged": True, "mix": 1,
         "page": 16, "hkv": 4, "d": 64},
        # moving whole sequences out of the cache
        {"name": "load-sequences", "kind": "load", "seqs": 16, "longest": 4096, "ragged": False, "mix": 0,
         "page": 64, "hkv": 8, "d": 128},
        # one user, short context: latency
        {"name": "decode-1x500", "kind": "decode", "seqs": 1, "longest": 500, "ragged": False, "mix": 0,
         "queries": 1, "page": 64, "hq": 32, "hkv": 8, "d": 128},
        # a server's batch with contexts of very different lengths
        {"name": "decode-96-ragged", "kind": "decode", "seqs": 96, "longest": 16000, "ragged": True, "mix": 7,
         "queries": 1, "page": 64, "hq": 32, "hkv": 8, "d": 128},
        # several proposed tokens checked at once, small heads and pages
        {"name": "decode-16x4-d64", "kind": "decode", "seqs": 16, "longest": 4001, "ragged": True, "mix": 2,
         "queries": 4, "page": 16, "hq": 16, "hkv": 4, "d": 64},
        # one user with a very long context
        {"name": "decode-1x131072", "kind": "decode", "seqs": 1, "longest": 131072, "ragged": False, "mix": 0,
         "queries": 1, "page": 128, "hq": 32, "hkv": 8, "d": 128},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("prompt", "store", "load", "decode"))
    d = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 4, 8))
    heads = rng.choice((1, 2, 3, 4, 8))
    case = {"kind": kind, "d": d, "hkv": hkv, "ragged": rng.random() < 0.7, "mix": rng.randrange(1 << 20)}
    if kind == "prompt":
        case["seqs"] = _log_int(rng, 1, 64)
        case["longest"] = _log_int(rng, 2, 8192 // case["seqs"])
        case["hq"] = hkv * heads
        case["causal"] = rng.random() < 0.8
        return case
    case["page"] = rng.choice((16, 32, 64, 128))
    if kind == "decode":
        case["seqs"] = _log_int(rng, 1, 128)
        case["longest"] = _log_int(rng, 8, 131072 // case["seqs"])
        case["queries"] = rng.choice((1, 1, 1, 2, 4))
        case["hq"] = hkv * heads
        return case
    case["seqs"] = _log_int(rng, 1, 128)
    case["longest"] = _log_int(rng, 1, 65536 // case["seqs"])
    if kind == "store":
        case["before"] = rng.choice((0, 1, 37, 700))
    return case


def _lengths(case):
    """The case's sequence lengths: all ``longest``, or that and others down to a fiftieth of it."""
    n, top = case["seqs"], case["longest"]
    if not case["ragged"]:
        return [top] * n
    r = random.Random(case["mix"])
    return [top] + [_log_int(r, max(1, top // 50), top) for _ in range(n - 1)]


def _row_bytes(d):
    """Bytes of one token of one KV head: codes and scales of K and V."""
    return d + d // 8


def work(case):
    n = _lengths(case)
    total, hkv, d = sum(n), case["hkv"], case["d"]
    if case["kind"] == "prompt":
        hq = case["hq"]
        pairs = sum(m * (m + 1) // 2 if case["causal"] else m * m for m in n)
        return {"bytes": total * (2 * hq + 2 * hkv) * d * 2 + total * hq * 4, "flops": 4 * pairs * hq * d}
    if case["kind"] == "decode":
        hq, nq = case["hq"], case["queries"]
        rows = case["seqs"] * nq * hq
        seen = sum(max(0, m - nq + 1 + i) for m in n for i in range(nq))
        return {"bytes": total * hkv * _row_bytes(d) + rows * (d * 4 + 4), "flops": 4 * seen * hq * d}
    values = 2 * total * hkv * d
    one_way = values * 2 + total * hkv * _row_bytes(d)
    # a division and a rounding for each stored value, a product for each one read
    return {"bytes": one_way * (2 if case["kind"] == "store" else 1), "flops": values * (3 if case["kind"] == "store" else 1)}


# ---------------------------------------------------------------------------
# The 4-bit format in elementary operations
# ---------------------------------------------------------------------------
def _quantise(x):
    """fp32 [..., d] to code bytes [..., d/2] and scale bytes [..., d/16]."""
    b = x.unflatten(-1, (-1, BLOCK))
    six = torch.full((), 6.0, device=x.device)  # a tensor: an exact division, not a product with 1/6
    s8 = (b.abs().amax(-1) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float().unsqueeze(-1)
    a = torch.where(s > 0, b.abs() / s, 0.0)
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(b)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], s8.view(torch.uint8)


def _dequantise(codes, scales):
    """Code and scale bytes back to fp32 [..., d]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    m = c & 7
    low = m.float() * 0.5
    high = (1.0 + 0.5 * (m & 1).float()) * torch.exp2((m >> 1).float() - 1.0)
    v = torch.where(m < 2, low, high)
    v = torch.where(c > 7, -v, v)
    s = scales.contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return (v.unflatten(-1, (-1, BLOCK)) * s).flatten(-2)


def _fields(cache, d):
    """Views of the cache [pages, hkv, bytes]: K codes, K scales, V codes, V scales, each
    [pages, hkv, groups, 16, bytes of a row]."""
    g = cache.unflatten(-1, (-1, GROUP * _row_bytes(d)))
    half, blocks = d // 2, d // BLOCK
    ends = [0]
    for width in (half, blocks, half, blocks):
        ends.append(ends[-1] + GROUP * width)
    return [g[..., ends[i]:ends[i + 1]].unflatten(-1, (GROUP, -1)) for i in range(4)]


def _places(state):
    """Page, group and row of every token of a packed store or load."""
    n, lens = state["cu"][1:] - state["cu"][:-1], state["seq_lens"]
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n.long(), output_size=state["tokens"])
    at = lens[seq] - n[seq] + torch.arange(state["tokens"], device=n.device) - state["cu"][seq]
    page = state["page_table"][seq, (at // state["page"]).long()].long()
    at = (at % state["page"]).long()
    return page, at // GROUP, at % GROUP


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _keys_values(g, tokens, hkv, d):
    """Keys whose channels differ in size, as those of trained models do, and plain values."""
    spread = torch.exp(0.6 * _normal(g, hkv, d))
    return (_normal(g, tokens, hkv, d) * spread).bfloat16(), _normal(g, tokens, hkv, d).bfloat16()


def _cache(g, case, lens):
    """A cache whose pages all hold quantised keys and values, and a page table in random order."""
    page, hkv, d = case["page"], case["hkv"], case["d"]
    need = [max(1, -(-m // page)) for m in lens]
    pages = sum(need) + 3
    width = max(need)
    cache = torch.empty((pages, hkv, page * _row_bytes(d)), dtype=torch.uint8, device="cuda")
    spread = torch.exp(0.6 * _normal(g, hkv, 1, 1, d))
    step = max(1, (1 << 26) // (hkv * page * d))
    for p in range(0, pages, step):
        part = cache[p:p + step]
        kc, ks, vc, vs = _fields(part, d)
        shape = (part.shape[0], hkv, page // GROUP, GROUP, d)
        for codes, scales, x in ((kc, ks, _normal(g, *shape) * spread), (vc, vs, _normal(g, *shape))):
            c, s = _quantise(x.bfloat16().float())
            codes.copy_(c)
            scales.copy_(s)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    need_t = torch.tensor(need, device="cuda")
    first = torch.cumsum(need_t, 0) - need_t
    col = torch.arange(width, device="cuda")
    used = col < need_t.unsqueeze(1)
    table = torch.where(used, order[(first.unsqueeze(1) + col).clamp(max=pages - 1)], 0).to(torch.int32)
    return cache, table.contiguous()


def prepare(case, seed):
    g = _generator(seed)
    lens, d, hkv = _lengths(case), case["d"], case["hkv"]
    total = sum(lens)
    state = {"kind": case["kind"], "d": d, "hkv": hkv, "scale": d ** -0.5}
    if case["kind"] == "prompt":
        # one projection's output: q, k and v are views of its rows
        hq = case["hq"]
        qkv = torch.empty((total, (hq + 2 * hkv) * d), dtype=torch.bfloat16, device="cuda")
        q, k, v = qkv.split((hq * d, hkv * d, hkv * d), dim=1)
        q.copy_(_normal(g, total, hq * d))
        kk, vv = _keys_values(g, total, hkv, d)
        k.copy_(kk.view(total, -1))
        v.copy_(vv.view(total, -1))
        state.update(q=q.view(total, hq, d), k=k.view(total, hkv, d), v=v.view(total, hkv, d), hq=hq,
                     lens=lens, causal=case["causal"])
        return state
    state["page"] = case["page"]
    before = case.get("before", 0)
    whole = [m + before for m in lens]
    state["cache"], state["page_table"] = _cache(g, case, whole)
    state["seq_lens"] = torch.tensor(whole, dtype=torch.int32, device="cuda")
    if case["kind"] == "decode":
        hq, nq = case["hq"], case["queries"]
        state.update(q=_normal(g, case["seqs"] * nq, hq, d).bfloat16(), hq=hq, queries=nq)
        return state
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    state.update(cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), tokens=total)
    if case["kind"] == "store":
        state["k"], state["v"] = _keys_values(g, total, hkv, d)
    return state


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------
def run(state):
    return _own(state) if own else _plain(state)


def _own(state):
    from exact_attention_20_gb300 import serve

    kind = state["kind"]
    if kind == "prompt":
        return serve.attention_packed(state["q"], state["k"], state["v"], state["lens"], causal=state["causal"],
                                      scale=state["scale"])
    if kind == "decode":
        return serve.kv4_attention(state["q"], state["cache"], state["page_table"], state["seq_lens"],
                                   n_queries=state["queries"], scale=state["scale"])
    if kind == "store":
        serve.kv4_store(state["cache"], state["k"], state["v"], state["page_table"], state["seq_lens"], state["cu"])
    return serve.kv4_load(state["cache"], state["page_table"], state["seq_lens"], state["cu"], state["tokens"],
                          d=state["d"])


def _plain(state):
    kind = state["kind"]
    if kind == "prompt":
        return _plain_prompt(state)
    if kind == "decode":
        return _plain_decode(state)
    page, group, row = _places(state)
    kc, ks, vc, vs = _fields(state["cache"], state["d"])
    if kind == "store":
        kc[page, :, group, row], ks[page, :, group, row] = _quantise(state["k"].float())
        vc[page, :, group, row], vs[page, :, group, row] = _quantise(state["v"].float())
    return (_dequantise(kc[page, :, group, row], ks[page, :, group, row]).bfloat16(),
            _dequantise(vc[page, :, group, row], vs[page, :, group, row]).bfloat16())


def _softmax_product(s, v):
    """exp(s - max) v / sum over the last dimension of the scores s (overwritten), and the
    logsumexp; a row whose scores are all -inf gives 0 and -inf."""
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = s.sum(-1, keepdim=True)
    return torch.matmul(s, v) / torch.where(l > 0, l, 1.0), (m + torch.log(l)).squeeze(-1)


def _plain_prompt(state):
    q, k, v = state["q"], state["k"], state["v"]
    total, hq, d = q.shape
    hkv = state["hkv"]
    lens = torch.tensor(state["lens"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(lens.numel(), device="cuda"), lens, output_size=total)
    hidden = seq.unsqueeze(1) != seq
    if state["causal"]:
        at = torch.arange(total, device="cuda")
        hidden |= at > at.unsqueeze(1)
    qf = q.float().view(total, hkv, hq // hkv, d).permute(1, 2, 0, 3)           # [hkv, G, T, d]
    kf, vf = (t.float().permute(1, 0, 2).unsqueeze(1) for t in (k, v))            # [hkv, 1, T, d]
    s = torch.matmul(qf, kf.transpose(-1, -2)).mul_(state["scale"])
    s.masked_fill_(hidden, -math.inf)
    o, lse = _softmax_product(s, vf)
    return o.permute(2, 0, 1, 3).reshape(total, hq, d).bfloat16(), lse.reshape(hq, total)


def _plain_decode(state):
    q, lens, nq, d, hkv = state["q"], state["seq_lens"], state["queries"], state["d"], state["hkv"]
    n, hq = lens.numel(), state["hq"]
    table = state["page_table"].long()
    kc, ks, vc, vs = (f[table].transpose(1, 2).flatten(2, 4) for f in _fields(state["cache"], d))  # [S, hkv, keys, ...]
    k, v = _dequantise(kc, ks).unsqueeze(2), _dequantise(vc, vs).unsqueeze(2)     # [S, hkv, 1, keys, d]
    qf = q.float().view(n, nq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)          # [S, hkv, G, nq, d]
    s = torch.matmul(qf, k.transpose(-1, -2)).mul_(state["scale"])
    last = lens.unsqueeze(1) - nq + torch.arange(nq, device="cuda")               # [S, nq]: each query's own place
    hidden = torch.arange(k.shape[-2], device="cuda") > last.unsqueeze(-1)        # [S, nq, keys]
    s.masked_fill_(hidden.view(n, 1, 1, nq, -1), -math.inf)
    o, lse = _softmax_product(s, v)
    return (o.permute(0, 3, 1, 2, 4).reshape(n * nq, hq, d).bfloat16(),
            lse.permute(1, 2, 0, 3).reshape(hq, n * nq))


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_64(x):
    """The e4m3 value nearest to x >= 0, ties to even, at most 448."""
    x = x.clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _stored_64(x):
    """What x stands for once stored, in float64."""
    b = x.double().unflatten(-1, (-1, BLOCK))
    s = _e4m3_64(b.abs().amax(-1, keepdim=True) / 6)
    a = b.abs() / torch.where(s > 0, s, 1.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=1.0, max=6.0))) - 1)
    return (torch.sign(b) * (torch.round(a / step) * step).clamp(max=6.0) * s).flatten(-2)


def _table_64(entry, count):
    return torch.tensor([entry(i) for i in range(count)], dtype=torch.float64, device="cuda")


def _read_64(cache, d, pages, first, count):
    """K and V of tokens first .. first + count - 1 of a sequence with these pages, float64 [count, hkv, d],
    by tables of the codes' and scales' values."""
    e2m1 = _table_64(lambda i: (-1) ** (i >> 3) * (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)[i & 7], 16)
    e4m3 = _table_64(lambda i: math.nan if i & 127 == 127 else (-1) ** (i >> 7) * (
        (i & 7) * 2.0 ** -9 if (i & 127) < 8 else (8 + (i & 7)) * 2.0 ** (((i >> 3) & 15) - 10)), 256)
    size = GROUP * _row_bytes(d)
    rows = cache[pages.long()].transpose(1, 2).reshape(pages.numel(), -1, size // GROUP * GROUP, cache.shape[1])
    rows = rows.reshape(-1, size, cache.shape[1])                                  # [groups, bytes, hkv]
    out = []
    for start in (0, size // 2):
        codes = rows[:, start:start + 8 * d].reshape(-1, d // 2, cache.shape[1])
        scales = rows[:, start + 8 * d:start + 9 * d].reshape(-1, d // 16, cache.shape[1])
        codes, scales = (t[first:first + count].transpose(1, 2).int() for t in (codes, scales))
        v = torch.empty((count, cache.shape[1], d), dtype=torch.float64, device="cuda")
        v[..., 0::2], v[..., 1::2] = e2m1[codes % 16], e2m1[codes // 16]
        out.append(v * e4m3[scales].repeat_interleave(16, -1))
    return out


def _attend_64(q, k, v, scale, first_row, causal):
    """One sequence and one KV head: q [n, G, d] at places first_row .. of keys k [m, d]; O [n, G, d], LSE [G, n]."""
    s = torch.einsum("ngd,md->gnm", q, k) * scale
    if causal:
        place = torch.arange(q.shape[0], device="cuda") + first_row
        s = s.masked_fill(torch.arange(k.shape[0], device="cuda") > place.unsqueeze(1), -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse).unsqueeze(-1))
    return torch.einsum("gnm,md->ngd", p, v), lse


def exact(case, seed):
    state = prepare(case, seed)
    kind, d, hkv = case["kind"], case["d"], case["hkv"]
    if kind == "store":
        return _stored_64(state["k"]), _stored_64(state["v"])
    lens = _lengths(case)
    if kind == "load":
        parts = [_read_64(state["cache"], d, state["page_table"][i], 0, m) for i, m in enumerate(lens)]
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    group = case["hq"] // hkv
    o = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros((case["hq"], o.shape[0]), dtype=torch.float64, device="cuda")
    at = 0
    for i, m in enumerate(lens):
        if kind == "prompt":
            k, v = state["k"][at:at + m].double(), state["v"][at:at + m].double()
            rows, first, causal = m, 0, case["causal"]
        else:
            k, v = _read_64(state["cache"], d, state["page_table"][i], 0, m)
            rows, first, causal = case["queries"], m - case["queries"], True
        q = state["q"][at:at + rows].double()
        for h in range(hkv):
            heads = slice(h * group, (h + 1) * group)
            for r in range(0, rows, 2048):  # rows at a time, to bound the scores' memory
                part = slice(at + r, at + min(rows, r + 2048))
                o[part, heads], lse[heads, part] = _attend_64(
                    q[r:r + 2048, heads], k[:, h], v[:, h], state["scale"], first + r, causal)
        at += rows
    return o, lse
