"""Rotary positions and drafted tokens: plain forms, inputs and cases for timing and comparing them.

Five operators are measured:

- ``rotary``: turning queries and keys by their positions, forward and backward;
- ``append``: turning new queries and keys and storing keys and values into the paged
  4-bit cache on the way (the stored tokens are read back as the values they stand for);
- ``tree``: attention of a tree of drafted tokens over the cache that holds them;
- ``verify``: drafted tokens against the target's probabilities, from given random numbers;
- ``keep``: moving the accepted path's tokens to the front of the tree's places in the
  cache (the tree's places are read back afterwards).

The angle of pair i at position p is 2 pi frac(p turns[i] / 2^64), ``turns`` being whole
numbers, so that far positions lose nothing.  A stored key is turned, rounded to bf16 and
then to the cache's 4 bits: 16 consecutive elements of a head share one e4m3 scale s =
e4m3(amax / 6), and each element is the e2m1 value nearest to x / s (ties to the even
code).  A page holds ``page`` tokens of every KV head, as groups of 16 tokens; a group is
[K codes 16 x d/2][K scales 16 x d/16][V codes 16 x d/2][V scales 16 x d/16] bytes, the
even element of a code byte in its low four bits.

A tree's nodes are the last ``nodes`` tokens of their sequence; ``parents`` names each
one's parent, -1 the context itself, -2 a place without a node.  In ``verify`` node 0 is
the token that the context ends with; a node's children were drawn from the draft's
distribution at that node (or are given, without one).
"""
import math
import random

import torch

own = False

GROUP = 16   # tokens of one group of a page
BLOCK = 16   # elements that share a scale
TURN = (1 << 128) * 10 ** 38 // 628318530717958647692528676655900576839  # 2^128 / (2 pi)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decoding step of a model that turns half of each head's elements, in pairs: latency
        {"name": "rotary-step-64", "kind": "rotary", "batch": 1, "tokens": 64, "hq": 32, "hkv": 8, "d": 128, "rot": 64,
         "interleaved": True, "factor": 1.0, "first": 200000, "dense": False},
        # a training step: [B, H, N, d] forward and backward
        {"name": "rotary-train-4x4096", "kind": "rotary", "batch": 4, "tokens": 4096, "hq": 32, "hkv": 32, "d": 128, "rot": 128,
         "interleaved": False, "factor": 1.0, "first": 0, "dense": True},
        # a decoding step's new tokens, far into long contexts: latency
        {"name": "append-step-96", "kind": "append", "seqs": 96, "longest": 1, "ragged": False, "mix": 0, "before": 700,
         "shift": 1000000, "page": 64, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "interleaved": False, "factor": 8.0},
        # the tokens of packed prompts
        {"name": "append-prompts", "kind": "append", "seqs": 40, "longest": 6000, "ragged": True, "mix": 5, "before": 0,
         "shift": 0, "page": 64, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "interleaved": False, "factor": 1.0},
        # one user, short context, a small tree: latency
        {"name": "tree-1x16", "kind": "tree", "seqs": 1, "longest": 600, "ragged": False, "mix": 0, "nodes": 16,
         "page": 64, "hq": 32, "hkv": 8, "d": 128},
        # a server's batch with contexts of very different lengths, and trees of different sizes
        {"name": "tree-32x24-ragged", "kind": "tree", "seqs": 32, "longest": 12001, "ragged": True, "mix": 7, "nodes": 24,
         "page": 64, "hq": 32, "hkv": 8, "d": 128},
        # large trees, small heads and pages
        {"name": "tree-8x64-d64", "kind": "tree", "seqs": 8, "longest": 4001, "ragged": True, "mix": 2, "nodes": 64,
         "page": 16, "hq": 16, "hkv": 4, "d": 64},
        # one user with a very long context and a large tree
        {"name": "tree-1x60-long", "kind": "tree", "seqs": 1, "longest": 131000, "ragged": False, "mix": 0, "nodes": 60,
         "page": 128, "hq": 32, "hkv": 8, "d": 128},
        # one user's tree of likely tokens, none drawn: latency
        {"name": "verify-1x16", "kind": "verify", "seqs": 1, "nodes": 16, "vocab": 32000, "drawn": False, "single": False,
         "temperature": 0.7, "mix": 3},
        # a server's batch of drawn trees, a large vocabulary in 32 bits
        {"name": "verify-48x24-drawn", "kind": "verify", "seqs": 48, "nodes": 24, "vocab": 128000, "drawn": True, "single": True,
         "temperature": 1.0, "mix": 4},
        # one user's accepted path: latency
        {"name": "keep-1x16", "kind": "keep", "seqs": 1, "nodes": 16, "longest": 600, "page": 64, "hkv": 8, "d": 128, "mix": 1},
        # a server's batch of accepted paths
        {"name": "keep-128x60", "kind": "keep", "seqs": 128, "nodes": 60, "longest": 500, "page": 64, "hkv": 8, "d": 128, "mix": 2},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("rotary", "append", "tree", "tree", "verify", "keep"))
    case = {"kind": kind, "mix": rng.randrange(1 << 20)}
    if kind == "verify":
        case["vocab"] = _log_int(rng, 500, 128000)
        case["seqs"] = _log_int(rng, 1, 48)
        case["nodes"] = _log_int(rng, 1, 24)
        case["drawn"] = rng.random() < 0.5
        case["single"] = rng.random() < 0.4
        case["temperature"] = rng.choice((0.0, 0.6, 1.0, 1.0))
        return case
    case["d"] = d = rng.choice((64, 128))
    case["hkv"] = rng.choice((1, 2, 4, 8))
    case["hq"] = case["hkv"] * rng.choice((1, 2, 3, 4))
    if kind in ("rotary", "append"):
        case["rot"] = rng.choice((16, 32, 48, 64, 64, d, d, d))
        case["interleaved"] = rng.random() < 0.4
        case["factor"] = rng.choice((1.0, 1.0, 4.0, 32.0))
    if kind == "rotary":
        case["dense"] = rng.random() < 0.5
        case["batch"] = rng.choice((1, 2, 3)) if case["dense"] else 1
        case["tokens"] = _log_int(rng, 1, 4096)
        case["first"] = rng.choice((0, 17, 4000000))
        return case
    case["page"] = rng.choice((16, 32, 64, 128))
    case["ragged"] = rng.random() < 0.7
    if kind == "append":
        case["seqs"] = _log_int(rng, 1, 128)
        case["longest"] = _log_int(rng, 1, 65536 // case["seqs"])
        case["before"] = rng.choice((0, 1, 37, 700))
        case["shift"] = rng.choice((0, 0, 100, 2000000))
        return case
    case["nodes"] = _log_int(rng, 2, 60)
    if kind == "tree":
        case["seqs"] = _log_int(rng, 1, 48)
        case["longest"] = _log_int(rng, 60, 131000 // case["seqs"])
    else:
        case["seqs"] = _log_int(rng, 1, 128)
        case["longest"] = _log_int(rng, 60, 500)
    return case


def _lengths(case):
    """The case's sequence lengths: all ``longest``, or that and others down to a fiftieth of it."""
    n, top = case["seqs"], case["longest"]
    if not case.get("ragged"):
        return [top] * n
    r = random.Random(case["mix"])
    return [top] + [_log_int(r, max(1, top // 50), top) for _ in range(n - 1)]


def _whole(case):
    """The lengths with the tree's nodes or the tokens held before."""
    return [m + case.get("before", 0) + case.get("nodes", 0) for m in _lengths(case)]


def _row_bytes(d):
    """Bytes of one token of one KV head: codes and scales of K and V."""
    return d + d // 8


def work(case):
    kind, d = case["kind"], case.get("d")
    if kind == "rotary":
        values = case["batch"] * case["tokens"] * (case["hq"] + case["hkv"]) * d
        return {"bytes": 2 * values * 4, "flops": 2 * values // d * case["rot"] * 3}
    if kind == "append":
        total, hq, hkv = sum(_lengths(case)), case["hq"], case["hkv"]
        bf16 = total * (hq + 2 * hkv) * d * 2 + total * (hq + 2 * hkv) * d * 2  # q, k, v in; q, and what is read back
        return {"bytes": bf16 + 2 * total * hkv * _row_bytes(d), "flops": total * ((hq + hkv) * case["rot"] * 3 + 4 * hkv * d * 3)}
    if kind == "tree":
        hq, hkv, n, whole = case["hq"], case["hkv"], case["nodes"], _whole(case)
        rows = case["seqs"] * n * hq
        return {"bytes": sum(whole) * hkv * _row_bytes(d) + rows * (d * 4 + 4), "flops": 4 * sum(_lengths(case)) * n * hq * d}
    if kind == "verify":
        # the root's row of every sequence at least: how many more are visited the inputs decide
        values = case["seqs"] * case["vocab"]
        return {"bytes": values * ((4 if case["single"] else 2) + (4 if case["drawn"] else 0)), "flops": 4 * values}
    tokens = case["seqs"] * case["nodes"] * case["hkv"]
    return {"bytes": tokens * (_row_bytes(d) * 2 + 4 * d), "flops": tokens * 2 * d}


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


def _places(state, seq, at):
    """Page, group and row of position ``at`` of sequence ``seq``."""
    page = state["page_table"][seq, (at // state["page"]).long()].long()
    at = (at % state["page"]).long()
    return page, at // GROUP, at % GROUP


def _new_tokens(state):
    """Sequence and position of every token that a packed call brings or reads."""
    n, lens = state["cu"][1:] - state["cu"][:-1], state["seq_lens"]
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n.long(), output_size=state["tokens"])
    return seq, lens[seq] - n[seq] + torch.arange(state["tokens"], device=n.device) - state["cu"][seq]


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


def _frequencies(case):
    """Radians a position of each pair; for factor > 1 pairs that turn less than once in 4096
    positions go that many times slower, those that turn over 32 times as before, the others between."""
    r, factor = case["rot"], case["factor"]
    out = []
    for i in range(r // 2):
        f = 10000.0 ** (-2.0 * i / r)
        slow = min(1.0, max(0.0, (32.0 - 4096.0 * f / (2 * math.pi)) / 31.0))
        out.append(f * (1.0 - slow) + f / factor * slow)
    return out


def _magnitude(case):
    return 1.0 + 0.1 * math.log(case["factor"])


def _turns(case):
    """The same in 2^-64 of a turn: whole numbers, taken from the exact values of the 64-bit frequencies."""
    out = []
    for f in _frequencies(case):
        num, den = f.as_integer_ratio()
        out.append(((num * TURN // den) >> 64) & ((1 << 64) - 1))
    return torch.tensor([t - (1 << 64) if t >> 63 else t for t in out], dtype=torch.int64, device="cuda")


def _tree(r, nodes, used):
    """Parents of a tree of ``used`` nodes, at most eight deep, the later ones without a node (-2)."""
    parents, depth = [-1], [0]
    for j in range(1, used):
        p = min(r.randrange(j), r.randrange(j))
        while depth[p] >= 8:
            p = r.randrange(j)
        parents.append(p)
        depth.append(depth[p] + 1)
    return parents + [-2] * (nodes - used)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cumulative(counts):
    cu = [0]
    for m in counts:
        cu.append(cu[-1] + m)
    return _int32(cu)


def prepare(case, seed):
    g, r = _generator(seed), random.Random(seed)
    kind = case["kind"]
    state = {"kind": kind}
    if kind == "verify":
        return _prepare_verify(state, case, g, r)
    d, hkv, hq = case["d"], case["hkv"], case.get("hq")
    state.update(d=d, hkv=hkv, hq=hq, scale=d ** -0.5)
    if kind in ("rotary", "append"):
        state.update(turns=_turns(case), rot=case["rot"], interleaved=case["interleaved"], magnitude=_magnitude(case))
    if kind == "rotary":
        b, n = case["batch"], case["tokens"]
        if case["dense"]:
            # heads first, each batch entry from its own first position on (documents cut into rows)
            start = torch.randint(0, 500, (b, 1), generator=g, device="cuda") + case["first"]
            state["positions"] = (start + torch.arange(n, device="cuda")).to(torch.int32)
            shapes = ((b, hq, n, d), (b, hkv, n, d))
            state["q"], state["k"], state["dq"], state["dk"] = (_normal(g, *s).bfloat16() for s in shapes + shapes)
        else:
            state["positions"] = (torch.randint(0, 4096, (n,), generator=g, device="cuda") + case["first"]).to(torch.int32)
            for names in (("q", "k"), ("dq", "dk")):
                x = _normal(g, n, (hq + 2 * hkv) * d).bfloat16()  # views of a fused projection's rows
                state[names[0]] = x[:, :hq * d].view(n, hq, d)
                state[names[1]] = x[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
        return state
    lens, whole = _lengths(case), _whole(case)
    state["page"] = case["page"]
    state["cache"], state["page_table"] = _cache(g, case, whole)
    state["seq_lens"] = _int32(whole)
    if kind == "append":
        total = sum(lens)
        state.update(cu=_cumulative(lens), tokens=total)
        x = torch.empty((total, (hq + 2 * hkv) * d), dtype=torch.bfloat16, device="cuda")
        q, k, v = x.split((hq * d, hkv * d, hkv * d), dim=1)
        q.copy_(_normal(g, total, hq * d))
        kk, vv = _keys_values(g, total, hkv, d)
        k.copy_(kk.view(total, -1))
        v.copy_(vv.view(total, -1))
        state.update(q=q.view(total, hq, d), k=k.view(total, hkv, d), v=v.view(total, hkv, d), positions=None)
        if case["shift"]:  # tokens dropped from the cache's front since: a token's position is not its place
            state["positions"] = (_new_tokens(state)[1] + case["shift"]).to(torch.int32)
        return state
    nodes, seqs = case["nodes"], case["seqs"]
    state["nodes"] = nodes
    if kind == "tree":
        used = [nodes if not case["ragged"] else r.randint(max(1, nodes // 2), nodes) for _ in range(seqs)]
        state["parents"] = _int32([_tree(r, nodes, u) for u in used])
        state["q"] = _normal(g, seqs * nodes, hq, d).bfloat16()
        return state
    # accepted paths: the root and nodes behind the places that the path will take, so that a second pass finds the same
    path, kept = [], []
    for _ in range(seqs):
        n = r.randint(1, max(1, min(8, nodes // 2)))
        path.append([0] + sorted(r.sample(range(n, nodes), n - 1)) + [-1] * (nodes - n))
        kept.append(n)
    state.update(path=_int32(path), kept=_int32(kept), cu=_cumulative([nodes] * seqs), tokens=seqs * nodes)
    return state


def _prepare_verify(state, case, g, r):
    """Target logits as wide as a language model's, a draft that comes near them, and its tree."""
    seqs, nodes, vocab = case["seqs"], case["nodes"], case["vocab"]
    parents = _int32([_tree(r, nodes, nodes if i % 5 or nodes < 3 else nodes - 2) for i in range(seqs)])
    logits = torch.empty((seqs, nodes, vocab), dtype=torch.float32 if case["single"] else torch.bfloat16, device="cuda")
    probs = torch.empty((seqs, nodes, vocab), dtype=torch.float32, device="cuda") if case["drawn"] else None
    tokens = torch.zeros((seqs, nodes), dtype=torch.int32, device="cuda")
    likely = torch.empty((seqs, nodes, min(nodes, vocab)), dtype=torch.int64, device="cuda")
    for i in range(nodes):
        base = 2.5 * _normal(g, seqs, vocab)
        logits[:, i] = base
        q = torch.softmax(base + 0.5 * _normal(g, seqs, vocab), -1)
        likely[:, i] = torch.topk(q, likely.shape[-1], dim=-1).indices
        if probs is not None:
            probs[:, i] = q
    count = torch.zeros((seqs, nodes), dtype=torch.int64, device="cuda")
    row = torch.arange(seqs, device="cuda")
    for j in range(1, nodes):
        p = parents[:, j].clamp(min=0).long()
        if probs is not None:  # drawn from the parent's distribution
            noise = torch.empty((seqs, vocab), device="cuda").exponential_(generator=g)
            tokens[:, j] = (probs[row, p] / noise).argmax(-1)
        else:                  # the parent's likeliest tokens, one after another
            tokens[:, j] = likely[row, p, count[row, p] % likely.shape[-1]]
            count[row, p] += 1
    state.update(logits=logits, tokens=tokens, parents=parents, probs=probs, temperature=case["temperature"],
                 uniforms=torch.rand((seqs, nodes), generator=g, device="cuda"))
    return state


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------
def run(state):
    return _own(state) if own else _plain(state)


def _own(state):
    from exact_attention_20_gb300 import draft, rotary, serve

    kind = state["kind"]
    if kind in ("rotary", "append"):
        rope = rotary.Rope(state["turns"], state["interleaved"], state["magnitude"])
    if kind == "rotary":
        q, k = rotary.rotate(state["q"], state["k"], rope, state["positions"])
        dq, dk = rotary.rotate_backward(state["dq"], state["dk"], rope, state["positions"])
        return q, k, dq, dk
    if kind == "append":
        q = rotary.kv4_append(state["cache"], state["q"], state["k"], state["v"], rope, state["page_table"],
                              state["seq_lens"], state["cu"], positions=state["positions"])
        return (q,) + serve.kv4_load(state["cache"], state["page_table"], state["seq_lens"], state["cu"],
                                     state["tokens"], d=state["d"])
    if kind == "tree":
        return draft.kv4_tree_attention(state["q"], state["cache"], state["page_table"], state["seq_lens"],
                                        state["parents"], scale=state["scale"])
    if kind == "verify":
        return draft.verify_tree(state["logits"], state["tokens"], state["parents"], state["uniforms"],
                                 draft_probs=state["probs"], temperature=state["temperature"])
    lens = draft.kv4_keep(state["cache"], state["page_table"], state["seq_lens"], state["path"], state["kept"],
                          d=state["d"])
    return (lens,) + serve.kv4_load(state["cache"], state["page_table"], state["seq_lens"], state["cu"],
                                    state["tokens"], d=state["d"])


def _plain(state):
    kind = state["kind"]
    if kind == "rotary":
        return (*_turned(state["q"], state, 1), *_turned(state["k"], state, 1),
                *_turned(state["dq"], state, -1), *_turned(state["dk"], state, -1))
    if kind == "append":
        return _plain_append(state)
    if kind == "tree":
        return _plain_tree(state)
    if kind == "verify":
        return _plain_verify(state)
    return _plain_keep(state)


def _cos_sin(positions, state):
    """cos and sin of each position's pairs, [..., rot/2] in 64 bits; whole numbers wrap as turns do."""
    turn = (positions.long().unsqueeze(-1) * state["turns"]).double() * (2.0 ** -64 * 2 * math.pi)
    return torch.cos(turn) * state["magnitude"], torch.sin(turn) * state["magnitude"]


def _rotate(x, c, s, state):
    """x [..., d] with its first rot elements turned; c, s broadcast to [..., rot/2]."""
    rot = state["rot"]
    y = x.clone()
    if state["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    return y


def _turned(x, state, sign):
    c, s = (t.float() for t in _cos_sin(state["positions"], state))
    axis = 1  # of the heads: [B, H, N, d] beside [B, N], or [T, H, d] beside [T]
    return (_rotate(x.float(), c.unsqueeze(axis), sign * s.unsqueeze(axis), state).bfloat16(),)


def _bf16(x):
    """64-bit values rounded to bf16 at once: through 32 bits a value near a tie could fall on it."""
    f = x.float()
    rest = x - f.double()
    i = f.view(torch.int32)
    tie = ((i & 0xffff) == 0x8000) & (rest != 0)
    i = torch.where(tie, torch.where((rest > 0) == (f > 0), i + 1, i - 1), i)
    return i.view(torch.float32).bfloat16()


def _plain_append(state):
    seq, at = _new_tokens(state)
    c, s = (t.unsqueeze(1) for t in _cos_sin(at if state["positions"] is None else state["positions"], state))
    q = _rotate(state["q"].float(), c.float(), s.float(), state).bfloat16()
    # 64 bits: a key that fell on the other side of a border of bf16 could fall to another of the 4-bit values
    k = _bf16(_rotate(state["k"].double(), c, s, state))
    place = _places(state, seq, at)
    kc, ks, vc, vs = _fields(state["cache"], state["d"])
    page, group, row = place
    kc[page, :, group, row], ks[page, :, group, row] = _quantise(k.float())
    vc[page, :, group, row], vs[page, :, group, row] = _quantise(state["v"].float())
    return (q,) + _read(state, place)


def _read(state, place):
    page, group, row = place
    kc, ks, vc, vs = _fields(state["cache"], state["d"])
    return (_dequantise(kc[page, :, group, row], ks[page, :, group, row]).bfloat16(),
            _dequantise(vc[page, :, group, row], vs[page, :, group, row]).bfloat16())


def _ancestors(parents):
    """Whether node i sees node j, [S, n, n]; a node whose line does not end at the context sees none."""
    n = parents.shape[1]
    j = torch.arange(n, device=parents.device)
    known = (parents >= 0) & (parents < j)
    step = (parents.unsqueeze(-1) == j) & known.unsqueeze(-1)
    see = (step | torch.eye(n, dtype=torch.bool, device=parents.device)).float()
    for _ in range(6):  # lines of up to 64 nodes
        see = (torch.matmul(see, see) > 0).float()
    rooted = torch.matmul(see, (parents == -1).float().unsqueeze(-1)) > 0
    return (see > 0) & rooted


def _softmax_product(s, v):
    """exp(s - max) v / sum over the last dimension of the scores s (overwritten), and the
    logsumexp; a row whose scores are all -inf gives 0 and -inf."""
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = s.sum(-1, keepdim=True)
    return torch.matmul(s, v) / torch.where(l > 0, l, 1.0), (m + torch.log(l)).squeeze(-1)


def _plain_tree(state):
    q, lens, nodes, d, hkv = state["q"], state["seq_lens"], state["nodes"], state["d"], state["hkv"]
    n, hq = lens.numel(), state["hq"]
    table = state["page_table"].long()
    kc, ks, vc, vs = (f[table].transpose(1, 2).flatten(2, 4) for f in _fields(state["cache"], d))  # [S, hkv, keys, ...]
    k, v = _dequantise(kc, ks).unsqueeze(2), _dequantise(vc, vs).unsqueeze(2)     # [S, hkv, 1, keys, d]
    qf = q.float().view(n, nodes, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3).unsqueeze(2)
    s = torch.matmul(qf, k.transpose(-1, -2)).mul_(state["scale"])                # [S, hkv, 1, G n, keys]
    see = _ancestors(state["parents"])
    keys = torch.arange(k.shape[-2], device="cuda")
    at = keys - (lens.unsqueeze(1) - nodes)                                       # [S, keys]: the node at a place
    line = torch.gather(see, 2, at.clamp(0, nodes - 1).unsqueeze(1).expand(-1, nodes, -1))
    context = (at < 0).unsqueeze(1) & see.any(-1, keepdim=True)
    hidden = ~torch.where((at < 0).unsqueeze(1), context, line & (at < nodes).unsqueeze(1))
    s.unflatten(3, (hq // hkv, nodes)).masked_fill_(hidden.view(n, 1, 1, 1, nodes, -1), -math.inf)
    o, lse = _softmax_product(s, v)
    o = o.squeeze(2).unflatten(2, (hq // hkv, nodes)).permute(0, 3, 1, 2, 4)
    lse = lse.squeeze(2).unflatten(2, (hq // hkv, nodes)).permute(1, 2, 0, 3)
    return o.reshape(n * nodes, hq, d).bfloat16(), lse.reshape(hq, n * nodes)


def _plain_verify(state):
    """In 64 bits: a token is found where a running sum passes a random number, next to a border."""
    logits, tokens, parents, u, probs = (state[x] for x in ("logits", "tokens", "parents", "uniforms", "probs"))
    seqs, nodes, vocab = logits.shape
    row = torch.arange(seqs, device="cuda")
    ids = torch.arange(vocab, device="cuda")

    def target(at):
        x = logits[row, at].double()
        if state["temperature"] == 0.0:
            return (ids == torch.max(x, -1).indices.unsqueeze(-1)).double()
        x = torch.exp((x - x.amax(-1, keepdim=True)) / state["temperature"])
        return x / x.sum(-1, keepdim=True)

    at = torch.zeros(seqs, dtype=torch.int64, device="cuda")
    left = target(at)
    path = torch.full((seqs, nodes), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    kept = torch.ones(seqs, dtype=torch.int64, device="cuda")
    for j in range(1, nodes):  # a node's children follow it, in the order in which they are tried
        child = parents[:, j] == at
        x = tokens[:, j].long()
        there = left[row, x]
        q = probs[row, at].double() if probs is not None else (ids == x.unsqueeze(-1)).double()
        taken = child & (u[:, j].double() * q[row, x] < there)
        rest = (left - q).clamp(min=0) if probs is not None else torch.where(q > 0, 0.0, left)
        total = rest.sum(-1, keepdim=True)
        rest = torch.where(total > 0, rest / torch.where(total > 0, total, 1.0), left)
        left = torch.where((child & ~taken).unsqueeze(-1), rest, left)
        at = torch.where(taken, j, at)
        path[row, kept.clamp(max=nodes - 1)] = torch.where(taken, j, path[row, kept.clamp(max=nodes - 1)]).to(torch.int32)
        kept = kept + taken
        left = torch.where(taken.unsqueeze(-1), target(at), left)
    c = torch.cumsum(left, -1)
    passed = c > u[:, :1].double() * c[:, -1:]
    return path, kept.to(torch.int32), passed.to(torch.uint8).argmax(-1).to(torch.int32)


def _plain_keep(state):
    lens, nodes, path, kept = state["seq_lens"], state["nodes"], state["path"], state["kept"]
    first = (lens - nodes).unsqueeze(1)
    col = torch.arange(nodes, device="cuda")
    source = torch.where(col < kept.unsqueeze(1), path, col)  # a place that is not taken keeps what it holds
    seq = torch.arange(lens.numel(), device="cuda").unsqueeze(1).expand(-1, nodes).reshape(-1)
    old = _places(state, seq, (first + source).reshape(-1))
    new = _places(state, seq, (first + col).reshape(-1))
    for f in _fields(state["cache"], state["d"]):
        f[new[0], :, new[1], new[2]] = f[old[0], :, old[1], old[2]]
    return (first.squeeze(1) + kept,) + _read(state, new)


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


def _nearest_bf16_64(x):
    """The bf16 value nearest to x in float64, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -126))) - 7)
    return torch.round(x / step) * step


def _rotated_64(x, positions, case, transpose):
    """x [tokens, heads, d] turned by each token's angles, as complex numbers."""
    f = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
    angle = torch.remainder(positions.double().unsqueeze(-1) * f, 2 * math.pi)
    w = torch.polar(torch.full_like(angle, _magnitude(case)), -angle if transpose else angle).unsqueeze(-2)
    out, r = x.double().clone(), case["rot"]
    pairs = out[..., :r].unflatten(-1, (r // 2, 2)) if case["interleaved"] else out[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * w)
    out[..., :r] = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return out


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


def _lines(parents):
    """Each node's line from the context, itself included, or nothing: lists of node numbers."""
    out = []
    for j, p in enumerate(parents):
        before = [] if p == -1 else out[p] if 0 <= p < j else None
        out.append(before + [j] if before or p == -1 else [])
    return out


def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    if kind == "verify":
        return _exact_verify(state)
    d, hkv = case["d"], case["hkv"]
    if kind == "rotary":
        out = []
        for name in ("q", "k", "dq", "dk"):
            x, positions = state[name], state["positions"]
            if case["dense"]:
                y = _rotated_64(x.transpose(1, 2).flatten(0, 1), positions.flatten(), case, name[0] == "d")
                out.append(y.unflatten(0, (x.shape[0], -1)).transpose(1, 2))
            else:
                out.append(_rotated_64(x, positions, case, name[0] == "d"))
        return tuple(out)
    lens, whole = _lengths(case), _whole(case)
    if kind == "append":
        at = torch.cat([torch.arange(w - m, w, device="cuda") for m, w in zip(lens, whole)]) + case["shift"]
        k = _nearest_bf16_64(_rotated_64(state["k"], at, case, False))
        return _rotated_64(state["q"], at, case, False), _stored_64(k), _stored_64(state["v"])
    nodes = case["nodes"]
    if kind == "keep":
        parts = []
        for i, w in enumerate(whole):
            k, v = _read_64(state["cache"], d, state["page_table"][i], w - nodes, nodes)
            path = state["path"][i, :int(state["kept"][i])].long()
            for t in (k, v):
                t[:path.numel()] = t[path].clone()
            parts.append((k, v))
        return None, torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    group, scale = case["hq"] // hkv, state["scale"]
    o = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((case["hq"], o.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    for i, w in enumerate(whole):
        k, v = _read_64(state["cache"], d, state["page_table"][i], 0, w)
        hidden = torch.ones((nodes, w), dtype=torch.bool)
        for j, line in enumerate(_lines(state["parents"][i].tolist())):
            if line:
                hidden[j, :w - nodes] = False
                hidden[j, [w - nodes + x for x in line]] = False
        hidden = hidden.cuda()
        rows = slice(i * nodes, (i + 1) * nodes)
        q = state["q"][rows].double()
        for h in range(hkv):
            heads = slice(h * group, (h + 1) * group)
            s = torch.einsum("ngd,md->gnm", q[:, heads], k[:, h]) * scale
            s = s.masked_fill(hidden, -math.inf)
            total = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(total == -math.inf, 0.0, total).unsqueeze(-1))
            o[rows, heads] = torch.einsum("gnm,md->ngd", p, v[:, h])
            lse[heads, rows] = total
    return o, lse


def _exact_verify(state):
    """Whole numbers, which have no other value: the walk of each sequence by lists of children."""
    logits, tokens, parents, u, probs = (state[x] for x in ("logits", "tokens", "parents", "uniforms", "probs"))
    seqs, nodes, vocab = logits.shape
    t = state["temperature"]
    paths, counts, last = [], [], []
    for i in range(seqs):
        line, par, tok, num = [0], parents[i].tolist(), tokens[i].tolist(), u[i].tolist()
        while True:
            at = line[-1]
            x = logits[i, at].double()
            if t > 0:
                p = torch.softmax(x / t, -1)
            else:
                p = torch.zeros_like(x)
                p[int(torch.nonzero(x == x.max())[0])] = 1.0
            found = None
            for j in (j for j in range(at + 1, nodes) if par[j] == at):
                q = probs[i, at].double() if probs is not None else torch.zeros_like(p).index_fill_(0, tokens[i, j:j + 1].long(), 1.0)
                if num[j] * float(q[tok[j]]) < float(p[tok[j]]):
                    found = j
                    break
                rest = torch.relu(p - q)
                if float(rest.sum()) > 0:
                    p = rest / rest.sum()
            if found is None:
                break
            line.append(found)
        c = torch.cumsum(p, -1)
        paths.append(line + [-1] * (nodes - len(line)))
        counts.append(len(line))
        last.append(int((c > num[0] * c[-1]).to(torch.uint8).argmax()))
    return _int32(paths), _int32(counts), _int32(last)
