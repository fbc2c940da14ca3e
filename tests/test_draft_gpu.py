"""GPU tests of drafted tokens: attention of trees over the 4-bit cache, verification, keeping, and a step of all.

The attention's tolerances are those of test_kv4_gpu (its ``compare``): P is
rounded to f16, sums are fp32, as there.  Verification and keeping are compared
exactly.
"""
import math

import pytest
import torch

from exact_attention_20_gb300 import build as fa_build
from tests import draft_reference as ref
from tests import kv4_reference as kv4_ref
from tests import test_kv4_gpu as kv4

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def draft():
    fa_build.build()
    from exact_attention_20_gb300 import draft as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def serve(draft):
    from exact_attention_20_gb300 import serve as mod
    mod.lib()
    return mod


def cpu_generator(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def check_rows(o, lse, q, cache, table, lens, parents, d, page, scale, g=(1.0, 1.0)):
    nodes = len(parents[0])
    for i, n in enumerate(lens):
        k, v = kv4_ref.read(cache, d, page, table[i].tolist()[:-(-n // page)], n, *g)
        rows = slice(i * nodes, (i + 1) * nodes)
        o64, lse64, bound, most = ref.attend(q[rows], k, v, parents[i], scale)
        kv4.compare(o[rows], lse[:, rows], o64, lse64, bound, most, n, float(v.abs().max()) if n else 0.0, d)
        for j, line in enumerate(ref.lines(parents[i], n - nodes)):
            if not line:
                assert (o[i * nodes + j] == 0).all() and torch.isneginf(lse[:, i * nodes + j]).all()


def check_tree(draft, serve, lens, parents, hq, hkv, d, page, seed=0, spread=1.0, q_scale=1.0, errors_are=0):
    nodes = len(parents[0])
    cache, table, _, _ = kv4.fill(serve, lens, hkv, d, page, seed, spread=spread)
    q = (torch.randn((len(lens) * nodes, hq, d), generator=kv4.generator(seed + 1), device=DEV) * q_scale).bfloat16()
    errors = kv4.int32([0])
    scale = d ** -0.5
    o, lse = draft.kv4_tree_attention(q, cache, table, kv4.int32(lens), kv4.int32(parents), scale=scale, errors=errors)
    torch.cuda.synchronize()
    assert errors.item() == errors_are
    check_rows(o, lse, q, cache, table, lens, parents, d, page, scale)
    return q, cache, table, o, lse


# (nodes, query heads, KV heads): 1 to 512 rows of a KV head, odd ones among them
SHAPES = [(1, 1, 1), (3, 4, 2), (7, 3, 1), (16, 8, 2), (13, 10, 2), (33, 4, 1), (24, 8, 2), (64, 2, 2), (43, 3, 1), (60, 8, 2),
          (64, 8, 1), (20, 16, 1)]


@pytest.mark.parametrize("nodes,hq,hkv", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_tree_attention_matches_definition(draft, serve, nodes, hq, hkv, d):
    g = cpu_generator(nodes)
    lens = [nodes, nodes + 1, nodes + 16, nodes + 127, 700 + nodes, 2049]
    parents = [ref.tree(g, nodes, roots=1 + i % 3, absent=0 if i % 2 else min(nodes - 1, i)) for i in range(len(lens))]
    check_tree(draft, serve, lens, parents, hq, hkv, d, 64, seed=nodes)


@pytest.mark.parametrize("nodes,hq", [(9, 1), (40, 4), (64, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_shorter_than_the_tree(draft, serve, nodes, hq, d):
    # places at positions below 0 have no node, nor do their children
    g = cpu_generator(1)
    lens = [0, 1, nodes - 1, nodes, 5]
    parents = [ref.tree(g, nodes, roots=nodes // 2) for _ in lens]
    check_tree(draft, serve, lens, parents, hq, 1, d, 16, seed=2)


@pytest.mark.parametrize("nodes,hq", [(6, 1), (6, 8), (33, 4)])
def test_places_without_a_node(draft, serve, nodes, hq):
    none = [-2] * nodes
    few = [-1, 0, -5, 2, 1, 3] + [4] * (nodes - 6)      # 3 hangs on an empty place, and 5 on 3
    chain = [-1] + list(range(nodes - 1))
    wrong = [-1, 5, 2, 0, 3, 4] + [-2] * (nodes - 6)     # 1 and 2 point at themselves or behind
    lens = [300, 300, 300, 300]
    check_tree(draft, serve, lens, [none, few, chain, wrong], hq, 1, 128, 32, seed=3, errors_are=draft.BAD_TREE)


@pytest.mark.parametrize("nodes,hq,hkv,d", [(8, 8, 2, 128), (60, 8, 2, 128), (64, 4, 1, 64), (31, 4, 1, 128)])
def test_long_contexts_in_several_parts(draft, serve, nodes, hq, hkv, d):
    g = cpu_generator(4)
    lens = [30011, 64 + 17, 9000]
    check_tree(draft, serve, lens, [ref.tree(g, nodes, absent=i) for i in range(3)], hq, hkv, d, 128, seed=4)


@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("nodes", [5, 50])
def test_page_sizes(draft, serve, page, nodes):
    g = cpu_generator(5)
    lens = [nodes + 28, 1000, 4097]
    check_tree(draft, serve, lens, [ref.tree(g, nodes) for _ in lens], 8, 2, 128, page, seed=5)


@pytest.mark.parametrize("nodes,hq", [(4, 2), (40, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences(draft, serve, nodes, hq, d):
    g = cpu_generator(6)
    lens = [(i * 37) % 400 for i in range(300)] + [3000]
    check_tree(draft, serve, lens, [ref.tree(g, nodes, absent=i % 2) for i in range(301)], hq, 1, d, 32, seed=6)


@pytest.mark.parametrize("spread,q_scale", [(6.0, 4.0), (1e-3, 1.0), (1.0, 1e-6), (1.0, 3e4), (30.0, 4.0)])
@pytest.mark.parametrize("nodes", [7, 48])
def test_value_ranges(draft, serve, spread, q_scale, nodes):
    g = cpu_generator(7)
    check_tree(draft, serve, [1500, 90], [ref.tree(g, nodes) for _ in range(2)], 8, 2, 128, 64, seed=7, spread=spread,
               q_scale=q_scale)


@pytest.mark.parametrize("nodes", [6, 48])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gk,gv", [(2.0 ** -9, 2.0 ** 7), (2.0 ** 40, 2.0 ** -40)])
def test_scales_of_the_tensors(draft, serve, nodes, d, gk, gv):
    lens, hq, hkv, page = [70, 3000], 8, 2, 32
    g = kv4.generator(8)
    table, pages = kv4.layout(lens, page, 8)
    cache = serve.kv4_cache(pages, hkv, d, page).fill_(0xFF)
    k = (torch.randn((sum(lens), hkv, d), generator=g, device=DEV) * gk).bfloat16()
    v = (torch.randn((sum(lens), hkv, d), generator=g, device=DEV) * gv).bfloat16()
    serve.kv4_store(cache, k, v, table, kv4.int32(lens), kv4.cumulative(lens), k_scale=gk, v_scale=gv)
    q = torch.randn((2 * nodes, hq, d), generator=g, device=DEV).bfloat16()
    parents = [ref.tree(cpu_generator(8), nodes) for _ in lens]
    scale = d ** -0.5 / gk
    o, lse = draft.kv4_tree_attention(q, cache, table, kv4.int32(lens), kv4.int32(parents), scale=scale, k_scale=gk, v_scale=gv)
    check_rows(o, lse, q, cache, table, lens, parents, d, page, scale, (gk, gv))


@pytest.mark.parametrize("nodes,hq", [(6, 2), (40, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_values_that_are_not_finite_reach_the_nodes_that_see_them(draft, serve, nodes, hq, d):
    lens, page = [nodes + 40, nodes + 200], 16
    cache, table, k, v = kv4.fill(serve, lens, 1, d, page, seed=16)
    v, k = v.clone(), k.clone()
    v[40 + 1, 0, 20] = math.nan               # node 1 of sequence 0
    k[40 + 3, 0, 1] = math.inf                # node 3
    v[lens[0] + 17, 0, 0] = math.inf          # sequence 1's context
    k[lens[0] + 200 + 2, 0, 5] = math.nan     # its node 2
    serve.kv4_store(cache, k, v, table, kv4.int32(lens), kv4.cumulative(lens))
    parents = [[-1, 0, 0, 1, 2, 4] + [-1] * (nodes - 6), [-1, 0, 0, 1, 2, -2] + [0] * (nodes - 6)]
    q = torch.randn((2 * nodes, hq, d), generator=kv4.generator(17), device=DEV).bfloat16()
    q[nodes + 5] = math.nan                   # a place without a node
    o, lse = draft.kv4_tree_attention(q, cache, table, kv4.int32(lens), kv4.int32(parents))
    for i, n in enumerate(lens):
        kk, vv = kv4_ref.read(cache, d, page, table[i].tolist()[:-(-n // page)], n)
        rows = slice(i * nodes, (i + 1) * nodes)
        o64, lse64, _, _ = ref.attend(q[rows], kk, vv, parents[i], d ** -0.5)
        assert torch.equal(torch.isnan(o[rows]), torch.isnan(o64))
        assert torch.equal(torch.isnan(lse[:, rows]), torch.isnan(lse64))
    assert torch.isnan(o[1, :, 16:32]).all() and not torch.isnan(o[[0, 2, 4, 5]]).any() and torch.isnan(o[3]).all()
    assert (o[nodes + 5] == 0).all() and torch.isneginf(lse[:, nodes + 5]).all()


@pytest.mark.parametrize("nodes,hq", [(4, 2), (40, 4)])
def test_garbage_around_a_sequence_does_not_matter(draft, serve, nodes, hq):
    lens, d = [nodes + 5, 777 + nodes], 128
    cache, table, k, v = kv4.fill(serve, lens, 2, d, 64, seed=14)  # 0xFF elsewhere: scales that are NaN
    other = serve.kv4_cache(cache.shape[0], 2, d, 64)
    serve.kv4_store(other, k, v, table, kv4.int32(lens), kv4.cumulative(lens))
    q = torch.randn((2 * nodes, 2 * hq, d), generator=kv4.generator(15), device=DEV).bfloat16()
    parents = kv4.int32([ref.tree(cpu_generator(9), nodes) for _ in lens])
    a, b = (draft.kv4_tree_attention(q, c, table, kv4.int32(lens), parents) for c in (cache, other))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("nodes", [4, 40])
@pytest.mark.parametrize("page", [16, 32])
def test_bad_pages_and_lengths_are_skipped_and_reported(draft, serve, nodes, page):
    d, n = 128, 128 + nodes
    cache, table, _, _ = kv4.fill(serve, [n, n], 1, d, page, seed=18)
    good, table = table, table.clone()
    table[1, 2] = -3
    q = torch.randn((2 * nodes, 4, d), generator=kv4.generator(19), device=DEV).bfloat16()
    parents = [ref.tree(cpu_generator(10), nodes) for _ in range(2)]
    errors = kv4.int32([0])
    o, lse = draft.kv4_tree_attention(q, cache, table, kv4.int32([n, n]), kv4.int32(parents), errors=errors)
    assert errors.item() == draft.BAD_PAGE
    k, v = kv4_ref.read(cache, d, page, good[1].tolist(), n)
    keep = [i for i in range(n) if i // page != 2]
    o64, lse64, bound, most = ref.attend(q[nodes:], k[keep], v[keep], parents[1], d ** -0.5)
    kv4.compare(o[nodes:], lse[:, nodes:], o64, lse64, bound, most, n, float(v.abs().max()), d)
    errors.zero_()
    lens = kv4.int32([good.shape[1] * page + 1, -1])  # past the table's pages, and below zero
    o, lse = draft.kv4_tree_attention(q, cache, good, lens, kv4.int32(parents), errors=errors)
    assert errors.item() & draft.BAD_POSITION
    assert torch.isneginf(lse[:, nodes:]).all() and (o[nodes:] == 0).all()


@pytest.mark.parametrize("nodes,hq", [(2, 8), (48, 8)])
def test_repeatable_bits_and_strided_queries(draft, serve, nodes, hq):
    g = cpu_generator(11)
    lens = [9000, 5 + nodes, 3000]
    parents = [ref.tree(g, nodes) for _ in lens]
    q, cache, table, o, lse = check_tree(draft, serve, lens, parents, hq, 2, 128, 64, seed=20)
    x = torch.randn((len(lens) * nodes, (hq + 4) * 128 + 8), generator=kv4.generator(21), device=DEV).bfloat16()
    view = x[:, 8:8 + hq * 128].view(-1, hq, 128)
    view.copy_(q)
    for qq in (q, view, q):
        o2, lse2 = draft.kv4_tree_attention(qq, cache, table, kv4.int32(lens), kv4.int32(parents), scale=128 ** -0.5)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_line_is_the_newest_tokens(draft, serve):
    # a tree without branches: kv4_attention of as many queries, the same bits where the same kernel takes both
    for nodes, hq in ((4, 4), (12, 8)):
        lens = [700, nodes, 33 + nodes]
        q, cache, table, o, lse = check_tree(draft, serve, lens, [[-1] + list(range(nodes - 1))] * 3, hq, 2, 128, 64, seed=22)
        o2, lse2 = serve.kv4_attention(q, cache, table, kv4.int32(lens), n_queries=nodes, scale=128 ** -0.5)
        assert ((o.double() - o2.double()).abs() <= 2.0 ** -7 * o2.double().abs() + 2.0 ** -9).all()
        assert ((lse - lse2).abs() <= 2.0 ** -18 * lse2.abs() + 2.0 ** -20).all()


# ---------------------------------------------------------------------------
# Verification
# ---------------------------------------------------------------------------
def make_verify(seed, n, nodes, V, drawn, fp32=True, spread=2.5, near=0.5):
    g, c = kv4.generator(seed), cpu_generator(seed)
    parents = [ref.tree(c, nodes, absent=(i % 3 == 2) * min(2, nodes - 1)) for i in range(n)]
    logits = (spread * torch.randn((n, nodes, V), generator=g, device=DEV)).to(torch.float32 if fp32 else torch.bfloat16)
    q = torch.softmax(logits.float() + near * torch.randn((n, nodes, V), generator=g, device=DEV), -1)
    noise = torch.empty((n, nodes, V), device=DEV).exponential_(generator=g)
    par = torch.tensor(parents, device=DEV).clamp(min=0)
    rows = torch.gather(q, 1, par.unsqueeze(-1).expand(-1, -1, V))
    tokens = ((rows / noise).argmax(-1) if drawn else (rows * noise).argmax(-1)).int()
    u = torch.rand((n, nodes), generator=g, device=DEV)
    return logits, tokens, parents, u, q if drawn else None


def check_verify(draft, logits, tokens, parents, u, probs, temperature, seqs=None):
    path, kept, token = draft.verify_tree(logits, tokens, kv4.int32(parents), u, draft_probs=probs, temperature=temperature)
    nodes = tokens.shape[1]
    lengths = []
    for i in range(tokens.shape[0]) if seqs is None else seqs:
        want, nxt = ref.verify(logits[i], tokens[i].tolist(), parents[i], u[i].tolist(), None if probs is None else probs[i],
                               temperature)
        assert path[i].tolist() == want + [-1] * (nodes - len(want)), i
        assert kept[i].item() == len(want) and token[i].item() == nxt, i
        lengths.append(len(want))
    return lengths


@pytest.mark.parametrize("V", [1, 2, 7, 255, 256, 257, 4097, 32000, 50257, 131072, 262144])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("fp32", [True, False])
def test_verify_matches_definition(draft, V, drawn, fp32):
    n = 24 if V <= 50257 else 3
    lengths = check_verify(draft, *make_verify(V, n, 12, V, drawn, fp32), 1.0)
    assert not drawn or max(lengths) > 1  # given tokens are any, and with a large vocabulary hardly ever kept


@pytest.mark.parametrize("temperature", [0.0, 0.05, 0.7, 3.0, 1e4])
@pytest.mark.parametrize("drawn", [True, False])
def test_verify_temperatures(draft, temperature, drawn):
    check_verify(draft, *make_verify(31, 30, 9, 5000, drawn, fp32=False), temperature)


@pytest.mark.parametrize("n,nodes", [(1, 1), (1, 64), (5, 64), (200, 3), (400, 2)])
@pytest.mark.parametrize("drawn", [True, False])
def test_verify_sizes(draft, n, nodes, drawn):
    # clusters of eight CTAs to one; long and wide trees; many children refused one after another
    check_verify(draft, *make_verify(n + nodes, n, nodes, 3001, drawn, near=2.0), 1.0, range(0, n, max(1, n // 40)))


def test_verify_rows_at_any_address(draft):
    # rows that start anywhere and end within vectors; two- and three-dimensional
    V, n, nodes = 777, 6, 5
    for dtype in (torch.float32, torch.bfloat16):
        for off in range(9):
            logits, tokens, parents, u, probs = make_verify(40 + off, n, nodes, V, True)
            wide = torch.full((n * nodes, V + 16), 50.0, dtype=dtype, device=DEV)  # 50: would be the likeliest by far
            wide[:, off:off + V] = logits.view(n * nodes, V).to(dtype)
            pw = torch.full((n * nodes, V + 11), 1.0, device=DEV)
            pw[:, off:off + V] = probs.view(n * nodes, V)
            a = draft.verify_tree(wide[:, off:off + V], tokens, kv4.int32(parents), u, draft_probs=pw[:, off:off + V])
            exact = wide[:, off:off + V].contiguous().view(n, nodes, V)
            b = draft.verify_tree(exact, tokens, kv4.int32(parents), u, draft_probs=probs)
            assert all(torch.equal(x, y) for x, y in zip(a, b))
            check_verify(draft, exact, tokens, parents, u, probs, 1.0)


def test_verify_at_the_borders(draft):
    # equal logits: running sums are exact, and a number that meets one goes to the next token
    V, n = 1024, 1024
    u = torch.arange(n, device=DEV).float().view(n, 1) / V
    for dtype in (torch.float32, torch.bfloat16):
        logits = torch.full((n, 1, V), 3.0, dtype=dtype, device=DEV)
        _, kept, token = draft.verify_tree(logits, torch.zeros((n, 1), dtype=torch.int32, device=DEV), kv4.int32([[-1]] * n), u)
        assert torch.equal(token, torch.arange(n, device=DEV).int()) and (kept == 1).all()
    # a child with p = 1/4: accepted below it, not at it
    logits = torch.zeros((3, 2, 4), device=DEV)
    u = torch.tensor([[0.0, 0.25 - 2.0 ** -25], [0.0, 0.25], [1.0 - 2.0 ** -24, 0.25]], device=DEV)
    path, kept, token = draft.verify_tree(logits, kv4.int32([[9, 3]] * 3), kv4.int32([[-1, 0]] * 3), u)
    assert kept.tolist() == [2, 1, 1] and token.tolist() == [0, 0, 2]  # token 3 is out once refused
    # drawn with q = p: always accepted, up to the largest number there is
    q = torch.full((3, 2, 4), 0.25, device=DEV)
    u[:, 1] = 1.0 - 2.0 ** -24
    assert draft.verify_tree(logits, kv4.int32([[9, 3]] * 3), kv4.int32([[-1, 0]] * 3), u, draft_probs=q)[1].tolist() == [2, 2, 2]


def test_verify_logits_that_are_not_finite(draft):
    V = 300
    x = torch.randn((7, 2, V), generator=kv4.generator(50), device=DEV)
    x[0, 0, 5:] = -math.inf                     # few tokens left
    x[1, 0] = -math.inf                         # none
    x[2, 0, 17] = math.nan                      # counts as -inf
    x[3, 0, 200] = math.inf                     # has everything
    x[4, 0, 100], x[4, 0, 7] = math.inf, math.inf
    x[5, 0] = -3.4e38                           # the type's lowest values
    x[5, 0, 9] = -3.3e38
    x[6, 0], x[6, 0, 0] = math.nan, -math.inf
    tokens = kv4.int32([[0, 4], [0, 4], [0, 17], [0, 200], [0, 7], [0, 9], [0, 3]])
    parents = [[-1, 0]] * 7
    u = torch.full((7, 2), 0.6, device=DEV)
    u[0, 1] = u[4, 1] = 0.3
    check_verify(draft, x, tokens, parents, u, None, 1.0)
    path, kept, token = draft.verify_tree(x, tokens, kv4.int32(parents), u)
    assert kept.tolist()[1:4] == [1, 1, 2] and token[1] == -1 and token[6] == -1 and kept.tolist()[4:6] == [2, 2]
    check_verify(draft, x, tokens, parents, u, None, 0.0)


def test_verify_trees_without_a_root_and_bad_tokens(draft):
    V = 50
    logits, _, _, u, _ = make_verify(60, 5, 6, V, False)
    parents = [[-2, 0, 0, 1, 1, 2], [0, -1, 1, 1, 2, 2], [-1, 0, 0, -1, 3, 9], [-1, 0, -2, 2, 0, 1], [-1, 0, 0, 0, 0, 0]]
    u[2:, 1:] = 0.0  # accepts whatever has any probability
    tokens = kv4.int32([[1] * 6, [1] * 6, [0, -1, V, 3, 3, 3], [0, -1, 5, 5, 7, 8], [0, V, 2 ** 31 - 1, -2 ** 31, 11, 12]])
    path, kept, token = draft.verify_tree(logits, tokens, kv4.int32(parents), u)
    assert kept.tolist() == [0, 0, 1, 2, 2] and token.tolist()[:2] == [-1, -1]
    assert path.tolist()[3] == [0, 4, -1, -1, -1, -1] and path.tolist()[4] == [0, 4, -1, -1, -1, -1]
    check_verify(draft, logits, tokens, parents, u, None, 1.0)


def test_verify_the_same_token_twice_and_nothing_left(draft):
    # a token refused once has nothing left; where it had everything, that stays
    logits = torch.zeros((2, 4, 8), device=DEV)
    logits[1, 0, 1:] = -math.inf
    tokens = kv4.int32([[0, 5, 5, 5], [0, 0, 0, 3]])
    u = torch.full((2, 4), 1.0 - 2.0 ** -24, device=DEV)
    u[0, 2:] = 0.0
    path, kept, token = draft.verify_tree(logits, tokens, kv4.int32([[-1, 0, 0, 0]] * 2), u)
    assert kept.tolist() == [1, 2] and token.tolist() == [7, 7]  # sequence 1 walks to node 1, whose row is even
    # numbers outside [0, 1) are taken as its ends
    u = torch.tensor([[1.5, math.nan], [-1.0, 2.0], [math.inf, 1.0], [math.nan, -3.0]], device=DEV)
    path, kept, token = draft.verify_tree(torch.zeros((4, 2, 8), device=DEV), kv4.int32([[0, 5]] * 4), kv4.int32([[-1, 0]] * 4), u)
    assert kept[1:].tolist() == [1, 1, 2] and token.tolist()[1:3] == [0, 7]


def test_verify_gives_the_targets_distribution(draft):
    # the first token out, over many draws of tree and numbers, is distributed as the target's sample: 5 sigma
    n, V = 40000, 6
    g = kv4.generator(70)
    p_logits, q = torch.randn(V, generator=g, device=DEV), torch.softmax(torch.randn(V, generator=g, device=DEV), -1)
    logits = p_logits.expand(n, 4, V).contiguous()
    parents = kv4.int32([[-1, 0, 0, 0]] * n)
    drawn = torch.multinomial(q, n * 4, replacement=True, generator=g).view(n, 4).int()
    given = torch.randint(0, V, (n, 4), generator=g, device=DEV).int()
    want = torch.softmax(p_logits.double(), -1)
    for tokens, probs in ((drawn, q.expand(n, 4, V).contiguous()), (given, None)):
        u = torch.rand((n, 4), generator=g, device=DEV)
        path, kept, nxt = draft.verify_tree(logits, tokens, parents, u, draft_probs=probs)
        first = torch.where(kept > 1, torch.gather(tokens, 1, path[:, 1:2].clamp(min=0).long()).squeeze(1), nxt)
        got = torch.bincount(first.long(), minlength=V).double() / n
        assert ((got - want).abs() <= 5 * (want * (1 - want) / n).sqrt()).all(), (got, want)
        assert 0.1 < float((kept > 1).double().mean()) < 1.0


# ---------------------------------------------------------------------------
# Keeping
# ---------------------------------------------------------------------------
def check_keep(draft, serve, lens, nodes, paths, hkv, d, page, seed):
    cache, table, _, _ = kv4.fill(serve, lens, hkv, d, page, seed, garbage=0xA5)
    before = cache.clone()
    padded = [p + [-1] * (nodes - len(p)) for p in paths]
    errors = kv4.int32([0])
    new = draft.kv4_keep(cache, table, kv4.int32(lens), kv4.int32(padded), kv4.int32([len(p) for p in paths]), d, errors=errors)
    assert errors.item() == 0 and new.tolist() == [n - nodes + len(p) for n, p in zip(lens, paths)]
    for i, (n, path) in enumerate(zip(lens, paths)):
        pages = table[i].tolist()[:-(-n // page)]
        was, now = kv4_ref.read(before, d, page, pages, n), kv4_ref.read(cache, d, page, pages, n)
        for a, b in zip(was, now):
            want = a.clone()
            want[n - nodes:n - nodes + len(path)] = a[[n - nodes + j for j in path]]
            assert torch.equal(b, want)
    changed = int((before != cache).sum())
    assert changed <= sum(j != x for p in paths for j, x in enumerate(p)) * hkv * serve.kv4_row_bytes(d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("hkv", [1, 3])
def test_keep_moves_the_path(draft, serve, d, page, hkv):
    nodes = 20
    lens = [20, 21, 35, 100, 500, 40]
    paths = [[0], [0, 1, 2], [0, 3, 9, 19], [0, 2, 3, 4, 5, 11], list(range(20)), []]
    check_keep(draft, serve, lens, nodes, paths, hkv, d, page, seed=1)


def test_keep_the_largest_tree_backwards(draft, serve):
    # every row moves onto one that moves too; not a path that verification gives, but defined
    check_keep(draft, serve, [64, 300], 64, [list(range(63, -1, -1)), [5] * 64], 2, 128, 32, seed=2)


def test_keep_skips_and_reports(draft, serve):
    d, page = 128, 16
    cache, table, _, _ = kv4.fill(serve, [40, 40, 40, 40], 1, d, page, seed=3)
    before, bad = cache.clone(), table.clone()
    bad[1, 2] = 99                              # positions 32 ... of sequence 1
    errors = kv4.int32([0])
    path = kv4.int32([[0, 10, -1, 3], [0, 2, 1, 3], [0, 1, 2, 3], [2, 3, 0, 1]])
    new = draft.kv4_keep(cache, bad, kv4.int32([40, 34, 2, 70]), path, kv4.int32([3, 3, 9, -4]), d, errors=errors)
    assert errors.item() == draft.BAD_PAGE | draft.BAD_POSITION
    assert new.tolist() == [39, 33, 2, 66]
    assert torch.equal(cache[[p for p in range(cache.shape[0]) if p != int(table[1, 1])]],
                       before[[p for p in range(cache.shape[0]) if p != int(table[1, 1])]])
    k, _ = kv4_ref.read(cache, d, page, table[1].tolist(), 34)
    was, _ = kv4_ref.read(before, d, page, table[1].tolist(), 34)
    assert torch.equal(k, was)  # 30 <- 30, 31 <- 32 refused, 32 refused


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d,hq,hkv,nodes,page", [(128, 8, 2, 12, 16), (64, 8, 2, 40, 64), (128, 4, 1, 60, 32)])
@pytest.mark.parametrize("drawn", [True, False])
def test_steps_of_speculative_decoding(draft, serve, d, hq, hkv, nodes, page, drawn):
    from exact_attention_20_gb300 import rotary
    rope = rotary.rope(d)
    g, c = kv4.generator(80), cpu_generator(80)
    lens, V, room = [70, 1, 300], 64, 5 * nodes + 40
    n = len(lens)
    table, pages = kv4.layout([x + room for x in lens], page, 80)
    cache = serve.kv4_cache(pages, hkv, d, page).fill_(0xFF)
    twin = cache.clone()  # the kept tokens alone, appended one step after another
    seq = kv4.int32(lens)
    q, k, v = (torch.randn((sum(lens), h, d), generator=g, device=DEV).bfloat16() for h in (hq, hkv, hkv))
    for store in (cache, twin):
        rotary.kv4_append(store, q, k, v, rope, table, seq, kv4.cumulative(lens))
    head = torch.randn((hq * d, V), generator=g, device=DEV) * 0.3
    cu = kv4.cumulative([nodes] * n)
    errors = kv4.int32([0])
    for step in range(4):
        parents = [ref.tree(c, nodes, absent=i) for i in range(n)]
        par, depth = kv4.int32(parents), kv4.int32([ref.depths(p) for p in parents])
        q, k, v = (torch.randn((n * nodes, h, d), generator=g, device=DEV).bfloat16() for h in (hq, hkv, hkv))
        whole = seq + nodes
        positions = (seq.unsqueeze(1) + depth).flatten().int()
        qr = rotary.kv4_append(cache, q, k, v, rope, table, whole, cu, positions=positions, errors=errors)
        o, lse = draft.kv4_tree_attention(qr, cache, table, whole, par, errors=errors)
        check_rows(o, lse, qr, cache, table, whole.tolist(), parents, d, page, d ** -0.5)
        logits = (o.view(n, nodes, -1).float() @ head).bfloat16()
        probs = torch.softmax(logits.float() + 0.2 * torch.randn(logits.shape, generator=g, device=DEV), -1)
        tokens = torch.multinomial(torch.gather(probs, 1, par.clamp(min=0).long().unsqueeze(-1).expand(-1, -1, V)).flatten(0, 1), 1,
                                   generator=g).view(n, nodes).int()
        u = torch.rand((n, nodes), generator=g, device=DEV)
        u[:, 1:] *= 0.5
        path, kept, _ = draft.verify_tree(logits, tokens, par, u, draft_probs=probs if drawn else None)
        for i in range(n):
            want, _ = ref.verify(logits[i], tokens[i].tolist(), parents[i], u[i].tolist(), probs[i] if drawn else None, 1.0)
            assert path[i, :kept[i]].tolist() == want
        new = draft.kv4_keep(cache, table, whole, path, kept, d, errors=errors)
        # the same cache as if the kept tokens had been appended alone, and the same attention of the last of them
        rows = torch.tensor([i * nodes + j for i in range(n) for j in path[i, :kept[i]].tolist()], device=DEV)
        rotary.kv4_append(twin, None, k[rows], v[rows], rope, table, new, kv4.cumulative(kept.tolist()), errors=errors)
        for i, m in enumerate(new.tolist()):
            a, b = (kv4_ref.read(x, d, page, table[i].tolist()[:-(-m // page)], m) for x in (cache, twin))
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        last = torch.tensor([i * nodes + path[i, kept[i] - 1].item() for i in range(n)], device=DEV)
        o1, lse1 = serve.kv4_attention(qr[last].contiguous(), cache, table, new, errors=errors)
        assert ((o1.double() - o[last].double()).abs() <= 2.0 ** -6 * o1.double().abs() + 2.0 ** -8).all()
        assert ((lse1 - lse[:, last]).abs() <= 2.0 ** -16 * (1 + lse1.abs())).all()
        seq = new
    assert errors.item() == 0 and max(seq.tolist()[i] - lens[i] for i in range(n)) > 4


def tree_step(draft, state, stream=None):
    out = list(draft.kv4_tree_attention(*state["attention"], stream=stream))
    out += draft.verify_tree(*state["verify"][:4], draft_probs=state["verify"][4], stream=stream)
    out.append(draft.kv4_keep(*state["keep"], stream=stream))
    return out


def make_step(serve, seed, nodes=24, lens=(6000, 900, 3000), hq=8, hkv=2, d=128):
    n = len(lens)
    cache, table, _, _ = kv4.fill(serve, list(lens), hkv, d, 64, seed=seed)
    logits, tokens, parents, u, probs = make_verify(seed, n, nodes, 4000, True)
    par = kv4.int32(parents)
    q = torch.randn((n * nodes, hq, d), generator=kv4.generator(seed), device=DEV).bfloat16()
    # nodes behind the kept places, so that keeping twice is keeping once
    path = kv4.int32([[0, 10, 12, 20] + [-1] * (nodes - 4)] * n)
    return dict(attention=(q, cache, table, kv4.int32(list(lens)), par), verify=(logits, tokens, par, u, probs),
                keep=(cache, table, kv4.int32(list(lens)), path, kv4.int32([4] * n), d))


@pytest.mark.parametrize("nodes", [4 * 6, 60])
def test_streams_and_graphs_at_once(draft, serve, nodes):
    states = [make_step(serve, 90 + i, nodes) for i in range(2)]
    for s in states:
        tree_step(draft, s)  # the path's rows are where they stay
    want = [[t.clone() for t in tree_step(draft, s)] for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    runs = [[], []]
    for _ in range(5):
        for i, s in enumerate(states):
            runs[i].append(tree_step(draft, s, stream=streams[i] if i else streams[i].cuda_stream))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for got in runs[i] for a, b in zip(want[i], got))
    graphs, outs = [], []
    for s in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(tree_step(draft, s))
        graphs.append(graph)
    for _ in range(5):
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(want[i], outs[i]))


def test_a_captured_step_follows_its_inputs(draft, serve):
    s = make_step(serve, 95)
    tree_step(draft, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tree_step(draft, s)
    par, lens, u = s["attention"][4], s["attention"][3], s["verify"][3]
    for i in range(3):
        par.copy_(kv4.int32([ref.tree(cpu_generator(96 + i), 24, absent=i) for _ in range(3)]))
        lens -= 17 * i
        u.copy_(torch.rand(u.shape, generator=kv4.generator(97 + i), device=DEV))
        graph.replay()
        held = [t.clone() for t in out]
        want = tree_step(draft, s)
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_nothing_to_do(draft, serve):
    cache = serve.kv4_cache(2, 1, 64, 16)
    table, none = torch.empty((0, 1), dtype=torch.int32, device=DEV), torch.empty((0, 4), dtype=torch.int32, device=DEV)
    q = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=DEV)
    o, lse = draft.kv4_tree_attention(q, cache, table, kv4.int32([]), none)
    assert o.shape == (0, 1, 64) and lse.shape == (1, 0)
    out = draft.verify_tree(torch.empty((0, 4, 10), device=DEV), none, none, torch.empty((0, 4), device=DEV))
    assert [t.shape[0] for t in out] == [0, 0, 0]
    assert draft.kv4_keep(cache, table, kv4.int32([]), none, kv4.int32([]), 64).shape == (0,)


@pytest.mark.parametrize("nodes", [4, 40])
def test_offsets_beyond_32_bits(draft, serve, nodes):
    lens, page, hq, hkv, d = [333, 40], 64, 8, 2, 128
    near, table, _, _ = kv4.fill(serve, lens, hkv, d, page, 95)
    n = near.shape[0]
    far = torch.empty((1 << 18, *near.shape[1:]), dtype=near.dtype, device=DEV)
    shift = far.shape[0] - n
    assert far[shift:].data_ptr() - far.data_ptr() > 1 << 32
    far[shift:] = near
    q = torch.randn((2 * nodes, hq, d), generator=kv4.generator(96), device=DEV).bfloat16()
    parents = kv4.int32([ref.tree(cpu_generator(97), nodes)] * 2)
    path = kv4.int32([[0, 2, 3] + [-1] * (nodes - 3)] * 2)
    got = []
    for c, t in ((near, table), (far, table + shift)):
        got.append(draft.kv4_tree_attention(q, c, t, kv4.int32(lens), parents))
        draft.kv4_keep(c, t, kv4.int32(lens), path, kv4.int32([3, 3]), d)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.equal(far[shift:], near)


def test_logits_beyond_32_bits(draft):
    nodes, V, step = 40, 1000, 1 << 26  # the last node's row starts 5.2 GB behind the first's
    g = kv4.generator(98)
    logits = torch.randn((1, nodes, V), generator=g, device=DEV).bfloat16()
    probs = torch.softmax(torch.randn((1, nodes, V), generator=g, device=DEV), -1)
    far = torch.empty((nodes - 1) * step + V, dtype=torch.bfloat16, device=DEV).as_strided((1, nodes, V), (nodes * step, step, 1))
    far_probs = torch.empty((nodes - 1) * step + V, device=DEV).as_strided((1, nodes, V), (nodes * step, step, 1))
    far.copy_(logits), far_probs.copy_(probs)
    parents = kv4.int32([[-1] + list(range(nodes - 1))])  # one line: the walk may reach the last row
    tokens = kv4.int32([[0] + logits[0, :-1].argmax(-1).tolist()])
    for p, fp, u in ((None, None, 0.0), (probs, far_probs, 0.0), (None, None, 0.999), (probs, far_probs, 0.999)):
        us = torch.full((1, nodes), u, device=DEV)
        a, b = draft.verify_tree(logits, tokens, parents, us, p), draft.verify_tree(far, tokens, parents, us, fp)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert u > 0 or a[1].tolist() == [nodes]


@pytest.mark.parametrize("nodes,hq", [(4, 4), (24, 8)])
def test_a_padded_batch_is_the_batch(draft, serve, nodes, hq):
    hkv, d, page, V = 2, 64, 16, 500
    lens = [130, 57]
    cache, table, _, _ = kv4.fill(serve, lens, hkv, d, page, 99)
    g = kv4.generator(100)
    q = torch.randn((2 * nodes, hq, d), generator=g, device=DEV).bfloat16()
    logits = torch.randn((2, nodes, V), generator=g, device=DEV)
    tokens = torch.randint(0, V, (2, nodes), generator=g, device=DEV).int()
    u = torch.rand((2, nodes), generator=g, device=DEV)
    parents = kv4.int32([ref.tree(cpu_generator(s), nodes) for s in (101, 102)])
    twin = cache.clone()
    errors = kv4.int32([0])

    def step(cache, q, table, lens, parents, logits, tokens, u):
        o, lse = draft.kv4_tree_attention(q, cache, table, lens, parents, errors=errors)
        path, kept, nxt = draft.verify_tree(logits, tokens, parents, u)
        return o, lse, path, kept, nxt, draft.kv4_keep(cache, table, lens, path, kept, d, errors=errors)

    def padded(x, fill, rows=1):  # the sequences at 1 and 3 of 5
        out = torch.full((5 * rows, *x.shape[1:]), fill, dtype=x.dtype, device=DEV)
        out[rows:2 * rows], out[3 * rows:4 * rows] = x[:rows], x[rows:]
        return out

    want = step(cache, q, table, kv4.int32(lens), parents, logits, tokens, u)
    got = step(twin, padded(q, math.nan, nodes), padded(table, -1), padded(kv4.int32(lens), 0), padded(parents, -2),
               padded(logits, math.nan), padded(tokens, -7), padded(u, math.nan))
    assert errors.item() == 0 and torch.equal(twin, cache)
    for i, (a, b) in enumerate(zip(want, got)):
        axis, rows = (1, nodes) if i == 1 else (0, nodes if i == 0 else 1)
        a, b = a.movedim(axis, 0), b.movedim(axis, 0)
        assert torch.equal(a, torch.cat([b[rows:2 * rows], b[3 * rows:4 * rows]]))
        rest = torch.cat([b[:rows], b[2 * rows:3 * rows], b[4 * rows:]])
        assert (rest == (0, -math.inf, -1, 0, -1, 0)[i]).all()


@pytest.mark.parametrize("offset,temperature", [(3e4, 1.0), (-3e4, 1.0), (1e6, 1.0), (-1e6, 20.0), (8.0, 1e-3), (11350.0, 1.0), (-11360.0, 1.0),
                                                (5675.0, 0.5), (1e30, 1e26), (-300.0, 1e4)])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("fp32", [True, False])
def test_verify_logits_far_from_zero(draft, offset, temperature, drawn, fp32):
    # on both sides of where differences to the maximum are taken first (11356.5 temperatures)
    logits, tokens, parents, u, probs = make_verify(103, 12, 8, 3001, drawn)
    logits = (logits.double() * temperature + offset).to(torch.float32 if fp32 else torch.bfloat16)
    check_verify(draft, logits, tokens, parents, u, probs, temperature)


@pytest.mark.parametrize("V", [999, 20000, 131072])
@pytest.mark.parametrize("drawn", [True, False])
def test_verify_does_not_depend_on_how_it_is_divided(draft, V, drawn):
    # many sequences at once (fewer threads each) and one by one; part of a wider row, whose tiles begin elsewhere
    n, nodes = 70, 6
    logits, tokens, parents, u, probs = make_verify(104, n, nodes, V, drawn)
    parents = kv4.int32(parents)
    want = draft.verify_tree(logits, tokens, parents, u, draft_probs=probs)
    for i in range(0, n, 3):
        one = slice(i, i + 1)
        got = draft.verify_tree(logits[one], tokens[one], parents[one], u[one], draft_probs=None if probs is None else probs[one])
        assert all(torch.equal(a[one], b) for a, b in zip(want, got))
    wide = torch.full((n, nodes, V + 5), math.nan, device=DEV)
    wide[..., 5:] = logits
    got = draft.verify_tree(wide.view(n * nodes, V + 5)[:, 5:], tokens, parents, u,
                            draft_probs=None if probs is None else probs.view(n * nodes, V))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("nodes,hq", [(8, 1), (9, 1), (3, 4), (5, 3), (16, 1), (17, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[600, 3], [2000], [3000, 1, 0, 700, 2500, 2999, 129, 64, 4000]])
def test_few_rows_over_little_and_much(draft, serve, nodes, hq, d, lens):
    # on both sides of where the tensor core's tiles take over
    parents = [ref.tree(cpu_generator(105 + i), nodes, roots=1 + i % 2) for i in range(len(lens))]
    check_tree(draft, serve, lens, parents, hq, 1, d, 64, seed=106)
