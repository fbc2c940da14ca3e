"""GPU tests of drafted tokens where clusters, masks and kernels meet their ends; definitions and helpers of test_draft_gpu."""
import pytest
import torch

from exact_attention_20_gb300 import build as fa_build
from tests import test_draft_gpu as plain
from tests import test_kv4_gpu as kv4

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def draft():
    fa_build.build()
    from exact_attention_20_gb300 import draft as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("V", [3000, 9000, 40000])
@pytest.mark.parametrize("drawn", [True, False])
def test_clusters_with_and_without_a_walk(draft, V, drawn):
    # clusters of 2, 8 and 16 CTAs, more of them than the card holds: walks of no pass beside walks of several
    n, nodes = 300, 5
    logits, tokens, parents, u, probs = plain.make_verify(200, n, nodes, V, drawn)
    for i in range(0, n, 2):
        parents[i] = [-2] * nodes if i % 4 else [0] + parents[i][1:]
    path, kept, token = draft.verify_tree(logits, tokens, kv4.int32(parents), u, draft_probs=probs)
    assert (kept[::2] == 0).all() and (token[::2] == -1).all() and (path[::2] == -1).all()
    plain.check_verify(draft, logits, tokens, parents, u, probs, 1.0, range(1, n, 14))
    none = draft.verify_tree(logits, tokens, kv4.int32([[-2] * nodes] * n), u, draft_probs=probs)
    assert (none[0] == -1).all() and (none[1] == 0).all() and (none[2] == -1).all()


@pytest.mark.parametrize("V", [300, 9000])
@pytest.mark.parametrize("fp32", [True, False])
def test_drawn_children_that_cannot_come(draft, V, fp32):
    # (the child's target logit against the row's largest, its q, its number, whether it is kept): u q(x) < r(x)
    inf, nan = float("inf"), float("nan")
    cases = [(-inf, 0.1, 0.0, False), (nan, 0.1, 0.0, False), (-inf, 0.0, 0.9, False), (nan, 0.0, 0.9, False),
             (-60.0, 1e-23, 0.9, False), (-60.0, 0.0, 0.9, True), (-60.0, 0.5, 0.0, True), (-40.0, 0.0, 0.9, True),
             (-200.0, 1e-30, 0.9, False), (-1.0, 0.0, 0.9, True)]
    n = 2 * len(cases)
    g = kv4.generator(210)
    logits = torch.randn((n, 3, V), generator=g, device=DEV)
    probs = torch.full((n, 3, V), 0.4 / V, device=DEV)
    u = torch.full((n, 3), 0.5, device=DEV)
    x, y = 17, V - 20
    tokens, parents = [], []
    for i, (logit, q, number, _) in enumerate(cases * 2):
        after = i >= len(cases)  # after a child that is refused: half of q is at it, and little of p
        logits[i, 0, x], probs[i, 0, x] = float(logits[i, 0].max()) + logit, q
        logits[i, 0, y], probs[i, 0, y] = -2.0, 0.5
        u[i, 1], u[i, 2] = (0.999, number) if after else (number, 0.5)
        tokens.append([0, y, x] if after else [0, x, -1])
        parents.append([-1, 0, 0])
    logits = logits.to(torch.float32 if fp32 else torch.bfloat16)
    lengths = plain.check_verify(draft, logits, kv4.int32(tokens), parents, u, probs, 1.0)
    assert [a == 2 for a in lengths[:len(cases)]] == [c[3] for c in cases]
    path = draft.verify_tree(logits, kv4.int32(tokens), kv4.int32(parents), u, draft_probs=probs)[0]
    kept = [row[1] == 2 for row in path[len(cases):].tolist()]
    # what is left of a child is max(r - q, 0): of those with a q of their own above their r, nothing
    assert kept == [c[3] and c[1] == 0.0 for c in cases] and not (path[len(cases):, 1] == 1).any()


def test_numbers_outside_the_unit_interval_of_drawn_children(draft):
    # they are taken as its ends, as those of given children are: below 0 and NaN as 0, from 1 on as 1
    V = 64
    u = torch.tensor([-1.0, float("nan"), -float("inf"), 0.0, 1.0, 7.0, float("inf")] * 3, device=DEV)
    n = u.numel()
    logits = torch.zeros((n, 2, V), device=DEV)
    logits[:7, 0, 9] = -float("inf")               # a child that cannot come,
    probs = torch.full((n, 2, V), 1.0 / V, device=DEV)
    probs[7:14, 0, 9] = 0.5 / V                    # one that always comes,
    probs[14:, 0, 9] = 2.0 / V                     # and one that comes below 1/2
    numbers = torch.stack((torch.full_like(u, 0.3), u), 1)
    kept = draft.verify_tree(logits, kv4.int32([[0, 9]] * n), kv4.int32([[-1, 0]] * n), numbers, draft_probs=probs)[1].tolist()
    assert kept == [1] * 7 + [2] * 7 + [2, 2, 2, 2, 1, 1, 1]


@pytest.mark.parametrize("nodes,hq,hkv", [(4, 4, 2), (1, 8, 1), (3, 4, 2), (5, 3, 1), (16, 1, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_line_in_the_decode_kernel_is_the_newest_tokens_bit_by_bit(draft, nodes, hq, hkv, d):
    # up to 8 rows of a KV head, and up to 16 over many contexts: the kernel that kv4_attention takes, with another mask
    from exact_attention_20_gb300 import serve
    lens = [700, nodes, 33 + nodes, 4000, 9001] + [3000 + 7 * i for i in range(60)] * (nodes * hq // hkv > 8)
    cache, table, _, _ = kv4.fill(serve, lens, hkv, d, 64, 220)
    q = torch.randn((len(lens) * nodes, hq, d), generator=kv4.generator(221), device=DEV).bfloat16()
    line = kv4.int32([[-1] + list(range(nodes - 1))] * len(lens))
    o, lse = draft.kv4_tree_attention(q, cache, table, kv4.int32(lens), line)
    o2, lse2 = serve.kv4_attention(q, cache, table, kv4.int32(lens), n_queries=nodes)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
