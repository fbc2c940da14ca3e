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
