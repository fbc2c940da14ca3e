"""Which layouts fa_rotate takes: every pair of tensors that shares an element is refused, and views that do not are taken."""
import ctypes
import random

import pytest
import torch

from exact_attention_20_gb300 import build as fa_build

A, STEP, D = 1 << 40, 1 << 36, 64


@pytest.fixture(scope="module")
def rotary():
    fa_build.build()
    from exact_attention_20_gb300 import rotary as mod
    mod.lib()
    return mod


def call(rotary, q, k, q_out, k_out, B, N, hq, hk):
    """fa_rotate's status for views given as (address, (batch, token, head) strides)."""
    s = (ctypes.c_longlong * 12)(*(x for t in (q, k, q_out, k_out) for x in t[1]))
    return rotary.lib().fa_rotate(q[0], k[0], q_out[0], k_out[0], None, A + 9 * STEP, B, N, hq, hk, D, D, 0, 1.0, 0, s, 0, None)


def taken(fa, rc):
    return rc in (fa.FA_ERR_LAUNCH, fa.FA_ERR_DEVICE)  # every check is behind it: there is no GPU


pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")


def view(shape, order, at=0, base=A):
    """(address, strides) of a view whose dimensions lie in memory in `order` with the extents of `shape`, from element `at` on."""
    strides, step = [0, 0, 0], D
    for i in reversed(order):
        strides[i], step = step, step * shape[i]
    return base + 2 * at, tuple(strides)


HEADS_FIRST, TOKENS_FIRST = (0, 2, 1), (0, 1, 2)  # of (batch, token, head)


@pytest.mark.parametrize("B,N,hq,hk,more", [(2, 16, 4, 2, 2), (3, 1, 4, 2, 0), (1, 7, 1, 1, 0), (2, 5, 8, 1, 1), (5, 1, 1, 1, 1)])
@pytest.mark.parametrize("order", [HEADS_FIRST, TOKENS_FIRST, (1, 2, 0), (1, 0, 2)])
def test_heads_of_one_tensor_in_place(rotary, B, N, hq, hk, more, order):
    fa = rotary.fa
    q = view((B, N, hq + hk + more), order)
    k = (q[0] + 2 * hq * q[1][2], q[1])
    assert taken(fa, call(rotary, q, k, q, k, B, N, hq, hk))
    other = (q[0] + STEP, q[1]), (k[0] + STEP, k[1])  # and out of place, the outputs being such views
    assert taken(fa, call(rotary, q, k, *other, B, N, hq, hk))
    near = (k[0] - 2 * q[1][2], k[1])                 # k from q's last head on
    assert call(rotary, q, near, q, near, B, N, hq, hk) == fa.FA_ERR_ALIAS
    assert call(rotary, q, k, q, near, B, N, hq, hk) == fa.FA_ERR_ALIAS
    assert call(rotary, q, k, (q[0] + 16, q[1]), k, B, N, hq, hk) == fa.FA_ERR_ALIAS


def test_heads_by_turns_and_tokens_of_one_tensor(rotary):
    fa, B, N, H = rotary.fa, 2, 9, 3
    q = (A, (N * H * 2 * D, H * 2 * D, 2 * D))        # [B, N, H, 2, d]: q and k by turns
    k = (A + 2 * D, q[1])
    assert taken(fa, call(rotary, q, k, q, k, B, N, H, H))
    q = view((B, 2 * N, H), HEADS_FIRST)              # the first N tokens of each head, and the others
    k = (q[0] + 2 * N * D, q[1])
    assert taken(fa, call(rotary, q, k, q, k, B, N, H, H))
    assert call(rotary, q, (k[0] - 2 * D, k[1]), q, (k[0] - 2 * D, k[1]), B, N, H, H) == fa.FA_ERR_ALIAS


def places(t, B, N, heads):
    return {t[0] // 16 + (b * t[1][0] + n * t[1][1] + h * t[1][2]) // 8 + e
            for b in range(B) for n in range(N) for h in range(heads) for e in range(D // 8)}


def test_no_pair_that_shares_an_element_is_taken(rotary):
    fa, r, shared, apart = rotary.fa, random.Random(5), 0, 0
    for _ in range(4000):
        B, N, hq, hk = (r.randint(1, 4) for _ in range(4))
        t = []
        for heads in (hq, hk):  # any extents around, any order, sometimes the same ones
            shape = [B + r.randint(0, 1), N + r.randint(0, 2), heads + r.randint(0, 4)]
            t.append(view(shape, r.sample(range(3), 3), D * r.randint(0, 40)))
        q, k = t
        if r.random() < 0.6:
            k = (q[0] + 2 * D * r.randint(0, 12), q[1])
        rc = call(rotary, q, k, q, k, B, N, hq, hk)
        common = not places(q, B, N, hq).isdisjoint(places(k, B, N, hk))
        if common:
            assert rc in (fa.FA_ERR_ALIAS, fa.FA_ERR_INVALID_ARG), (q, k, B, N, hq, hk)
        shared += common
        apart += taken(fa, rc)
    assert shared > 1000 and apart > 800
