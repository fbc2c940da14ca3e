"""GPU tests of rotary positions on views of one tensor, in place and as outputs: the same bits as apart."""
import pytest
import torch

from exact_attention_20_gb300 import build as fa_build
from tests import test_kv4_gpu as kv4

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def rotary():
    fa_build.build()
    from exact_attention_20_gb300 import rotary as mod
    mod.lib()
    return mod


def heads_first(x, B, N, hq, hk, d):        # [B, heads, N, d]
    return x.view(B, hq + hk + 1, N, d)[:, :hq], x.view(B, hq + hk + 1, N, d)[:, hq:hq + hk]


def rows(x, B, N, hq, hk, d):               # [B, N, heads, d] as a projection leaves it
    y = x.view(B, N, hq + hk + 1, d)
    return y[:, :, :hq].transpose(1, 2), y[:, :, hq:hq + hk].transpose(1, 2)


def one_token(x, B, N, hq, hk, d):          # [B, heads * d]: a step's rows, whose token stride says nothing
    y = x.view(B * N, (hq + hk + 1) * d)
    return y[:, :hq * d].view(B * N, hq, 1, d), y[:, hq * d:(hq + hk) * d].view(B * N, hk, 1, d)


def by_turns(x, B, N, hq, hk, d):           # [B, N, heads, 2, d]
    y = x[:B * N * hq * 2 * d].view(B, N, hq, 2, d)
    return y[:, :, :, 0].transpose(1, 2), y[:, :, :, 1].transpose(1, 2)


@pytest.mark.parametrize("layout", [heads_first, rows, one_token, by_turns])
@pytest.mark.parametrize("B,N,hq,hk,d", [(2, 33, 4, 2, 128), (3, 1, 6, 3, 64), (64, 1, 8, 8, 128)])
@pytest.mark.parametrize("rot,interleaved", [(64, False), (32, True)])
def test_views_of_one_tensor(rotary, layout, B, N, hq, hk, d, rot, interleaved):
    rope = rotary.rope(rot, interleaved=interleaved)
    x = torch.randn(B * N * max(hq + hk + 1, 2 * hq) * d, generator=kv4.generator(B), device=DEV).bfloat16()
    x = x[:B * N * (hq + hk + 1) * d] if layout is not by_turns else x
    q, k = layout(x, B, N, hq, hk, d)
    pos = torch.randint(0, 10 ** 6, (q.shape[2],), generator=kv4.generator(1), device=DEV).int()
    want = rotary.rotate(q.contiguous(), k.contiguous(), rope, pos)
    other = torch.full_like(x, 7.0)
    out = layout(other, B, N, hq, hk, d)
    rotary.fa_rotate(q, k, *out, rope, pos)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    held = x.clone()
    rotary.fa_rotate(q, k, q, k, rope, pos)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    for a, b, was in zip(layout(held, B, N, hq, hk, d), out, (q, k)):  # everything else stays as it was
        a.copy_(was)
        b.fill_(7.0)
    assert torch.equal(held, x) and (other == 7.0).all()
    rotary.fa_rotate(q, k, q, k, rope, pos, backward=True)
    back = rotary.rotate_backward(*want, rope, pos)
    assert torch.equal(q, back[0]) and torch.equal(k, back[1])
