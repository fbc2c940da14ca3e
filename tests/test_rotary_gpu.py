"""GPU tests of rotary positions: turning queries, keys and gradients, and appending to the 4-bit cache.

Tolerance of a turned value y of a pair (a, b): its rounding to bf16 is 2^-8
|y| (below the normal range 2^-134); before it, cos and sin are off by 2^-23.3
(the turn rounded to fp32) and 2^-23 (the functions, and the product with m),
two products and a sum by 2^-23 together: 2^-21 m (|a| + |b|) at the most.

Appended keys are rounded to bf16 from a sum right to about 2^-42 and are
compared bit for bit with the definition in 64 bits; so is what is stored.
"""
import math

import pytest
import torch

from exact_attention_20_gb300 import build as fa_build
from tests import kv4_reference as kv4_ref
from tests import rotary_reference as ref
from tests import test_kv4_gpu as kv4

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def rotary():
    fa_build.build()
    from exact_attention_20_gb300 import rotary as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def serve(rotary):
    return rotary.serve


def normal(seed, *shape):
    return torch.randn(shape, generator=kv4.generator(seed), device=DEV).bfloat16()


def compare(y, want, size):
    err = (y.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -134 + 2.0 ** -21 * size
    assert (err <= tol).all(), (err - tol).max().item()


ROPES = [(16, False, {}), (16, True, {}), (48, False, {}), (64, True, {}), (64, False, dict(scaling="linear", factor=4.0)),
         (64, False, dict(scaling="base", factor=8.0))]
ROPES = [(d, *r) for d in (64, 128) for r in ROPES + [(128, False, {}), (128, True, dict(scaling="parts", factor=16.0))] if r[0] <= d]


@pytest.mark.parametrize("d,rot,interleaved,scaling", ROPES)
@pytest.mark.parametrize("hq,hk,T", [(1, 1, 1), (8, 2, 37), (3, 3, 700), (5, 1, 16)])
def test_tokens_first(rotary, d, rot, interleaved, scaling, hq, hk, T):
    rope = rotary.rope(rot, interleaved=interleaved, **scaling)
    q, k = normal(1, T, hq, d), normal(2, T, hk, d)
    pos = torch.randint(0, 100000, (T,), generator=kv4.generator(3), device=DEV).int()
    pos[0] = 2 ** 31 - 1
    for backward, f in ((False, rotary.rotate), (True, rotary.rotate_backward)):
        yq, yk = f(q, k, rope, pos)
        compare(yq, *ref.rotate(q, pos, rope, backward))
        compare(yk, *ref.rotate(k, pos, rope, backward))
        assert torch.equal(yq[..., rot:], q[..., rot:]) and torch.equal(f(q, None, rope, pos), yq)


@pytest.mark.parametrize("B,hq,hk,N,d", [(1, 1, 1, 1, 64), (2, 4, 2, 129, 128), (3, 2, 2, 17, 64), (2, 3, 1, 2000, 128)])
@pytest.mark.parametrize("positions", ["none", "shared", "each"])
def test_heads_first(rotary, B, hq, hk, N, d, positions):
    rope = rotary.rope(d)
    q, k = normal(4, B, hq, N, d), normal(5, B, hk, N, d)
    each = torch.arange(N, device=DEV).int().repeat(B, 1)
    pos = None
    if positions == "shared":
        pos = torch.randint(-5, 10 ** 7, (N,), generator=kv4.generator(6), device=DEV).int()
        each = pos.repeat(B, 1)
    elif positions == "each":
        pos = each = torch.randint(-5, 10 ** 7, (B, N), generator=kv4.generator(6), device=DEV).int()
    yq, yk = rotary.rotate(q, k, rope, pos)
    for x, y in ((q, yq), (k, yk)):
        for b in range(B):
            want, size = ref.rotate(x[b].transpose(0, 1), each[b], rope)
            compare(y[b].transpose(0, 1), want, size)


def test_far_positions_lose_nothing(rotary):
    # position p + a whole number of the first pair's turns: the turns' low bits matter, not the position's size
    rope = rotary.rope(128)
    pos = torch.tensor([2 ** 31 - 1, 2 ** 31 - 2, 10 ** 9 + 7, -2 ** 31, -1], device=DEV).int()
    x = torch.zeros((5, 1, 128), device=DEV)
    x[..., :64] = 1.0  # cos and sin themselves
    y = rotary.rotate(x.bfloat16(), None, rope, pos)
    compare(y, *ref.rotate(x.bfloat16(), pos, rope))
    f = rotary.frequencies(128)
    for i in range(5):  # and against radians, in 64 bits with the product's error bounded
        angle = [math.fmod(pos[i].item() * w, 2 * math.pi) for w in f]
        want = torch.tensor([math.cos(a) for a in angle], dtype=torch.float64, device=DEV)
        assert ((y[i, 0, :64].double() - want).abs() <= 2.0 ** -8 + 2.0 ** -20).all()


def test_strided_views_and_in_place(rotary):
    T, hq, hk, d = 90, 6, 2, 128
    rope = rotary.rope(64, interleaved=True)
    x = torch.randn((T, (hq + 2 * hk) * d + 8), generator=kv4.generator(7), device=DEV).bfloat16()
    q, k = x[:, 8:8 + hq * d].view(T, hq, d), x[:, 8 + hq * d:8 + (hq + hk) * d].view(T, hk, d)
    want = rotary.rotate(q.contiguous(), k.contiguous(), rope)
    got = rotary.rotate(q, k, rope)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    rest = x[:, 8 + (hq + hk) * d:].clone()
    rotary.fa_rotate(q, k, q, k, rope)  # in place, columns of the same rows
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(x[:, 8 + (hq + hk) * d:], rest)
    q4 = normal(8, 2, 5, 33, 64)
    want = rotary.rotate(q4, None, rope)
    flip = q4.transpose(1, 2).contiguous().transpose(1, 2)  # tokens first in memory
    assert torch.equal(rotary.rotate(flip, None, rope), want)
    rotary.fa_rotate(flip, None, flip, None, rope)
    assert torch.equal(flip, want)
    out = torch.full((2, 5, 40, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    rotary.fa_rotate(q4, None, out[:, :, 3:36], None, rope)
    assert torch.equal(out[:, :, 3:36], want) and (out[:, :, :3] == 7).all() and (out[:, :, 36:] == 7).all()
    one = normal(9, 1, 1, 33, 64).expand(2, 5, 33, 64)  # a broadcast input
    assert torch.equal(rotary.rotate(one, None, rope), rotary.rotate(one.contiguous(), None, rope))


def test_backward_is_the_gradient(rotary):
    # by differences: a turn is linear, so a step of any size gives the gradient of sum(w * y) but for y's roundings
    T, H, d = 5, 2, 64
    rope = rotary.rope(48, scaling="parts", factor=8.0)
    x, w = normal(10, T, H, d), normal(11, T, H, d)
    pos = torch.arange(100, 100 + T, device=DEV).int()
    grad = rotary.rotate_backward(w, None, rope, pos)
    compare(grad, *ref.rotate(w, pos, rope, backward=True))
    g = kv4.generator(12)
    for _ in range(20):
        t, h, e = (int(torch.randint(0, n, (1,), generator=g, device=DEV)) for n in (T, H, d))
        up, down = x.clone(), x.clone()
        up[t, h, e], down[t, h, e] = 64.0, -64.0
        a, b = rotary.rotate(up, None, rope, pos).double(), rotary.rotate(down, None, rope, pos).double()
        step = ((a - b) * w.double()).sum().item() / 128.0
        # two values of magnitude up to 64 m (|a| + |b| <= 68 m) enter, each rounded to bf16 twice
        tol = 2 * 2 * (2.0 ** -8 + 2.0 ** -20) * 68 * rope.magnitude * w.double().abs().max().item() / 128.0
        assert abs(step - grad[t, h, e].item()) <= tol + 2.0 ** -8 * abs(step)


def test_values_that_are_not_finite(rotary):
    x = normal(13, 4, 1, 64)
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 63] = math.inf, math.nan, -math.inf
    rope = rotary.rope(32)
    y = rotary.rotate(x, None, rope, torch.tensor([0, 5, 9, 9], device=DEV).int())
    assert not torch.isfinite(y[0, 0, 3]) and not torch.isfinite(y[0, 0, 19])
    keep = [e for e in range(32) if e not in (3, 19)]
    assert torch.isfinite(y[0, 0, keep]).all() and torch.isnan(y[1, 0, 40]) and y[2, 0, 63] == -math.inf
    assert torch.isfinite(y[1, 0, :32]).all() and torch.isfinite(y[3]).all()
    big = torch.full((1, 1, 64), 3.0e38, dtype=torch.bfloat16, device=DEV)  # a sum past bf16's range
    y = rotary.rotate(big, None, rotary.rope(64), torch.tensor([-1], device=DEV).int())
    assert torch.isinf(y[0, 0, 0]) or y[0, 0, 0].abs() > 3e38


def test_nothing_to_do(rotary):
    rope = rotary.rope(64)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    assert rotary.rotate(none, None, rope).shape == (0, 2, 64)
    none = torch.empty((2, 2, 0, 64), dtype=torch.bfloat16, device=DEV)
    assert rotary.rotate(none, none, rope)[1].shape == (2, 2, 0, 64)


# ---------------------------------------------------------------------------
# Appending
# ---------------------------------------------------------------------------
def check_append(rotary, before, new, hq, hkv, d, page, rope, seed, shift=None, behind=0, strided=False, scales=(1.0, 1.0)):
    serve = rotary.serve
    lens = [a + b for a, b in zip(before, new)]
    T = sum(new) + behind
    table, pages = kv4.layout(lens, page, seed)
    cache = serve.kv4_cache(pages, hkv, d, page).fill_(0xA5)
    twin = cache.clone()
    x = torch.randn((T, (hq + 2 * hkv) * d + 8), generator=kv4.generator(seed), device=DEV)
    x[:, hq * d:(hq + hkv) * d] *= torch.exp(torch.randn(hkv * d, generator=kv4.generator(seed + 1), device=DEV))
    x = x.bfloat16()
    q, k, v = (x[:, a:b].view(T, -1, d) for a, b in ((0, hq * d), (hq * d, (hq + hkv) * d), ((hq + hkv) * d, (hq + 2 * hkv) * d)))
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    place = torch.tensor([p for a, b in zip(before, new) for p in range(a, a + b)] + [0] * behind).int()
    pos = place if shift is None else place + shift
    q_out, k_out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((T, hkv, d), 7.0, dtype=torch.bfloat16, device=DEV)
    args = (table, kv4.int32(lens), kv4.cumulative(new))
    errors = kv4.int32([0])
    rotary.fa_kv4_append(cache, q, k, v, rope, *args, q_out, k_out, positions=None if shift is None else pos.to(DEV),
                         k_scale=scales[0], v_scale=scales[1], errors=errors)
    assert errors.item() == 0
    n = sum(new)
    want, size = ref.rotate(q[:n], pos[:n].to(DEV), rope)
    compare(q_out[:n], want, size)
    want, _ = ref.rotate(k[:n], pos[:n].to(DEV), rope)
    assert torch.equal(k_out[:n], ref.bf16(want))
    assert (q_out[n:] == 7).all() and (k_out[n:] == 7).all()
    # what is stored is what storing the turned keys stores; every other byte stays
    serve.kv4_store(twin, ref.bf16(want).contiguous() if n else k[:0], v[:n], *args, k_scale=scales[0], v_scale=scales[1])
    assert torch.equal(cache, twin)
    kk, vv = serve.kv4_load(cache, *args, T, d, k_scale=scales[0], v_scale=scales[1])
    assert torch.equal(kk[:n].double(), kv4_ref.stored(ref.bf16(want), scales[0]))
    assert torch.equal(vv[:n].double(), kv4_ref.stored(v[:n], scales[1]))
    # without q, and the allocating form
    other = twin.clone().fill_(0xA5)
    none, again = rotary.kv4_append(other, None, k, v, rope, *args, positions=None if shift is None else pos.to(DEV), return_k=True,
                                    k_scale=scales[0], v_scale=scales[1])
    assert none is None and torch.equal(again[:n], k_out[:n]) and torch.equal(other, cache)


@pytest.mark.parametrize("d,rot,interleaved,scaling", ROPES)
def test_append_is_rotate_and_store(rotary, d, rot, interleaved, scaling):
    rope = rotary.rope(rot, interleaved=interleaved, **scaling)
    check_append(rotary, [0, 5, 31, 100, 0], [17, 1, 3, 0, 200], 4, 2, d, 16, rope, seed=rot, behind=3)
    check_append(rotary, [700] * 20, [1] * 20, 6, 3, d, 64, rope, seed=rot + 1, shift=10 ** 6, strided=True)


@pytest.mark.parametrize("hq,hkv,page", [(1, 1, 1024), (12, 4, 32), (8, 8, 128)])
def test_append_many_tokens(rotary, hq, hkv, page):
    check_append(rotary, [3, 0, 500], [2500, 1, 3001], hq, hkv, 128, page, rotary.rope(128), seed=20, scales=(2.0 ** -3, 2.0 ** 5))


def test_append_to_more_sequences_than_shared_memory_holds(rotary):
    new = [(i * 5) % 4 for i in range(5000)]
    check_append(rotary, [i % 7 for i in range(5000)], new, 1, 1, 64, 16, rotary.rope(32, interleaved=True), seed=21)


def test_append_skips_and_reports_bad_places(rotary, serve):
    d = 64
    rope = rotary.rope(d)
    x = torch.ones((6, 1, d), dtype=torch.bfloat16, device=DEV)
    cache = serve.kv4_cache(4, 1, d, 16).fill_(0x5A)
    table, cu, errors = kv4.int32([[0, 4], [1, 2], [-1, 3]]), kv4.int32([0, 2, 4, 6]), kv4.int32([0])
    pos = torch.arange(6, device=DEV).int()
    q, k = rotary.kv4_append(cache, x, x, x, rope, table, kv4.int32([18, 1, 2]), cu, positions=pos, return_k=True, errors=errors)
    assert errors.item() == serve.BAD_PAGE | serve.BAD_POSITION
    assert (cache[[0, 2, 3]] == 0x5A).all() and 0 < int((cache[1] != 0x5A).sum()) <= serve.kv4_row_bytes(d)
    want, size = ref.rotate(x, pos, rope)  # turned all the same
    compare(q, want, size)
    assert torch.equal(k, ref.bf16(want))


def test_append_of_values_that_are_not_finite(rotary, serve):
    d, n = 128, 8
    k, v = normal(22, n, 1, d), normal(23, n, 1, d)
    k[1, 0, 5], k[2, 0, 100], v[3, 0, 17] = math.inf, math.nan, -math.inf
    table, pages = kv4.layout([n], 16)
    cache = serve.kv4_cache(pages, 1, d, 16)
    args = (table, kv4.int32([n]), kv4.int32([0, n]))
    _, kr = rotary.kv4_append(cache, None, k, v, rotary.rope(128), *args, return_k=True)
    kk, vv = serve.kv4_load(cache, *args, n, d)
    bad = ~torch.isfinite(kr).view(n, 1, 8, 16).all(-1, keepdim=True).expand(-1, -1, -1, 16).flatten(-2)
    assert torch.equal(torch.isnan(kk), bad) and bad[1, 0, 0] and bad[1, 0, 64] and bad[2, 0, 32] and bad[2, 0, 96]
    assert int(bad.sum()) == 64 and int(torch.isnan(vv).sum()) == 16


def test_streams_and_a_captured_step(rotary, serve):
    d, hq, hkv = 128, 8, 2
    rope = rotary.rope(128)
    table, pages = kv4.layout([90, 90], 16, 24)
    cache = serve.kv4_cache(pages, hkv, d, 16)
    lens, cu = kv4.int32([60, 30]), kv4.int32([0, 1, 2])
    q, k, v = normal(25, 2, hq, d), normal(26, 2, hkv, d), normal(27, 2, hkv, d)
    side = torch.cuda.Stream()
    want = rotary.kv4_append(cache, q, k, v, rope, table, lens, cu)
    bytes_ = cache.clone()
    cache.zero_()
    torch.cuda.synchronize()
    got = rotary.kv4_append(cache, q, k, v, rope, table, lens, cu, stream=side)
    rot = rotary.rotate(q, k, rope, lens - 1, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(rot[0], want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = rotary.kv4_append(cache, q, k, v, rope, table, lens, cu)
    cache.zero_()
    g.replay()
    assert torch.equal(out, want) and torch.equal(cache, bytes_ )
    lens += 1
    g.replay()
    assert torch.equal(out, rotary.rotate(q, None, rope, lens - 1))


def test_offsets_beyond_32_bits(rotary, serve):
    T, step = 140, 1 << 24  # the last token's row starts 4.7 GB behind the first's
    rope = rotary.rope(64, interleaved=True)
    q, k = normal(90, T, 3, 128), normal(91, T, 2, 128)
    far = torch.empty((T - 1) * step + 5 * 128, dtype=torch.bfloat16, device=DEV)
    far_q, far_k = far.as_strided((T, 3, 128), (step, 128, 1)), far.as_strided((T, 2, 128), (step, 128, 1), 3 * 128)
    far_q.copy_(q), far_k.copy_(k)
    want = rotary.rotate(q, k, rope)
    assert all(torch.equal(a, b) for a, b in zip(rotary.rotate(far_q, far_k, rope), want))
    # appended from there to pages behind 4 GB of the cache, and read back
    pages = 1 << 18
    near = serve.kv4_cache(3, 2, 128, 64, device=DEV)
    cache = torch.empty((pages, *near.shape[1:]), dtype=near.dtype, device=DEV)
    assert cache[-3:].data_ptr() - cache.data_ptr() > 1 << 32
    args = kv4.int32([T]), kv4.int32([0, T])
    qs = []
    for c, first, a, b in ((near, 0, q, k), (cache, pages - 3, far_q, far_k)):
        c[-3:].fill_(0xA5)
        table = kv4.int32([[first + 2, first, first + 1]])
        qs.append(rotary.kv4_append(c, a, b, b, rope, table, *args))
        qs += serve.kv4_load(c, table, *args, T, 128)
    assert torch.equal(near, cache[-3:]) and all(torch.equal(a, b) for a, b in zip(qs[:3], qs[3:]))
    # and in place
    rotary.fa_rotate(far_q, far_k, far_q, far_k, rope)
    assert torch.equal(far_q, want[0]) and torch.equal(far_k, want[1])
