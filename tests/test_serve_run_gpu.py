"""GPU tests of the serving operators as a server uses them: together, on streams of their own, and captured.

The attention's tolerances are those of test_kv4_gpu (its ``compare``) and of
test_packed_gpu; everything else here is compared bit for bit.
"""
import math

import pytest
import torch

from exact_attention_20_gb300 import build as fa_build
from tests import kv4_reference as ref
from tests import test_kv4_gpu as kv4
from tests import test_packed_gpu as packed

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def serve():
    fa_build.build()
    from exact_attention_20_gb300 import serve as mod
    mod.lib()
    return mod


class Server:
    """Prompts of these lengths, their cache, and tables with room for more tokens."""

    def __init__(self, serve, lens, hq, hkv, d, page=16, room=40, seed=0):
        self.serve, self.lens, self.hq, self.hkv, self.d, self.page = serve, list(lens), hq, hkv, d, page
        self.g = kv4.generator(seed)
        self.table, pages = kv4.layout([n + room for n in lens], page, seed)
        self.cache = serve.kv4_cache(pages, hkv, d, page).fill_(0xFF)
        self.seq_lens = kv4.int32(self.lens)

    def tokens(self, n):
        """q, k, v of n tokens, views of one projection's output."""
        x = torch.randn((n, (self.hq + 2 * self.hkv) * self.d), generator=self.g, device=DEV).bfloat16()
        q, k, v = x.split((self.hq * self.d, self.hkv * self.d, self.hkv * self.d), 1)
        return q.view(n, self.hq, self.d), k.view(n, self.hkv, self.d), v.view(n, self.hkv, self.d)

    def held(self, i):
        n = self.lens[i]
        return ref.read(self.cache, self.d, self.page, self.table[i].tolist()[:-(-n // self.page)], n)

    def fill(self):
        """Keys and values for every token so far."""
        _, k, v = self.tokens(sum(self.lens))
        self.serve.kv4_store(self.cache, k, v, self.table, self.seq_lens, kv4.cumulative(self.lens))
        return self

    def check(self, q, o, lse, nq):
        for i, n in enumerate(self.lens):
            k, v = self.held(i)
            rows = slice(i * nq, (i + 1) * nq)
            kv4.compare(o[rows], lse[:, rows], *ref.attend(q[rows], k, v, self.d ** -0.5), n, float(v.abs().max()), self.d)


@pytest.mark.parametrize("d,hq,hkv,page", [(128, 8, 2, 16), (64, 12, 4, 64)])
def test_prompts_then_steps(serve, d, hq, hkv, page):
    s = Server(serve, [70, 1, 300, 16], hq, hkv, d, page)
    # the prompts: attention, and their keys and values into the cache
    q, k, v = s.tokens(sum(s.lens))
    o, lse = serve.attention_packed(q, k, v, s.lens)
    o64, lse64, bound, most = packed.reference(q, k, v, s.lens, True, d ** -0.5)
    packed.compare(o, lse, o64, lse64, bound, most, d, max(s.lens))
    serve.kv4_store(s.cache, k, v, s.table, s.seq_lens, kv4.cumulative(s.lens))
    # steps of one token, then of three, across page ends
    for nq in (1, 1, 3, 1, 12):
        s.lens = [n + nq for n in s.lens]
        s.seq_lens += nq
        q, k, v = s.tokens(nq * len(s.lens))
        serve.kv4_store(s.cache, k, v, s.table, s.seq_lens, kv4.cumulative([nq] * len(s.lens)))
        o, lse = serve.kv4_attention(q, s.cache, s.table, s.seq_lens, n_queries=nq)
        s.check(q, o, lse, nq)
    # what is held, read back, attended to as packed prompts: the same last rows
    kk, vv = serve.kv4_load(s.cache, s.table, s.seq_lens, kv4.cumulative(s.lens), sum(s.lens), d)
    at = 0
    for i, n in enumerate(s.lens):
        held = s.held(i)
        assert torch.equal(kk[at:at + n].double(), held[0]) and torch.equal(vv[at:at + n].double(), held[1])
        at += n
    whole = torch.zeros((sum(s.lens), hq, d), dtype=torch.bfloat16, device=DEV)
    at = 0
    for i, n in enumerate(s.lens):
        whole[at + n - 12:at + n] = q[i * 12:(i + 1) * 12]
        at += n
    o2, lse2 = serve.attention_packed(whole, kk, vv, s.lens)
    o64, lse64, bound, most = packed.reference(whole, kk, vv, s.lens, True, d ** -0.5)
    packed.compare(o2, lse2, o64, lse64, bound, most, d, max(s.lens))
    at = 0
    for i, n in enumerate(s.lens):  # both operators, the same rows: each within its roundings of the same values
        rows, last = slice(i * 12, (i + 1) * 12), slice(at + n - 12, at + n)
        assert ((o[rows].double() - o2[last].double()).abs() <= 2.0 ** -6 * bound[last] + 2.0 ** -7 * o64[last].abs()).all()
        assert ((lse[:, rows] - lse2[:, last]).abs() <= 1e-3).all()
        at += n


def test_shared_pages_are_read_by_both(serve):
    d, lens = 128, [64, 64]
    cache, table, k, v = kv4.fill(serve, [64], 2, d, 16, seed=1)
    two = table.repeat(2, 1).contiguous()
    q = torch.randn((1, 8, d), generator=kv4.generator(2), device=DEV).bfloat16().repeat(2, 1, 1)
    o, lse = serve.kv4_attention(q, cache, two, kv4.int32(lens))
    assert torch.equal(o[0], o[1]) and torch.equal(lse[:, 0], lse[:, 1])


def test_queries_and_values_as_strided_views(serve):
    # token strides and starts that 32-byte accesses do not fit (16 bytes apart)
    d, heads, n = 64, 3, 90
    x = torch.randn((n, 3 * heads * d + 8), generator=kv4.generator(3), device=DEV).bfloat16()
    q, k, v = (x[:, 8 + i * heads * d:8 + (i + 1) * heads * d].view(n, heads, d) for i in range(3))
    assert k.data_ptr() % 32 == 16 and k.stride(0) % 16 == 8
    table, pages = kv4.layout([n], 32)
    cache = serve.kv4_cache(pages, heads, d, 32)
    lens, cu = kv4.int32([n]), kv4.int32([0, n])
    serve.kv4_store(cache, k, v, table, lens, cu)
    flat = torch.empty(2 * n * heads * d + 8, dtype=torch.bfloat16, device=DEV)
    kk, vv = flat[8:8 + n * heads * d].view(n, heads, d), flat[8 + n * heads * d:].view(n, heads, d)
    serve.fa_kv4_load(cache, table, lens, cu, kk, vv)
    assert torch.equal(kk.double(), ref.stored(k)) and torch.equal(vv.double(), ref.stored(v))
    a = serve.kv4_attention(q[-2:], cache, table, lens, n_queries=2)
    b = serve.kv4_attention(q[-2:].contiguous(), cache, table, lens, n_queries=2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = serve.attention_packed(q, k, v, [n])
    b = serve.attention_packed(q.contiguous(), k.contiguous(), v.contiguous(), [n])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def everything(serve, s, q, k, v, stream=None):
    """One call of each operator; the outputs."""
    nq = q.shape[0] // len(s.lens)
    cu = kv4.cumulative([nq] * len(s.lens))
    serve.kv4_store(s.cache, k, v, s.table, s.seq_lens, cu, stream=stream)
    out = list(serve.kv4_attention(q, s.cache, s.table, s.seq_lens, n_queries=nq, stream=stream))
    out += serve.kv4_load(s.cache, s.table, s.seq_lens, cu, k.shape[0], s.d, stream=stream)
    out += serve.attention_packed(q, k, v, [nq] * len(s.lens), stream=stream)
    return out


def test_streams(serve):
    # a torch stream, a raw handle and the current stream give the same bits, whatever else is queued
    s = Server(serve, [900, 5, 2000], 8, 2, 128, 64).fill()
    q, k, v = s.tokens(6)
    want = everything(serve, s, q, k, v)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    for _ in range(20):
        busy.add_(1)  # the current stream has work to do meanwhile
    for stream in (side, side.cuda_stream):
        got = everything(serve, s, q, k, v, stream=stream)
        side.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a.cpu(), b.cpu())
    with torch.cuda.stream(side):
        got = everything(serve, s, q, k, v)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(want, everything(serve, s, q, k, v, stream=0)))


def test_two_streams_at_once(serve):
    # calls that split work, at once on two streams: no workspace is shared
    a, b = (Server(serve, [6000, 3000], 8, 2, 128, 64, seed=i).fill() for i in (4, 5))
    qa, qb = a.tokens(2), b.tokens(2)
    pa, pb = packed.make([3000, 500], 8, 2, 128, 6), packed.make([3000, 500], 8, 2, 128, 7)

    def work(s, q, x):
        return [*serve.kv4_attention(q[0], s.cache, s.table, s.seq_lens), *serve.attention_packed(*x, [3000, 500])]

    wa, wb = work(a, qa, pa), work(b, qb, pb)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    ga, gb = [], []
    for _ in range(10):
        with torch.cuda.stream(sa):
            ga.append(work(a, qa, pa))
        with torch.cuda.stream(sb):
            gb.append(work(b, qb, pb))
    torch.cuda.synchronize()
    for want, runs in ((wa, ga), (wb, gb)):
        for got in runs:
            assert all(torch.equal(x, y) for x, y in zip(want, got))


def capture(f):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    return g, out


def test_captured_steps_follow_the_tables(serve):
    # a decoding step captured once, replayed while the sequences grow, pages change hands and one sequence ends
    s = Server(serve, [700, 16, 1], 8, 2, 128, 16, room=20, seed=8)
    q, k, v = (t.contiguous() for t in s.tokens(3))
    pq, pk, pv = s.tokens(sum(s.lens))
    serve.kv4_store(s.cache, pk, pv, s.table, s.seq_lens, kv4.cumulative(s.lens))
    cu, before = kv4.cumulative([1, 1, 1]), s.cache.clone()

    def step():
        serve.kv4_store(s.cache, k, v, s.table, s.seq_lens, cu)
        return serve.kv4_attention(q, s.cache, s.table, s.seq_lens)

    g, (o, lse) = capture(step)
    s.cache.copy_(before)
    for i in range(18):
        for t, x in zip((q, k, v), s.tokens(3)):
            t.copy_(x)
        s.seq_lens += 1
        if i == 9:
            s.seq_lens[1] = 1     # a new sequence in the second place
        s.lens = s.seq_lens.tolist()
        g.replay()
        if i in (0, 8, 9, 17):
            s.check(q, o, lse, 1)
        held = s.cache.clone()
        want = step()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(held, s.cache)


def test_two_captured_graphs_at_once(serve):
    a, b = (packed.make([2500, 100], 8, 2, 128, i) for i in (9, 10))
    s = Server(serve, [5000], 8, 2, 128, 64, seed=11)
    pq, pk, pv = s.tokens(5000)
    serve.kv4_store(s.cache, pk, pv, s.table, s.seq_lens, kv4.cumulative([5000]))
    q1, q2 = s.tokens(1)[0], s.tokens(1)[0]
    graphs, wants = [], []
    for x, q in ((a, q1), (b, q2)):
        f = lambda x=x, q=q: [*serve.attention_packed(*x, [2500, 100]), *serve.kv4_attention(q, s.cache, s.table, s.seq_lens)]  # noqa: E731
        wants.append([t.clone() for t in f()])
        graphs.append(capture(f))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for want, (_, got) in zip(wants, graphs):
        for x, y in zip(want, got):
            assert torch.equal(x[:2600] if x.dim() == 3 else x, y[:2600] if y.dim() == 3 else y)


def test_what_ran_before_is_not_disturbed(serve):
    # the dense operators and the status word beside the serving ones
    from exact_attention_20_gb300 import fa
    from exact_attention_20_gb300.inputs import make_qkv
    q, k, v = make_qkv(1, 4, 2048, 128, seed=12, device=DEV)
    want = fa.attention(q, k, v, causal=True)
    s = Server(serve, [3000, 50], 8, 2, 128, 64, seed=13).fill()
    x = s.tokens(2)
    everything(serve, s, *x)
    got = fa.attention(q, k, v, causal=True)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert fa.device_status() == fa.FA_OK
    # one sequence, one head of a group: the packed operator is the dense one
    o, lse = serve.attention_packed(*(t[0].transpose(0, 1).contiguous() for t in (q, k, v)), [2048])
    assert ((o.transpose(0, 1).float() - want[0][0].float()).abs() <= 1e-2).all()
    assert ((lse - want[1][0]).abs() <= 1e-4).all()
    assert math.isfinite(float(lse.sum()))
