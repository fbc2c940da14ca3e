"""GPU tests of the paged 4-bit cache: storing, loading, and the attention over it.

What is stored is exact by definition, so store and load are compared bit for
bit with the format's definition in 64 bits.

The attention's tolerances: the cache's values are exact inputs (the reference
reads the same bytes).  P is rounded to f16 (relative error at most 2^-11; a
value below 2^-14 of the scale in use, 2^-22 of a maximum, by at most 2^-33 of
the maximum), which moves O by at most 2^-11 (w|V| + |O|) + keys 2^-33 max|V|;
a score's error e of at most (d + 16) 2^-22 scale sum|q||k| (sums of the matrix
instruction may truncate: four times the rounding's 2^-24) moves it by at most
2 e (w|V| + |O|), the exponentials and sums by less than 2^-12 (w|V| + |O|); O's
rounding to bf16 is 2^-8 |O|.  The logsumexp moves by e, by keys 2^-24 from
its sum, and by a few 2^-24 |LSE|.
"""
import math

import pytest
import torch

from exact_attention_20_gb300 import build as fa_build
from tests import kv4_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def serve():
    fa_build.build()
    from exact_attention_20_gb300 import serve as mod
    mod.lib()
    return mod


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def layout(lens, page_size, seed=0, spare=2):
    """A page table in random order for these lengths: the table, and the number of pages."""
    need = [-(-n // page_size) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed)).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [10 ** 6] * (max(need + [1]) - n))  # entries past a sequence are not read
        at += n
    return int32(table).view(len(lens), max(need + [1])), sum(need) + spare


def cumulative(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return int32(out)


def fill(serve, lens, heads, d, page_size, seed=0, garbage=0xFF, spread=1.0):
    """A cache holding random keys and values of these lengths; all other bytes are `garbage`."""
    g = generator(seed)
    table, pages = layout(lens, page_size, seed)
    cache = serve.kv4_cache(pages, heads, d, page_size)
    cache.fill_(garbage)
    T = sum(lens)
    k = (torch.randn((T, heads, d), generator=g, device=DEV) * spread).bfloat16()
    v = torch.randn((T, heads, d), generator=g, device=DEV).bfloat16()
    errors = int32([0])
    serve.kv4_store(cache, k, v, table, int32(lens), cumulative(lens), errors=errors)
    assert errors.item() == 0
    return cache, table, k, v


# ---------------------------------------------------------------------------
# Store and load
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page_size", [16, 64, 1024])
@pytest.mark.parametrize("heads", [1, 3, 8])
def test_stored_values_are_the_formats(serve, d, page_size, heads):
    lens = [1, 0, 17, 300, 16, 1025, 31]
    cache, table, k, v = fill(serve, lens, heads, d, page_size, seed=1)
    kk, vv = serve.kv4_load(cache, table, int32(lens), cumulative(lens), sum(lens), d)
    assert torch.equal(kk.double(), ref.stored(k)) and torch.equal(vv.double(), ref.stored(v))
    at = 0
    for i, n in enumerate(lens):  # and they lie where the format says
        a, b = ref.read(cache, d, page_size, table[i].tolist()[:-(-n // page_size)], n)
        assert torch.equal(a, ref.stored(k[at:at + n])) and torch.equal(b, ref.stored(v[at:at + n]))
        at += n


def test_every_bf16_value_and_tie(serve):
    # a block's largest element fixes the scale: every bf16 magnitude against
    # scales of all eight significands, near and at the ties between codes
    d, rows = 64, []
    mags = torch.arange(0, 0x7F80, 1, dtype=torch.int32)
    for top in range(0x4000, 0x4080, 9):  # largest element: 2 to 4, fifteen significands
        rest = mags[(mags <= top) & (mags > top - 0x0500)]
        rest = torch.cat([rest, rest.new_zeros((-len(rest)) % 15)]).view(-1, 15)
        rows.append(torch.cat([torch.full((len(rest), 1), top, dtype=torch.int32), rest], 1))
    x = torch.cat(rows)
    x = torch.cat([x, x.new_zeros(((-len(x)) % 4, 16))]).view(-1, d)
    sign = torch.randint(0, 2, x.shape, generator=torch.Generator().manual_seed(3), dtype=torch.int32) << 15
    x = (x | sign).to(torch.int16).view(torch.bfloat16).to(DEV).unsqueeze(1)
    n = x.shape[0]
    table, pages = layout([n], 64)
    cache = serve.kv4_cache(pages, 1, d, 64)
    serve.kv4_store(cache, x, x, table, int32([n]), int32([0, n]))
    k, v = serve.kv4_load(cache, table, int32([n]), int32([0, n]), n, d)
    assert torch.equal(k.double(), ref.stored(x)) and torch.equal(v.double(), ref.stored(x))


@pytest.mark.parametrize("g_k,g_v", [(1.0, 1.0), (2.0 ** -12, 2.0 ** 9), (2.0 ** 40, 2.0 ** -40)])
def test_scales_ranges_and_values_that_are_not_finite(serve, g_k, g_v):
    d, n = 128, 64
    x = torch.randn((n, 2, d), generator=generator(4), device=DEV)
    x = x * torch.exp2(torch.randint(-30, 30, (n, 2, 8, 1), generator=generator(5), device=DEV).float()
                       ).expand(-1, -1, -1, 16).flatten(-2)
    x[3] = 0
    x[5, 0, 17], x[5, 1, 40], x[6, 0, 127] = math.inf, -math.inf, math.nan
    x[7, 0, :16], x[7, 0, 16:32] = 3e38, 1e-40   # saturates; too small for any scale
    x = x.bfloat16()
    table, pages = layout([n], 16)
    cache = serve.kv4_cache(pages, 2, d, 16)
    args = (table, int32([n]), int32([0, n]))
    serve.kv4_store(cache, x, x, *args, k_scale=g_k, v_scale=g_v)
    k, v = serve.kv4_load(cache, *args, n, d, k_scale=g_k, v_scale=g_v)
    for got, g in ((k, g_k), (v, g_v)):
        want = ref.stored(x, g)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        # a value of the format times g may itself lie outside bf16's normal range
        assert torch.equal(torch.nan_to_num(got.double()), torch.nan_to_num(want).bfloat16().double())
        assert torch.isnan(got).sum() == 48


def test_store_writes_its_own_places_only(serve):
    # appending to sequences in the middle of their pages: every other byte stays
    d, heads, page = 128, 2, 32
    before, new = [5, 0, 31, 100], [1, 3, 2, 0]
    after = [a + b for a, b in zip(before, new)]
    table, pages = layout(after, page, seed=6)
    cache = serve.kv4_cache(pages, heads, d, page).fill_(0xA5)
    k = torch.randn((8, heads, d), generator=generator(6), device=DEV).bfloat16()  # two tokens behind the last sequence
    serve.kv4_store(cache, k, -k, table, int32(after), cumulative(new))
    back = torch.full((8, heads, d), 7.0, dtype=torch.bfloat16, device=DEV)
    back_v = back.clone()
    serve.fa_kv4_load(cache, table, int32(after), cumulative(new), back, back_v)
    assert torch.equal(back[:6].double(), ref.stored(k[:6])) and torch.equal(back_v[:6].double(), ref.stored(-k[:6]))
    assert (back[6:] == 7.0).all() and (back_v[6:] == 7.0).all()
    assert int((cache != 0xA5).sum()) <= 6 * heads * serve.kv4_row_bytes(d)
    touched = torch.zeros_like(cache, dtype=torch.bool)
    at, rb = 0, serve.kv4_row_bytes(d)
    for i, n in enumerate(new):
        for x in range(before[i], after[i]):
            p, off = table[i, x // page].item(), x % page // 16 * 16 * rb
            for v in (0, 1):
                a, r = off + v * 8 * rb, x % 16
                touched[p, :, a + r * d // 2:a + (r + 1) * d // 2] = True
                touched[p, :, a + 8 * d + r * d // 16:a + 8 * d + (r + 1) * d // 16] = True
    assert (cache[~touched] == 0xA5).all()


def test_store_takes_views_of_a_fused_projection(serve):
    d, heads, lens = 64, 4, [100, 37]
    x = torch.randn((137, 3 * heads * d), generator=generator(7), device=DEV).bfloat16()
    k, v = x[:, heads * d:2 * heads * d].view(137, heads, d), x[:, 2 * heads * d:].view(137, heads, d)
    table, pages = layout(lens, 64)
    cache = serve.kv4_cache(pages, heads, d, 64)
    serve.kv4_store(cache, k, v, table, int32(lens), cumulative(lens))
    kk, vv = serve.kv4_load(cache, table, int32(lens), cumulative(lens), 137, d)
    assert torch.equal(kk.double(), ref.stored(k)) and torch.equal(vv.double(), ref.stored(v))


def test_more_sequences_than_shared_memory_holds(serve):
    lens = [(i * 5) % 4 for i in range(5000)]
    cache, table, k, v = fill(serve, lens, 1, 64, 16, seed=8)
    kk, vv = serve.kv4_load(cache, table, int32(lens), cumulative(lens), sum(lens), 64)
    assert torch.equal(kk.double(), ref.stored(k)) and torch.equal(vv.double(), ref.stored(v))


def test_bad_pages_and_positions_are_skipped_and_reported(serve):
    d, heads, page = 64, 1, 16
    k = torch.ones((6, heads, d), dtype=torch.bfloat16, device=DEV)
    cache = serve.kv4_cache(4, heads, d, page).fill_(0x5A)
    table = int32([[0, 4], [1, 2], [-1, 3]])
    cu = int32([0, 2, 4, 6])
    errors = int32([0])
    serve.kv4_store(cache, k, k, table, int32([18, 1, 2]), cu, errors=errors)  # page 4; position -1; page -1
    assert errors.item() == serve.BAD_PAGE | serve.BAD_POSITION
    # sequence 1's second token (position 0) is the only one stored
    assert (cache[[0, 2, 3]] == 0x5A).all()
    assert int((cache[1] != 0x5A).sum()) <= serve.kv4_row_bytes(d)
    errors.zero_()
    kk, vv = serve.kv4_load(cache, table, int32([18, 1, 2]), cu, 6, d, errors=errors)
    assert errors.item() == serve.BAD_PAGE | serve.BAD_POSITION
    # 1 stands for 6 * 0.171875, the e4m3 value nearest to 1/6
    assert (kk[3] == 1.03125).all() and (kk[[0, 1, 2, 4, 5]] == 0).all() and (vv[[0, 1, 2, 4, 5]] == 0).all()
    errors.zero_()
    serve.kv4_store(cache, k, k, table, int32([33, 34, 40]), cu, errors=errors)  # past the tables' 32 positions
    assert errors.item() == serve.BAD_POSITION or errors.item() == serve.BAD_POSITION | serve.BAD_PAGE


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def check_attention(serve, lens, hq, hkv, d, page_size, nq=1, seed=0, spread=1.0, q_scale=1.0):
    cache, table, _, _ = fill(serve, lens, hkv, d, page_size, seed, spread=spread)
    q = (torch.randn((len(lens) * nq, hq, d), generator=generator(seed + 1), device=DEV) * q_scale).bfloat16()
    errors = int32([0])
    scale = d ** -0.5
    o, lse = serve.kv4_attention(q, cache, table, int32(lens), n_queries=nq, scale=scale, errors=errors)
    torch.cuda.synchronize()
    assert errors.item() == 0
    for i, n in enumerate(lens):
        k, v = ref.read(cache, d, page_size, table[i].tolist()[:-(-n // page_size)], n)
        rows = slice(i * nq, (i + 1) * nq)
        compare(o[rows], lse[:, rows], *ref.attend(q[rows], k, v, scale), n, float(v.abs().max()) if n else 0.0, d)
    return q, cache, table, o, lse


def compare(o, lse, o64, lse64, bound, most, n, vmax, d):
    assert torch.equal(torch.isneginf(lse64), torch.isneginf(lse)) and not torch.isnan(lse).any()
    e = (d + 16) * 2.0 ** -22 * most
    tol = (2.0 ** -11 + 2.0 ** -12 + 2 * e) * bound + n * 2.0 ** -33 * vmax + 2.0 ** -8 * o64.abs()
    err = (o.double() - o64).abs()
    assert (err <= tol).all(), f"{(err - tol).max().item():.3g}"
    if o64.numel() >= 4096 and e < 2.0 ** -10:  # O's rounding dominates: 2^-8 / sqrt(3) in the root mean square at the most
        assert err.norm() <= 2.0 ** -8 * o64.norm()
    fin = torch.isfinite(lse64)
    tol = e + (n + 8) * 2.0 ** -24 + 2.0 ** -21 * lse64[fin].abs()
    assert ((lse.double() - lse64)[fin].abs() <= tol).all(), (lse.double() - lse64)[fin].abs().max()


LENS = {
    "one": [1],
    "group-edges": [15, 16, 17, 127, 128, 129],
    "empty-ones": [0, 40, 0, 513],
    "long": [5000],
    "ragged": [3, 2049, 700, 64, 1300, 1],
}


@pytest.mark.parametrize("name", LENS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (6, 2), (8, 1), (12, 1), (32, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_matches_definition(serve, name, hq, hkv, d):
    check_attention(serve, LENS[name], hq, hkv, d, 64, seed=len(name))


@pytest.mark.parametrize("nq", [2, 3, 4, 8])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (5, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_several_queries_see_up_to_themselves(serve, nq, hq, hkv, d):
    # lengths below nq leave queries without a key
    check_attention(serve, [0, 1, 2, nq, 17, 127, 130, 600], hq, hkv, d, 16, nq=nq, seed=nq)


@pytest.mark.parametrize("nq,hq", [(1, 96), (5, 40), (1, 128)])
def test_more_rows_than_one_row_tile(serve, nq, hq):
    check_attention(serve, [100, 1, 700], hq, 1, 64, 32, nq=nq, seed=9)


@pytest.mark.parametrize("page_size", [16, 32, 128, 1024])
def test_page_sizes(serve, page_size):
    check_attention(serve, [33, 1000, 4097], 8, 2, 128, page_size, seed=10)


def test_many_sequences(serve):
    check_attention(serve, [(i * 37) % 400 for i in range(300)], 4, 2, 64, 32, seed=11)


def test_long_context(serve):
    check_attention(serve, [70001], 4, 1, 128, 128, seed=12)


@pytest.mark.parametrize("spread,q_scale", [(6.0, 4.0), (1e-3, 1.0), (1.0, 1e-6), (1.0, 3e4), (30.0, 4.0)])
def test_value_ranges(serve, spread, q_scale):
    # peaked rows whose reference moves often; keys and queries far from 1
    check_attention(serve, [1500, 90], 8, 2, 128, 64, seed=13, spread=spread, q_scale=q_scale)


def test_garbage_past_the_sequence_does_not_matter(serve):
    # the cache's unused bytes hold 0xFF (scales NaN) in every test here; another filling gives the same bits
    lens, d = [5, 77, 1000], 128
    cache, table, k, v = fill(serve, lens, 2, d, 64, seed=14)
    other = serve.kv4_cache(cache.shape[0], 2, d, 64)
    serve.kv4_store(other, k, v, table, int32(lens), cumulative(lens))
    q = torch.randn((3, 8, d), generator=generator(15), device=DEV).bfloat16()
    a, b = (serve.kv4_attention(q, c, table, int32(lens)) for c in (cache, other))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d", [64, 128])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(serve, d):
    lens, nq, page = [40, 200], 4, 16
    cache, table, k, v = fill(serve, lens, 1, d, page, seed=16)
    v, k = v.clone(), k.clone()
    v[37, 0, 20] = math.nan          # seen by sequence 0's queries 1 to 3 (positions 36 to 39)
    v[40 + 3, 0, 0] = math.inf       # seen by all of sequence 1's
    k[40 + 198, 0, 5] = math.nan     # seen by its queries 2 and 3
    serve.kv4_store(cache, k, v, table, int32(lens), cumulative(lens))
    q = torch.randn((8, 2, d), generator=generator(17), device=DEV).bfloat16()
    o, lse = serve.kv4_attention(q, cache, table, int32(lens), n_queries=nq)
    for i, n in enumerate(lens):
        kk, vv = ref.read(cache, d, page, table[i].tolist()[:-(-n // page)], n)
        o64, lse64, _, _ = ref.attend(q[4 * i:4 * i + 4], kk, vv, d ** -0.5)
        assert torch.equal(torch.isnan(o[4 * i:4 * i + 4]), torch.isnan(o64))
        assert torch.equal(torch.isnan(lse[:, 4 * i:4 * i + 4]), torch.isnan(lse64))
    assert torch.isnan(o[1:4, :, 16:32]).all() and not torch.isnan(o[0]).any()


def test_attention_skips_bad_pages_and_reports_them(serve):
    d = 128
    cache, table, _, _ = fill(serve, [64, 64], 1, d, 16, seed=18)
    table = table.clone()
    good = table.clone()
    table[1, 2] = -3
    q = torch.randn((2, 4, d), generator=generator(19), device=DEV).bfloat16()
    errors = int32([0])
    o, lse = serve.kv4_attention(q, cache, table, int32([64, 64]), errors=errors)
    assert errors.item() == serve.BAD_PAGE
    k, v = ref.read(cache, d, 16, good[1].tolist(), 64)
    keep = [i for i in range(64) if i // 16 != 2]
    o64, lse64, bound, most = ref.attend(q[1:2], k[keep], v[keep], d ** -0.5)
    compare(o[1:2], lse[:, 1:2], o64, lse64, bound, most, 48, float(v.abs().max()), d)
    errors.zero_()
    lens = int32([65, -1])  # past the table's four pages, and below zero
    o, lse = serve.kv4_attention(q, cache, good, lens, errors=errors)
    assert errors.item() == serve.BAD_POSITION
    assert torch.isneginf(lse[:, 1]).all() and (o[1] == 0).all()


def test_repeatable_bits(serve):
    q, cache, table, o, lse = check_attention(serve, [9000, 5, 3000], 8, 2, 128, 64, seed=20)
    for _ in range(3):
        o2, lse2 = serve.kv4_attention(q, cache, table, int32([9000, 5, 3000]), scale=128 ** -0.5)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_nothing_to_do(serve):
    cache = serve.kv4_cache(2, 1, 64, 16)
    none = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=DEV)
    table = torch.empty((0, 1), dtype=torch.int32, device=DEV)
    serve.kv4_store(cache, none, none, table, int32([]), int32([0]))
    k, v = serve.kv4_load(cache, table, int32([]), int32([0]), 0, 64)
    o, lse = serve.kv4_attention(none, cache, table, int32([]))
    assert k.shape == (0, 1, 64) and o.shape == (0, 1, 64) and lse.shape == (1, 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g_k,g_v", [(2.0 ** -9, 2.0 ** 7), (2.0 ** 5, 2.0 ** -12), (2.0 ** 40, 2.0 ** -40)])
def test_attention_with_scales_of_the_tensors(serve, d, g_k, g_v):
    # a product with a power of two is exact, so nothing else changes: whole items, and a cut one
    lens, hq, hkv, page = [70, 3000], 8, 2, 32
    table, pages = layout(lens, page, 21)
    cache = serve.kv4_cache(pages, hkv, d, page).fill_(0xFF)
    g = generator(21)
    k = (torch.randn((sum(lens), hkv, d), generator=g, device=DEV) * g_k).bfloat16()
    v = (torch.randn((sum(lens), hkv, d), generator=g, device=DEV) * g_v).bfloat16()
    serve.kv4_store(cache, k, v, table, int32(lens), cumulative(lens), k_scale=g_k, v_scale=g_v)
    q = torch.randn((2, hq, d), generator=g, device=DEV).bfloat16()
    scale = d ** -0.5 / g_k
    o, lse = serve.kv4_attention(q, cache, table, int32(lens), scale=scale, k_scale=g_k, v_scale=g_v)
    for i, n in enumerate(lens):
        kk, vv = ref.read(cache, d, page, table[i].tolist()[:-(-n // page)], n, g_k, g_v)
        compare(o[i:i + 1], lse[:, i:i + 1], *ref.attend(q[i:i + 1], kk, vv, scale), n, float(vv.abs().max()), d)


def split(serve, n, nq, hq, hkv, d, max_pages, page):
    import ctypes
    need = ctypes.c_size_t(0)
    rc = serve.lib().fa_kv4_attention_workspace(n, nq, hq, hkv, d, max_pages, page, ctypes.byref(need))
    assert rc == 0
    return need.value > 0


@pytest.mark.parametrize("lens,nq,hq,hkv,d", [
    # more sequences than a CTA has threads (512; 256 for the 32-row tile at d = 128), most of them empty or short
    ([0, 1, 0, 2] * 300 + [9000] + [1, 0, 33] * 50, 1, 4, 2, 64),
    ([5000] + [i % 3 for i in range(1500)] + [4000, 17], 1, 4, 1, 128),
    ([i * 53 % 1400 for i in range(600)], 1, 2, 1, 64),              # ranges end within many of them
    ([0] * 299 + [3000] + [1] * 300 + [2000], 4, 8, 1, 128),
    ([0] * 1100 + [600], 1, 1, 1, 64),
])
def test_more_sequences_than_threads_with_cut_items(serve, lens, nq, hq, hkv, d):
    page = 64
    assert split(serve, len(lens), nq, hq, hkv, d, -(-max(lens) // page), page)
    check_attention(serve, lens, hq, hkv, d, page, nq=nq, seed=22)


def test_a_store_of_refused_tokens_alone_leaves_the_cache(serve):
    d, page = 64, 16
    k = torch.ones((6, 1, d), dtype=torch.bfloat16, device=DEV)
    cache = serve.kv4_cache(4, 1, d, page).fill_(0x5A)
    before = cache.clone()
    table = int32([[0, 4], [1, 2], [-1, 3]])
    errors = int32([0])
    # positions 31 (page 4 of 4) and 32 (past the table), 32 and 33, 38 and 39
    serve.kv4_store(cache, k, k, table, int32([33, 34, 40]), int32([0, 2, 4, 6]), errors=errors)
    assert errors.item() == serve.BAD_PAGE | serve.BAD_POSITION
    assert torch.equal(cache, before)
