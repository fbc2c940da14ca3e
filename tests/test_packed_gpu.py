"""GPU tests of the attention over packed prompts against its definition in 64 bits.

Tolerances, from the roundings the operator documents.  With w the exact
softmax weights, P's rounding to bf16 (relative error at most 2^-8) moves a row
of O by at most 2^-7 sum_j w_j |v_j - O| <= 2^-7 (w|V| + |O|), since the weights
are normalised by the sum of the rounded values; O's own rounding adds
2^-8 |O|.  The fp32 scores, exponentials and sums move the weights by a
relative error far below 2^-12 at these sizes (score error at most (d + 8)
2^-24 scale sum|q||k|), taken as 2^-11 (w|V| + |O|).  Over a whole tensor of
zero-mean values both roundings act as independent errors of at most
2^-8 / sqrt(3) relative in the root mean square, together below 2^-8 of the
tensor's norm.  The logsumexp moves by the score error, by len 2^-24 from its
sum and by a few 2^-24 |LSE| from the logarithm.
"""
import math

import pytest
import torch

from exact_attention_20_gb300 import build as fa_build

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def serve():
    fa_build.build()
    from exact_attention_20_gb300 import serve as mod
    mod.lib()
    return mod


def make(lens, hq, hkv, d, seed=0, tail=0, fused=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    T = sum(lens) + tail
    x = torch.randn((T, (hq + 2 * hkv) * d), generator=g, device=DEV).bfloat16()
    q, k, v = x.split((hq * d, hkv * d, hkv * d), dim=1)
    if not fused:
        q, k, v = (t.contiguous() for t in (q, k, v))
    return q.view(T, hq, d), k.view(T, hkv, d), v.view(T, hkv, d)


def reference(q, k, v, lens, causal, scale):
    """O, LSE, the row bound w|V| + |O| of every sequence's rows, and the largest scale sum|q||k|, in 64 bits."""
    T, hq, d = q.shape
    group = hq // k.shape[1]
    o = torch.zeros((T, hq, d), dtype=torch.float64, device=DEV)
    wv = torch.zeros_like(o)
    lse = torch.zeros((hq, T), dtype=torch.float64, device=DEV)
    most, at = 0.0, 0
    for n in lens:
        if n == 0:
            continue
        rows = slice(at, at + n)
        qs, ks, vs = (t[rows].double().transpose(0, 1) for t in (q, k, v))
        ks, vs = (t.repeat_interleave(group, 0) for t in (ks, vs))
        s = qs @ ks.transpose(1, 2) * scale
        most = max(most, float((qs.abs() @ ks.abs().transpose(1, 2)).max()) * scale)
        if causal:
            i = torch.arange(n, device=DEV)
            hidden = i > i.unsqueeze(1)
            s = s.masked_fill(hidden, -math.inf)
        lse[:, rows] = torch.logsumexp(s, -1)
        w = torch.softmax(s, -1)
        o[rows] = (w @ vs).transpose(0, 1)
        wv[rows] = (w @ vs.abs()).transpose(0, 1)
        at += n
    return o, lse, wv + o.abs(), most


def check(serve, lens, hq, hkv, d, causal, seed=0, tail=0, fused=False):
    q, k, v = make(lens, hq, hkv, d, seed, tail, fused)
    scale = d ** -0.5
    T, n = q.shape[0], sum(lens)
    o = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((hq, T), 7.0, device=DEV)
    serve.fa_fwd_packed(q, k, v, o, lse, lens, causal=causal, scale=scale)
    torch.cuda.synchronize()
    assert (o[n:] == 7.0).all() and (lse[:, n:] == 7.0).all(), "rows behind the last sequence were written"
    o64, lse64, bound, most = reference(q, k, v, lens, causal, scale)
    compare(o[:n], lse[:, :n], o64[:n], lse64[:, :n], bound[:n], most, d, max(lens, default=0))


def compare(o, lse, o64, lse64, bound, most, d, longest):
    err = (o.double() - o64).abs()
    tol = (2.0 ** -7 + 2.0 ** -11) * bound + 2.0 ** -8 * o64.abs()
    assert torch.isfinite(o.float()).all()
    assert (err <= tol).all(), f"max excess {(err - tol).max().item():.3g} at {(err - tol).argmax().item()}"
    if o64.numel() >= 4096:
        assert err.norm() <= 2.0 ** -8 * o64.norm(), f"norm-wise {(err.norm() / o64.norm()).item():.3g}"
    tol = (d + 8) * 2.0 ** -24 * most + (longest + 8) * 2.0 ** -24 + 2.0 ** -21 * lse64.abs()
    assert ((lse.double() - lse64).abs() <= tol).all(), (lse.double() - lse64).abs().max()


LENS = {
    "one-token": [1],
    "one-short": [37],
    "tile-edges": [127, 128, 129, 1, 255, 256, 257],
    "empty-ones": [0, 5, 0, 0, 300, 0],
    "many-short": [1, 2, 3, 17, 31, 64, 5, 1, 1, 90] * 6,
    "long": [1500],
    "ragged": [700, 3, 1025, 64, 513],
}


@pytest.mark.parametrize("name", LENS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (8, 2), (8, 1), (6, 2), (5, 1), (28, 4)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_matches_definition(serve, name, hq, hkv, d, causal):
    check(serve, LENS[name], hq, hkv, d, causal, seed=len(name))


@pytest.mark.parametrize("hq,hkv", [(32, 1), (48, 1), (128, 1), (130, 2)])
def test_large_groups(serve, hq, hkv):
    # few tokens to a tile: 4, 2, 1 and (65 heads) 1 with unused rows
    check(serve, [5, 150, 1], hq, hkv, 64, True, seed=2)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_views_of_a_fused_projection_and_rows_behind(serve, d, causal):
    check(serve, [33, 400, 129], 8, 2, d, causal, seed=3, tail=77, fused=True)


@pytest.mark.parametrize("lens,hq,hkv,causal", [
    ([4096], 4, 1, True),             # few items: keys split over the CTAs
    ([4096], 2, 2, False),
    ([6000, 10, 2000], 8, 2, True),   # items cut by the equal ranges
    ([3333, 3333], 12, 4, False),
])
def test_split_items(serve, lens, hq, hkv, causal):
    import ctypes
    arr = (ctypes.c_int * len(lens))(*lens)
    need = ctypes.c_size_t(0)
    rc = serve.lib().fa_fwd_packed_workspace(arr, len(lens), sum(lens), hq, hkv, 128, int(causal), ctypes.byref(need))
    assert rc == 0 and need.value > 0, "the call must split items"
    check(serve, lens, hq, hkv, 128, causal, seed=4)


@pytest.mark.parametrize("lens,hq,hkv,d,causal", [
    ([1800, 3, 0, 900, 700, 1, 1500], 8, 8, 128, True),          # short items of many lengths
    ([1800, 3, 0, 900, 700, 1, 1500], 16, 8, 128, False),
    ([300, 1, 1999, 0, 40] * 4, 12, 4, 64, True),
    ([4096], 32, 32, 64, True),                                  # long ones, even without a cut
    ([6000, 100], 16, 1, 64, True),
    ([(37 * i) % 500 + 450 for i in range(110)], 8, 1, 64, True),  # more blocks than are dealt
])
def test_more_items_than_ctas(serve, lens, hq, hkv, d, causal):
    import ctypes
    arr = (ctypes.c_int * len(lens))(*lens)
    need = ctypes.c_size_t(1)
    rc = serve.lib().fa_fwd_packed_workspace(arr, len(lens), sum(lens), hq, hkv, d, int(causal), ctypes.byref(need))
    assert rc == 0 and need.value == 0, "no item is cut"
    check(serve, lens, hq, hkv, d, causal, seed=8)


def test_more_sequences_than_one_launch_takes(serve):
    lens = [(i * 7) % 13 for i in range(2500)]
    check(serve, lens, 4, 2, 64, True, seed=5)


def test_repeatable_bits(serve):
    lens = [5000, 77, 1200]
    q, k, v = make(lens, 8, 2, 128, seed=6)
    first = serve.attention_packed(q, k, v, lens)
    for _ in range(3):
        again = serve.attention_packed(q, k, v, lens)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_no_tokens(serve):
    q, k, v = make([0], 4, 2, 64, tail=3)
    o = torch.full((3, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((4, 3), 7.0, device=DEV)
    serve.fa_fwd_packed(q, k, v, o, lse, [])
    serve.fa_fwd_packed(q, k, v, o, lse, [0, 0])
    assert (o == 7.0).all() and (lse == 7.0).all()
    o, lse = serve.attention_packed(q[:0], k[:0], v[:0], [0])
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)


def exact_rows(q, k, v, n, causal, scale):
    """One sequence, row by row from the keys it sees alone, in 64 bits: O [n, hq, d] (NaN and infinities as they come)."""
    group = q.shape[1] // k.shape[1]
    kd, vd = (t.double().repeat_interleave(group, 1) for t in (k, v))
    o = torch.zeros((n, q.shape[1], q.shape[2]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((q.shape[1], n), dtype=torch.float64, device=DEV)
    for i in range(n):
        seen = i + 1 if causal else n
        s = torch.einsum("hd,mhd->hm", q[i].double(), kd[:seen]) * scale
        lse[:, i] = torch.logsumexp(s, -1)
        o[i] = torch.einsum("hm,mhd->hd", torch.softmax(s, -1), vd[:seen])
    return o, lse


def same_but_for_rounding(o, o64):
    """Non-finite where the reference is, of the same kind; elsewhere within the rounding (see above, with w|V| <= 4)."""
    assert torch.equal(torch.isnan(o.float()), torch.isnan(o64))
    assert torch.equal(torch.isposinf(o.float()), torch.isposinf(o64))
    assert torch.equal(torch.isneginf(o.float()), torch.isneginf(o64))
    fin = torch.isfinite(o64)
    tol = (2.0 ** -7 + 2.0 ** -11) * (4 + o64[fin].abs()) + 2.0 ** -8 * o64[fin].abs()
    assert ((o.double() - o64)[fin].abs() <= tol).all()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (3, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(serve, hq, hkv, d, causal):
    lens = [300, 70, 129, 40]
    q, k, v = make(lens, hq, hkv, d, seed=7, tail=100)
    v, k = v.clone(), k.clone()
    at = [0, 300, 370, 499, 539]
    v[at[0] + 299, 0, 3] = math.nan       # the last token's row alone sees it
    v[at[0] + 130, 0, 5] = math.inf
    v[at[0] + 131, 0, 5] = -math.inf      # from here on NaN in that column
    v[at[0] + 255, 0, d - 1] = -math.inf  # an edge of tiles
    v[at[0] + 0, 0, 7] = math.nan         # every row
    v[at[1]:at[2]] = math.nan             # a whole sequence, its neighbours untouched
    k[at[2] + 64, 0, 0] = math.nan        # a key: the rows that see it are NaN throughout
    v[at[4]:], k[at[4]:], q[at[4]:] = math.nan, math.inf, math.nan  # behind the last sequence
    o, lse = serve.attention_packed(q, k, v, lens, causal=causal)
    for a, n in zip(at, lens):
        o64, lse64 = exact_rows(q[a:a + n], k[a:a + n], v[a:a + n], n, causal, d ** -0.5)
        same_but_for_rounding(o[a:a + n], o64)
        assert torch.equal(torch.isnan(lse[:, a:a + n]), torch.isnan(lse64))
    assert torch.isfinite(o[at[3]:at[4]].float()).all()


def test_not_finite_values_in_split_items(serve):
    lens = [2100]
    q, k, v = make(lens, 4, 1, 128, seed=8)
    v = v.clone()
    for token, col in ((2099, 0), (2001, 1), (1500, 2), (17, 3), (1990, 127)):
        v[token, 0, col] = math.inf if token % 2 else math.nan
    o, _ = serve.attention_packed(q, k, v, lens)
    for token in list(range(0, 40)) + list(range(1495, 1510)) + list(range(1960, 2100)):
        s = torch.einsum("hd,md->hm", q[token].double(), k[:token + 1, 0].double()) * 128 ** -0.5
        same_but_for_rounding(o[token:token + 1], (torch.softmax(s, -1) @ v[:token + 1, 0].double()).unsqueeze(0))
    assert torch.isfinite(o[:17].float()).all()


def test_scores_that_are_all_minus_infinity(serve):
    # a row without weight: O = 0, LSE = -inf, and its neighbours as they are
    q, k, v = make([50], 1, 1, 64, seed=9)
    k, q = k.clone(), q.clone()
    q[:, 0, 0], k[:, 0, 0] = 1.0, -math.inf
    k[20, 0, 0] = 0.0
    o, lse = serve.attention_packed(q, k, v, [50])
    assert torch.isneginf(lse[0, :20]).all() and (o[:20] == 0).all()
    assert torch.isfinite(lse[0, 20:]).all() and torch.equal(o[20:, 0].float(), v[20, 0].float().expand(30, -1))


def rows_without_weight(serve, lens, hq, hkv, d, causal, none, bad, seed):
    """The keys before `none` of every sequence score -inf in every row, and V is not finite at the tokens `bad` of each.

    Rows that see no other key have to give O = 0 and LSE = -inf, whatever V holds.  Returns the inputs and O.
    """
    q, k, v = make(lens, hq, hkv, d, seed=seed)
    q[:, :, 0] = 1.0
    at, empty = 0, torch.zeros(sum(lens), dtype=torch.bool, device=DEV)
    for n in lens:
        k[at:at + none, :, 0] = -math.inf
        empty[at:at + (min(none, n) if causal else n if none >= n else 0)] = True
        for i, (token, col) in enumerate(bad):
            v[at + token, :, col] = math.nan if i % 2 else math.inf
        at += n
    o, lse = serve.attention_packed(q, k, v, lens, causal=causal)
    assert torch.isneginf(lse[:, empty]).all() and (o[empty] == 0).all()
    assert not torch.isneginf(lse[:, ~empty]).any()
    return q, k, v, o


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (3, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_without_weight_are_zero_whatever_the_values(serve, hq, hkv, d):
    # values behind them (30: in reach of the tile's product), and values that they see (5)
    lens = [50, 300]
    q, k, v, o = rows_without_weight(serve, lens, hq, hkv, d, True, 20, [(30, 1), (33, 0), (5, 2)], seed=10)
    cols = [c for c in range(d) if c != 2]  # a row with weight elsewhere: 0 * inf from its keys without weight may be NaN
    at = 0
    for n in lens:
        o64, _ = exact_rows(q[at:at + n], k[at:at + n], v[at:at + n], n, True, d ** -0.5)
        same_but_for_rounding(o[at + 20:at + n, :, cols], o64[20:, :, cols])
        at += n


@pytest.mark.parametrize("d", [64, 128])
def test_rows_without_weight_where_all_keys_are_seen(serve, d):
    rows_without_weight(serve, [40, 150, 300], 4, 2, d, False, 300, [(30, 1), (5, 2)], seed=11)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_without_weight_in_split_items(serve, d, causal):
    import ctypes
    need = ctypes.c_size_t(0)
    rc = serve.lib().fa_fwd_packed_workspace((ctypes.c_int * 1)(4200), 1, 4200, 4, 1, d, int(causal), ctypes.byref(need))
    assert rc == 0 and need.value > 0, "the call must split items"
    none = 4160 if causal else 4200
    q, k, v, o = rows_without_weight(serve, [4200], 4, 1, d, causal, none, [(4190, 1), (4158, 3), (17, 2)], seed=12)
    cols = [c for c in range(d) if c not in (2, 3)]
    for token in range(4160, 4200) if causal else ():
        s = torch.einsum("hd,md->hm", q[token].double(), k[:token + 1, 0].double()) * d ** -0.5
        o64 = (torch.softmax(s, -1) @ v[:token + 1, 0].double()).unsqueeze(0)
        same_but_for_rounding(o[token:token + 1, :, cols], o64[:, :, cols])


def test_a_long_prompt_whose_last_value_is_not_finite(serve):
    # The rows before the last one are taken anew, each over 2^19 keys, a warp's
    # 32 one after another: that lasts longer than the 2 s after which the CTA's
    # other warps, at the next prompt's items already, give up where nothing moves.
    from exact_attention_20_gb300 import fa
    n, d, lens = 1 << 19, 64, [1 << 19, 3000]
    q, k, v = make(lens, 1, 1, d, seed=13)
    v[n - 1, 0, 9] = math.nan
    o, lse = serve.attention_packed(q, k, v, lens)
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    assert torch.isnan(o[n - 1, 0, 9]) and int(torch.isnan(o).sum()) == 1
    rows = torch.arange(n - 128, n - 1, device=DEV)
    kd, vd = k[:n, 0].double(), v[:n, 0].double().nan_to_num(0.0)
    for part in rows.split(16):
        qd = q[part, 0].double()
        s = (qd @ kd.T) * d ** -0.5
        s.masked_fill_(torch.arange(n, device=DEV) > part.unsqueeze(1), -math.inf)
        w = torch.softmax(s, -1)
        o64 = w @ vd
        bound = w @ vd.abs() + o64.abs()
        # P and O in bf16 as everywhere; the fp32 sums of n terms 2^-24 n^1/2 and the scores below 2^-11
        err = (o[part, 0].double() - o64).abs()
        assert (err <= (2.0 ** -7 + 2.0 ** -11) * bound + 2.0 ** -8 * o64.abs()).all()
    o64, lse64, bound, most = reference(q[n:], k[n:], v[n:], lens[1:], True, d ** -0.5)
    compare(o[n:], lse[:, n:], o64, lse64, bound, most, d, lens[1])


@pytest.mark.parametrize("lens,hq,hkv,causal", [
    ([4096], 4, 1, True),
    ([4096], 2, 2, False),
    ([6000, 10, 2000], 8, 2, True),
    ([3333, 3333], 12, 4, False),
    ([10635], 1, 1, True),            # items of up to six parts
])
def test_split_items_of_head_size_64(serve, lens, hq, hkv, causal):
    import ctypes
    arr = (ctypes.c_int * len(lens))(*lens)
    need = ctypes.c_size_t(0)
    rc = serve.lib().fa_fwd_packed_workspace(arr, len(lens), sum(lens), hq, hkv, 64, int(causal), ctypes.byref(need))
    assert rc == 0 and need.value > 0, "the call must split items"
    check(serve, lens, hq, hkv, 64, causal, seed=14)


@pytest.mark.parametrize("scale", [1.0, 0.02, 1e-6])
@pytest.mark.parametrize("d", [64, 128])
def test_scales(serve, scale, d):
    # 1: peaked rows, whose references move; 1e-6: nearly the mean of V
    lens = [700, 33, 300]
    q, k, v = make(lens, 8, 2, d, seed=15)
    o, lse = serve.attention_packed(q, k, v, lens, scale=scale)
    o64, lse64, bound, most = reference(q, k, v, lens, True, scale)
    # scores up to `most` = scale sum|q||k| are off by (d + 8) 2^-24 of it, which moves a weight by twice that
    bound = bound * (1 + 2 * (d + 8) * 2.0 ** -24 * most / 2.0 ** -7)
    compare(o, lse, o64, lse64, bound, most, d, max(lens))


@pytest.mark.parametrize("d", [64, 128])
def test_split_items_in_several_launches(serve, d):
    # a launch takes 1024 sequences; each has items to cut, and the launches share the workspace one after another
    import ctypes
    lens = [5000] + [i % 2 for i in range(1100)] + [6001] + [1, 0] * 500 + [3000]
    need = []
    for part in (lens[:1024], lens[1024:2048], lens[2048:], lens):
        b = ctypes.c_size_t(0)
        arr = (ctypes.c_int * len(part))(*part)
        assert serve.lib().fa_fwd_packed_workspace(arr, len(part), sum(part), 2, 1, d, 1, ctypes.byref(b)) == 0
        need.append(b.value)
    assert min(need[:3]) > 0 and need[3] == max(need[:3])
    check(serve, lens, 2, 1, d, True, seed=16)
