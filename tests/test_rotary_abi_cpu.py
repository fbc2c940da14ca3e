"""The rotary entry points reject bad arguments before touching CUDA, header, library and binding agree, and the
frequencies are what they say (no compute call here)."""
import ctypes
import math
import os
import re

import pytest
import torch

from exact_attention_20_gb300 import build as fa_build
from tests import rotary_reference as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fa_gb300_rotary.h")
A, STEP = 1 << 40, 1 << 36
Q, K, V, QO, KO, CACHE, TABLE, LENS, CU, ERR, POS, TURNS = (A + i * STEP for i in range(12))


@pytest.fixture(scope="module")
def rotary():
    fa_build.build()
    from exact_attention_20_gb300 import rotary as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def fa(rotary):
    return rotary.fa


def test_header_library_and_binding_agree(rotary):
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(fa_\w+)\s*\(", text))
    assert names == set(rotary.SIGNATURES) == {"fa_rotate", "fa_kv4_append"}
    for name in names:
        assert hasattr(rotary.lib(), name)


DENSE = dict(q=(8 * 100 * 64, 64, 100 * 64), k=(2 * 100 * 64, 64, 100 * 64))  # [2, 8 and 2, 100, 64]


def rotate(rotary, strides=None, **over):
    a = dict(q=Q, k=K, qo=QO, ko=KO, pos=POS, turns=TURNS, B=2, N=100, Hq=8, Hk=2, d=64, rot=64, inter=0, m=1.0, back=0)
    a.update(over)
    s = strides or [*DENSE["q"], *DENSE["k"], *DENSE["q"], *DENSE["k"]]
    ps = a.pop("ps", 100)
    s = None if strides == "null" else (ctypes.c_longlong * 12)(*s)
    return rotary.lib().fa_rotate(*a.values(), s, ps, None)


@pytest.mark.parametrize("over", [
    dict(d=96), dict(rot=8), dict(rot=24), dict(rot=80), dict(rot=0), dict(inter=2), dict(m=0.0), dict(m=float("nan")),
    dict(m=float("inf")), dict(B=-1), dict(B=65536), dict(N=-1), dict(B=32768, N=32769), dict(Hq=0), dict(Hk=-1), dict(back=2),
    dict(ps=99), dict(ps=-1), dict(strides=[*DENSE["q"][:2], 12, *DENSE["k"], *DENSE["q"], *DENSE["k"]]),
    dict(strides=[-64, *DENSE["q"][1:], *DENSE["k"], *DENSE["q"], *DENSE["k"]]),
    dict(strides=[*DENSE["q"], *DENSE["k"], 0, *DENSE["q"][1:], *DENSE["k"]]),           # outputs on top of one another
    dict(strides=[*DENSE["q"], *DENSE["k"], *DENSE["q"], DENSE["k"][0], 56, DENSE["k"][2]]),
])
def test_rotate_invalid(rotary, fa, over):
    assert rotate(rotary, **over) == fa.FA_ERR_INVALID_ARG


def test_rotate_null_alignment_and_alias(rotary, fa):
    for name in ("q", "k", "qo", "ko", "turns"):
        assert rotate(rotary, **{name: None}) == fa.FA_ERR_NULL, name
    assert rotate(rotary, strides="null") == fa.FA_ERR_NULL
    for name, addr, off in (("q", Q, 8), ("k", K, 8), ("qo", QO, 8), ("ko", KO, 8), ("turns", TURNS, 4), ("pos", POS, 2)):
        assert rotate(rotary, **{name: addr + off}) == fa.FA_ERR_ALIGN, name
    end = 2 * 8 * 100 * 64 * 2
    for over in (dict(qo=Q + 16), dict(qo=K), dict(ko=Q + end - 16), dict(ko=QO + 64), dict(qo=POS), dict(ko=TURNS),
                 dict(ko=Q)):
        assert rotate(rotary, **over) == fa.FA_ERR_ALIAS, over
    # in place with other strides: not its own places
    row = 12 * 64
    packed = [0, row, 64] * 4
    one = dict(B=1, N=100, ps=0, q=Q, k=Q + 8 * 128, qo=Q, ko=Q + 8 * 128)
    assert rotate(rotary, strides=[0, row, 64, 0, row, 64, 0, 2 * row, 64, 0, row, 64], **one) == fa.FA_ERR_ALIAS
    # columns of the same rows may be turned in place, but not on top of one another
    assert rotate(rotary, strides=packed, **{**one, "k": Q + 7 * 128, "ko": Q + 7 * 128}) == fa.FA_ERR_ALIAS
    if not torch.cuda.is_available():
        assert rotate(rotary, strides=packed, **one) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_DEVICE)
        assert rotate(rotary) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_DEVICE)
        assert rotate(rotary, k=None, ko=None, Hk=0) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_DEVICE)


def test_nothing_to_rotate(rotary, fa):
    assert rotate(rotary, N=0, q=None, k=None, qo=None, ko=None) == fa.FA_OK
    assert rotate(rotary, B=0) == fa.FA_OK


def append(rotary, **over):
    a = dict(q=Q, k=K, v=V, qo=QO, ko=KO, cache=CACHE, table=TABLE, lens=LENS, cu=CU, pos=POS, turns=TURNS, T=64, n=2,
             max_pages=4, num_pages=16, page=16, Hq=8, Hkv=2, d=64, rot=64, inter=0, m=1.0, qs=512, ks=128, vs=128, kg=1.0,
             vg=1.0, errors=ERR, stream=None)
    a.update(over)
    return rotary.lib().fa_kv4_append(*a.values())


@pytest.mark.parametrize("over", [
    dict(n=-1), dict(max_pages=0), dict(num_pages=0), dict(page=8), dict(page=24), dict(Hkv=0), dict(d=32), dict(kg=3.0),
    dict(vg=0.0), dict(T=-1), dict(T=(1 << 30) + 1), dict(Hq=-1), dict(Hq=(1 << 16) + 1), dict(qs=504), dict(qs=516), dict(ks=120),
    dict(vs=132), dict(rot=72), dict(rot=0), dict(inter=-1), dict(m=-1.0), dict(qs=(1 << 32) + 8),
])
def test_append_invalid(rotary, fa, over):
    assert append(rotary, **over) == fa.FA_ERR_INVALID_ARG


def test_append_null_alignment_and_alias(rotary, fa):
    fine = dict(q=Q, k=K, v=V, qo=QO, ko=KO, cache=CACHE, table=TABLE, lens=LENS, cu=CU, pos=POS, turns=TURNS)
    for name in fine:
        if name not in ("ko", "pos"):
            assert append(rotary, **{name: None}) == fa.FA_ERR_NULL, name
        off = 4 if name == "turns" else 2 if name in ("table", "lens", "cu", "pos") else 8
        assert append(rotary, **{name: fine[name] + off}) == fa.FA_ERR_ALIGN, name
    assert append(rotary, errors=ERR + 2) == fa.FA_ERR_ALIGN
    for over in (dict(k=CACHE), dict(qo=Q), dict(ko=K), dict(qo=V), dict(qo=CACHE + 64), dict(ko=QO + 16), dict(errors=LENS),
                 dict(errors=CACHE), dict(errors=QO + 4), dict(pos=QO), dict(turns=KO), dict(cu=CACHE)):
        assert append(rotary, **over) == fa.FA_ERR_ALIAS, over
    if not torch.cuda.is_available():
        assert append(rotary) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_DEVICE)
        assert append(rotary, q=None, qo=None, Hq=0, ko=None, pos=None, errors=None) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_DEVICE)


def test_append_without_tokens_is_done(rotary, fa):
    assert append(rotary, T=0) == fa.FA_OK and append(rotary, n=0, table=None, lens=None, cu=None) == fa.FA_OK


def test_frequencies(rotary):
    f = rotary.frequencies(64, base=500.0)
    assert len(f) == 32 and f[0] == 1.0 and abs(f[31] / 500.0 ** (-62 / 64) - 1) < 1e-14
    assert [a / 4 for a in f] == rotary.frequencies(64, base=500.0, scaling="linear", factor=4.0)
    b = rotary.frequencies(64, scaling="base", factor=4.0)
    assert b[0] == 1.0 and abs(b[31] * 4 / rotary.frequencies(64)[31] - 1) < 1e-12
    p, plain = rotary.frequencies(128, scaling="parts", factor=8.0), rotary.frequencies(128)
    for a, c in zip(p, plain):
        times = 4096 * c / (2 * math.pi)
        assert a == c if times >= 32 else a == c / 8 if times <= 1 else c / 8 < a < c
    for bad in (dict(rot_dim=20), dict(rot_dim=0), dict(rot_dim=256), dict(rot_dim=64, base=1.0), dict(rot_dim=64, factor=0.5),
                dict(rot_dim=64, scaling="other"), dict(rot_dim=64, scaling="parts", slow=4.0, fast=4.0),
                dict(rot_dim=64, base=math.inf), dict(rot_dim=64, factor=math.nan)):
        with pytest.raises(ValueError):
            rotary.frequencies(**bad)


def test_turns(rotary):
    # a quarter of a turn, one radian, a whole turn and a bit; and the largest position's angle
    t = rotary.turns([math.pi / 2, 1.0, 2 * math.pi, 0.0], device="cpu")
    assert t.dtype == torch.int64
    assert abs(t[0].item() / 2.0 ** 62 - 1) < 2.0 ** -52 and abs(t[1].item() / 2.0 ** 64 * 2 * math.pi - 1) < 2.0 ** -52
    assert abs((t[2].item() + 2 ** 63) % 2 ** 64 - 2 ** 63) < 2 ** 13 and t[3] == 0  # 2 pi in 64 bits is not quite one
    r = rotary.rope(128, device="cpu")
    c, _ = ref.cos_sin(torch.tensor([10 ** 6]), r.turns, r.magnitude)
    want = [math.cos(math.fmod(10 ** 6 * f, 2 * math.pi)) for f in rotary.frequencies(128)]
    assert max(abs(a - b) for a, b in zip(c[0].tolist(), want)) < 1e-9
    assert rotary.rope(64, scaling="parts", factor=math.e, device="cpu").magnitude == pytest.approx(1.1)


def test_binding_checks(rotary):
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    r = rotary.rope(64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        rotary.rotate(x, x, r)
    for bad in (dict(q=x.float()), dict(q=x[0]), dict(k=x[:3]), dict(k=x[None]), dict(rope=r.turns),
                dict(rope=rotary.rope(128, device="cpu")), dict(rope=rotary.Rope(r.turns.int())),
                dict(rope=rotary.Rope(r.turns[:4])), dict(positions=torch.zeros(3, dtype=torch.int32)),
                dict(positions=torch.zeros(4, dtype=torch.int64)), dict(q=x.transpose(1, 2).contiguous().transpose(1, 2))):
        a = dict(q=x, k=x, rope=r)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            rotary.rotate(**a)
    with pytest.raises(TypeError):
        rotary.fa_rotate(x, x, x, None, r)
    cache = torch.zeros((2, 2, 16 * 72), dtype=torch.uint8)
    table, n, cu = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in (dict(q=x[:2]), dict(k=x.half()), dict(v=x[:, :1]), dict(cu_seqlens=n), dict(positions=n), dict(rope=None)):
        a = dict(cache=cache, q=x, k=x, v=x, rope=r, page_table=table, seq_lens=n, cu_seqlens=cu)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            rotary.kv4_append(**a)
    with pytest.raises(TypeError):
        rotary.fa_kv4_append(cache, x, x, x, r, table, n, cu, None)
