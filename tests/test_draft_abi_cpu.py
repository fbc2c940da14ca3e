"""The drafted tokens' entry points reject bad arguments before touching CUDA, and header, library and binding agree (no
compute call here)."""
import ctypes
import os
import re

import pytest
import torch

from exact_attention_20_gb300 import build as fa_build

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fa_gb300_draft.h")
A, STEP = 1 << 40, 1 << 36
Q, O, L, WS, CACHE, TABLE, LENS, PAR, ERR, LOGITS, TOK, U, DRAFT, PATH, KEPT, NEXT, NEW = (A + i * STEP for i in range(17))


@pytest.fixture(scope="module")
def draft():
    fa_build.build()
    from exact_attention_20_gb300 import draft as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def fa(draft):
    return draft.fa


def test_header_library_and_binding_agree(draft):
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(fa_\w+)\s*\(", text))
    assert names == set(draft.SIGNATURES) == {"fa_kv4_tree_attention", "fa_kv4_tree_attention_workspace", "fa_verify_tree",
                                              "fa_kv4_keep"}
    for name in names:
        assert hasattr(draft.lib(), name)
    assert f"#define FA_KV4_BAD_TREE {draft.BAD_TREE}" in text


def attention(draft, **over):
    a = dict(q=Q, cache=CACHE, table=TABLE, lens=LENS, par=PAR, o=O, lse=L, n=2, nodes=16, Hq=8, Hkv=2, d=64, max_pages=4,
             num_pages=16, page=16, qs=512, scale=0.125, kg=1.0, vg=1.0, errors=ERR, ws=None, wb=0, stream=None)
    a.update(over)
    return draft.lib().fa_kv4_tree_attention(*a.values())


def verify(draft, **over):
    a = dict(logits=LOGITS, fp32=0, tok=TOK, par=PAR, u=U, dp=DRAFT, path=PATH, kept=KEPT, next=NEXT, n=3, nodes=8, V=1000,
             ls=1000, ds=1000, temperature=1.0, stream=None)
    a.update(over)
    return draft.lib().fa_verify_tree(*a.values())


def keep(draft, **over):
    a = dict(cache=CACHE, table=TABLE, lens=LENS, path=PATH, kept=KEPT, new=NEW, n=2, nodes=16, max_pages=4, num_pages=16, page=16,
             Hkv=2, d=64, errors=ERR, stream=None)
    a.update(over)
    return draft.lib().fa_kv4_keep(*a.values())


CACHE_INVALID = [dict(n=-1), dict(max_pages=0), dict(num_pages=0), dict(page=8), dict(page=24), dict(page=2048), dict(Hkv=0),
                 dict(d=32), dict(nodes=0), dict(nodes=65), dict(nodes=-1)]


@pytest.mark.parametrize("call", [attention, keep])
@pytest.mark.parametrize("over", CACHE_INVALID)
def test_cache_invalid(draft, fa, call, over):
    assert call(draft, **over) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("call,over", [
    (attention, dict(Hq=7)), (attention, dict(Hq=0)), (attention, dict(Hq=258)), (attention, dict(scale=0.0)),
    (attention, dict(scale=float("nan"))), (attention, dict(qs=504)), (attention, dict(qs=513)), (attention, dict(kg=3.0)),
    (attention, dict(vg=0.0)), (attention, dict(scale=3e38, kg=2.0 ** 40)), (attention, dict(n=1 << 30)),
    (verify, dict(fp32=2)), (verify, dict(n=-1)), (verify, dict(nodes=0)), (verify, dict(nodes=65)), (verify, dict(V=0)),
    (verify, dict(V=(1 << 18) + 1, ls=1 << 19, ds=1 << 19)), (verify, dict(ls=999)), (verify, dict(ds=999)),
    (verify, dict(ls=(1 << 32) + 1)), (verify, dict(temperature=-1.0)), (verify, dict(temperature=float("nan"))),
    (verify, dict(temperature=float("inf"))), (verify, dict(temperature=1e-38)), (verify, dict(n=(1 << 24) + 1)),
    (keep, dict(n=1 << 20, Hkv=1 << 16)),
])
def test_invalid(draft, fa, call, over):
    assert call(draft, **over) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("call,names", [(attention, "q cache table lens par o lse"), (verify, "logits tok par u path kept next"),
                                        (keep, "cache table lens path kept new")])
def test_null_and_alignment(draft, fa, call, names):
    fine = dict(q=Q, cache=CACHE, table=TABLE, lens=LENS, par=PAR, o=O, lse=L, logits=LOGITS, tok=TOK, u=U, path=PATH, kept=KEPT,
                next=NEXT, new=NEW)
    for name in names.split():
        assert call(draft, **{name: None}) == fa.FA_ERR_NULL, name
        off = 8 if name in ("q", "cache", "o") else 1 if name == "logits" else 2
        assert call(draft, **{name: fine[name] + off}) == fa.FA_ERR_ALIGN, name
    if call is verify:
        assert verify(draft, dp=DRAFT + 2) == fa.FA_ERR_ALIGN and verify(draft, fp32=1, logits=LOGITS + 2) == fa.FA_ERR_ALIGN
    else:
        assert call(draft, errors=ERR + 1) == fa.FA_ERR_ALIGN


def test_alias(draft, fa):
    for over in (dict(o=Q), dict(o=CACHE + 16), dict(lse=PAR), dict(lse=O), dict(o=LENS), dict(errors=PAR), dict(errors=LENS + 4),
                 dict(ws=O, wb=4096), dict(ws=PAR, wb=4096)):
        assert attention(draft, **over) == fa.FA_ERR_ALIAS, over
    assert attention(draft, ws=WS + 64, wb=4096) == fa.FA_ERR_ALIGN
    for over in (dict(path=TOK), dict(kept=PAR), dict(next=U), dict(path=LOGITS + 64), dict(next=DRAFT), dict(kept=PATH + 4),
                 dict(next=KEPT)):
        assert verify(draft, **over) == fa.FA_ERR_ALIAS, over
    for over in (dict(new=LENS), dict(new=KEPT), dict(path=CACHE), dict(errors=CACHE), dict(errors=NEW), dict(kept=NEW),
                 dict(table=CACHE + 64)):
        assert keep(draft, **over) == fa.FA_ERR_ALIAS, over


def test_without_work_is_done(draft, fa):
    assert attention(draft, n=0, q=None, o=None, lse=None, par=None) == fa.FA_OK
    assert verify(draft, n=0, logits=None) == fa.FA_OK and keep(draft, n=0, path=None) == fa.FA_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")
def test_valid_calls_without_a_device_fail_loudly(draft, fa):
    for call in (attention, verify, keep):
        assert call(draft) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_DEVICE)
    assert verify(draft, dp=None, ds=0, temperature=0.0) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_DEVICE)
    b = ctypes.c_size_t(0)
    f = draft.lib().fa_kv4_tree_attention_workspace
    assert f(2, 16, 8, 2, 64, 4, 16, ctypes.byref(b)) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_DEVICE)


def test_workspace_checks(draft, fa):
    b = ctypes.c_size_t(0)
    f = draft.lib().fa_kv4_tree_attention_workspace
    assert f(2, 16, 8, 2, 64, 4, 16, None) == fa.FA_ERR_NULL
    assert f(2, 65, 8, 2, 64, 4, 16, ctypes.byref(b)) == fa.FA_ERR_INVALID_ARG
    assert f(2, 16, 8, 3, 64, 4, 16, ctypes.byref(b)) == fa.FA_ERR_INVALID_ARG


def test_binding_checks(draft):
    q = torch.zeros((8, 2, 64), dtype=torch.bfloat16)
    cache = torch.zeros((2, 2, 16 * 72), dtype=torch.uint8)
    table, lens = torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    par = torch.zeros((2, 4), dtype=torch.int32)
    for bad in (dict(q=q[:7]), dict(q=q.float()), dict(cache=cache[:, :, :100]), dict(page_table=table.long()),
                dict(seq_lens=lens[:1]), dict(parents=par[:1]), dict(parents=par.long()), dict(parents=par[0]),
                dict(parents=torch.zeros((2, 65), dtype=torch.int32)), dict(parents=par[:, :0])):
        a = dict(q=q, cache=cache, page_table=table, seq_lens=lens, parents=par)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            draft.kv4_tree_attention(**a)
    logits, u = torch.zeros((2, 4, 10)), torch.zeros((2, 4))
    for bad in (dict(logits=logits.double()), dict(logits=logits[:1]), dict(logits=logits[..., ::2]), dict(tokens=par.long()),
                dict(parents=par[:, :3]), dict(uniforms=u.double()), dict(uniforms=u[:1]), dict(draft_probs=logits.bfloat16()),
                dict(draft_probs=logits[..., :9]), dict(logits=torch.zeros((2, 5, 10))[:, :4]), dict(logits=logits.view(80))):
        a = dict(logits=logits, tokens=par, parents=par, uniforms=u)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            draft.verify_tree(**a)
    for bad in (dict(path=par.long()), dict(path=par[:1]), dict(n_kept=lens.long()), dict(d=96), dict(n_kept=par)):
        a = dict(cache=cache, page_table=table, seq_lens=lens, path=par, n_kept=lens, d=64)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            draft.kv4_keep(**a)
    with pytest.raises(TypeError):
        draft.fa_kv4_tree_attention(q, cache, table, lens, par, None, None)
    with pytest.raises(TypeError):
        draft.fa_verify_tree(logits, par, par, u, None, None, None)
    with pytest.raises(TypeError):
        draft.fa_kv4_keep(cache, table, lens, par, lens, None, 64)
    for call in (lambda: draft.kv4_tree_attention(q, cache, table, lens, par), lambda: draft.verify_tree(logits, par, par, u),
                 lambda: draft.kv4_keep(cache, table, lens, par, lens, 64)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
