"""The serving operators' C entry points reject bad arguments before touching CUDA, and the header, the library and the
binding agree (no compute call here)."""
import ctypes
import os
import re

import pytest
import torch

from exact_attention_20_gb300 import build as fa_build

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fa_gb300_serve.h")

# fake, aligned, far-apart addresses: every call fails its host checks before any CUDA call
A, STEP = 1 << 40, 1 << 36
Q, K, V, O, L, WS, CACHE, TABLE, LENS, CU, ERR = (A + i * STEP for i in range(11))


@pytest.fixture(scope="module")
def serve():
    fa_build.build()
    from exact_attention_20_gb300 import serve as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def fa(serve):
    return serve.fa


def test_header_library_and_binding_agree(serve):
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(fa_\w+)\s*\(", text))
    assert names == set(serve.SIGNATURES) == {
        "fa_fwd_packed", "fa_fwd_packed_workspace", "fa_kv4_store", "fa_kv4_load", "fa_kv4_attention",
        "fa_kv4_attention_workspace"}
    for name in names:
        assert hasattr(serve.lib(), name)


def lens(*n):
    return (ctypes.c_int * max(1, len(n)))(*n)


def packed(serve, **over):
    a = dict(q=Q, k=K, v=V, o=O, lse=L, seq_lens=lens(100, 28), n=2, T=128, Hq=8, Hkv=2, d=64, qs=512, ks=128, vs=128,
             causal=1, scale=0.125, ws=None, wb=0, stream=None)
    a.update(over)
    return serve.lib().fa_fwd_packed(*a.values())


@pytest.mark.parametrize("over", [
    dict(n=-1), dict(T=-1), dict(T=(1 << 30) + 1), dict(Hq=0), dict(Hkv=0), dict(Hkv=3), dict(Hq=258),
    dict(d=96), dict(d=0), dict(causal=2), dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0), dict(scale=3e38),
    dict(T=127), dict(seq_lens=lens(-1, 5)), dict(seq_lens=lens(2 ** 31 - 1, 2 ** 31 - 1)),
    dict(qs=511), dict(qs=504), dict(qs=516), dict(ks=120), dict(vs=(1 << 32) + 8),
])
def test_packed_invalid(serve, fa, over):
    assert packed(serve, **over) == fa.FA_ERR_INVALID_ARG


def test_packed_null_alignment_and_alias(serve, fa):
    for name in ("q", "k", "v", "o", "lse", "seq_lens"):
        assert packed(serve, **{name: None}) == fa.FA_ERR_NULL, name
    for name, addr in (("q", Q), ("k", K), ("v", V), ("o", O)):
        assert packed(serve, **{name: addr + 8}) == fa.FA_ERR_ALIGN, name
    assert packed(serve, lse=L + 2) == fa.FA_ERR_ALIGN
    assert packed(serve, ws=WS + 128) == fa.FA_ERR_ALIGN
    row = 8 * 64 * 2
    assert packed(serve, o=Q + 127 * row) == fa.FA_ERR_ALIAS
    # a strided q reaches as far as its last token does
    assert packed(serve, qs=1024, o=Q + 200 * row) == fa.FA_ERR_ALIAS
    assert packed(serve, lse=O + 64) == fa.FA_ERR_ALIAS
    assert packed(serve, lse=V + 4) == fa.FA_ERR_ALIAS
    assert packed(serve, ws=O, wb=256) == fa.FA_ERR_ALIAS
    assert packed(serve, ws=K, wb=256) == fa.FA_ERR_ALIAS


def test_packed_without_tokens_is_done(serve, fa):
    assert packed(serve, seq_lens=lens(0, 0)) == fa.FA_OK
    assert packed(serve, seq_lens=None, n=0) == fa.FA_OK
    assert packed(serve, seq_lens=lens(0), n=1, T=0, q=None, k=None, v=None, o=None, lse=None) == fa.FA_OK


def test_packed_workspace_checks(serve, fa):
    b = ctypes.c_size_t(0)
    f = serve.lib().fa_fwd_packed_workspace
    assert f(lens(100, 28), 2, 128, 8, 2, 64, 1, None) == fa.FA_ERR_NULL
    assert f(None, 2, 128, 8, 2, 64, 1, ctypes.byref(b)) == fa.FA_ERR_NULL
    assert f(lens(100, 28), 2, 127, 8, 2, 64, 1, ctypes.byref(b)) == fa.FA_ERR_INVALID_ARG
    assert f(lens(100, 28), 2, 128, 8, 2, 32, 1, ctypes.byref(b)) == fa.FA_ERR_INVALID_ARG


def store(serve, **over):
    a = dict(k=K, v=V, cache=CACHE, table=TABLE, lens=LENS, cu=CU, T=64, n=2, max_pages=4, num_pages=16, page=16, Hkv=2,
             d=64, ks=128, vs=128, kg=1.0, vg=1.0, errors=ERR, stream=None)
    a.update(over)
    return serve.lib().fa_kv4_store(*a.values())


def load(serve, **over):
    a = dict(cache=CACHE, table=TABLE, lens=LENS, cu=CU, k=K, v=V, T=64, n=2, max_pages=4, num_pages=16, page=16, Hkv=2,
             d=64, kg=1.0, vg=1.0, errors=ERR, stream=None)
    a.update(over)
    return serve.lib().fa_kv4_load(*a.values())


def attention(serve, **over):
    a = dict(q=Q, cache=CACHE, table=TABLE, lens=LENS, o=O, lse=L, n=2, Lq=1, Hq=8, Hkv=2, d=64, max_pages=4,
             num_pages=16, page=16, qs=512, scale=0.125, kg=1.0, vg=1.0, errors=ERR, ws=None, wb=0, stream=None)
    a.update(over)
    return serve.lib().fa_kv4_attention(*a.values())


CACHE_INVALID = [dict(n=-1), dict(max_pages=0), dict(num_pages=0), dict(page=8), dict(page=24), dict(page=2048),
                 dict(page=0), dict(Hkv=0), dict(d=32), dict(kg=0.0), dict(kg=3.0), dict(vg=-1.0), dict(vg=float("inf")),
                 dict(kg=2.0 ** 41), dict(vg=2.0 ** -41), dict(vg=float("nan"))]


@pytest.mark.parametrize("call", [store, load, attention])
@pytest.mark.parametrize("over", CACHE_INVALID)
def test_cache_invalid(serve, fa, call, over):
    assert call(serve, **over) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("call,over", [
    (store, dict(T=-1)), (store, dict(T=(1 << 30) + 1)), (store, dict(ks=120)), (store, dict(vs=132)), (load, dict(T=-1)),
    (attention, dict(Lq=0)), (attention, dict(Hq=7)), (attention, dict(Hq=0)), (attention, dict(Hq=258)),
    (attention, dict(scale=0.0)), (attention, dict(scale=float("inf"))), (attention, dict(qs=504)),
    (attention, dict(qs=513)), (attention, dict(scale=3e38, kg=2.0 ** 40)), (attention, dict(scale=1e-38, kg=2.0 ** -40)), (attention, dict(n=1 << 30, Lq=2)), (attention, dict(n=1 << 20, Hkv=1 << 16, Hq=1 << 16)),
])
def test_cache_calls_invalid(serve, fa, call, over):
    assert call(serve, **over) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("call,names", [(store, "k v cache table lens cu"), (load, "k v cache table lens cu"),
                                        (attention, "q cache table lens o lse")])
def test_cache_calls_null_and_alignment(serve, fa, call, names):
    fine = dict(k=K, v=V, cache=CACHE, table=TABLE, lens=LENS, cu=CU, q=Q, o=O, lse=L)
    for name in names.split():
        assert call(serve, **{name: None}) == fa.FA_ERR_NULL, name
        off = 8 if name in ("k", "v", "cache", "q", "o") else 2
        assert call(serve, **{name: fine[name] + off}) == fa.FA_ERR_ALIGN, name
    assert call(serve, errors=ERR + 1) == fa.FA_ERR_ALIGN


def test_cache_calls_alias(serve, fa):
    end = 16 * 2 * 16 * 72  # the cache's bytes
    assert store(serve, k=CACHE + end - 16) == fa.FA_ERR_ALIAS
    assert store(serve, lens=CACHE) == fa.FA_ERR_ALIAS
    assert store(serve, errors=CACHE + 64) == fa.FA_ERR_ALIAS
    assert store(serve, errors=TABLE) == fa.FA_ERR_ALIAS
    assert load(serve, k=V + 16) == fa.FA_ERR_ALIAS
    assert load(serve, v=CACHE + end - 16) == fa.FA_ERR_ALIAS
    assert load(serve, k=CU - 64) == fa.FA_ERR_ALIAS
    assert attention(serve, o=CACHE + 16) == fa.FA_ERR_ALIAS
    assert attention(serve, o=Q) == fa.FA_ERR_ALIAS
    assert attention(serve, lse=LENS) == fa.FA_ERR_ALIAS
    assert attention(serve, lse=O) == fa.FA_ERR_ALIAS
    assert attention(serve, ws=O, wb=4096) == fa.FA_ERR_ALIAS
    assert attention(serve, errors=LENS + 4) == fa.FA_ERR_ALIAS
    assert attention(serve, ws=WS + 64, wb=4096) == fa.FA_ERR_ALIGN


def test_cache_calls_without_work_are_done(serve, fa):
    assert store(serve, T=0) == fa.FA_OK and store(serve, n=0, table=None, lens=None, cu=None) == fa.FA_OK
    assert load(serve, T=0) == fa.FA_OK and attention(serve, n=0, q=None, o=None, lse=None) == fa.FA_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")
def test_valid_calls_without_a_device_fail_loudly(serve, fa):
    for call in (packed, store, load, attention):
        assert call(serve) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_DEVICE)
    b = ctypes.c_size_t(0)
    assert serve.lib().fa_kv4_attention_workspace(2, 1, 8, 2, 64, 4, 16, ctypes.byref(b)) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_DEVICE)
    assert serve.lib().fa_kv4_attention_workspace(2, 1, 8, 2, 64, 4, 16, None) == fa.FA_ERR_NULL


def test_binding_checks(serve):
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        serve.attention_packed(x, x, x, [4])
    with pytest.raises(TypeError):
        serve.fa_fwd_packed(x.float(), x, x, x, torch.zeros(2, 4), [4])
    with pytest.raises(ValueError):
        serve.fa_fwd_packed(x, x, x[:3], x, torch.zeros(2, 4), [4])
    for lens, error in (([5], ValueError), ([-1, 5], ValueError), ([2 ** 32 + 4], ValueError),
                        ([2 ** 32 + 4, -2 ** 32], ValueError), ([2.5], TypeError), (torch.tensor([1.0]), TypeError)):
        with pytest.raises(error):
            serve.attention_packed(x, x, x, lens)
    with pytest.raises(TypeError):
        serve.fa_fwd_packed(x, x, x, None, None, [4])
    with pytest.raises(ValueError):
        serve.kv4_row_bytes(96)
    cache = torch.zeros((2, 2, 16 * 72), dtype=torch.uint8)
    table, n, cu = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in (dict(cache=cache[:, :, :100]), dict(page_table=table.long()), dict(seq_lens=cu), dict(cu_seqlens=n),
                dict(k=x.transpose(0, 1)), dict(v=x[:2]), dict(k=x.half())):
        args = dict(cache=cache, k=x, v=x, page_table=table, seq_lens=n, cu_seqlens=cu)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            serve.kv4_store(**args)
    with pytest.raises(ValueError):
        serve.kv4_attention(x, cache, table, n, n_queries=0)
    with pytest.raises(ValueError):
        serve.kv4_attention(x, cache, table, n, n_queries=2)  # four rows, one sequence
