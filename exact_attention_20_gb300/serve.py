"""ctypes binding of the serving operators of libfa_gb300.so (include/fa_gb300_serve.h).

Attention over packed prompts with grouped heads, and a paged 4-bit cache of
keys and values.  As in ``fa``, this module checks tensor metadata, passes raw
pointers, sizes and strides through the C ABI and turns status codes into
``fa.FAError``; there is no CPU fallback.

Streams: a call runs on ``stream`` (a torch stream, a raw handle, or None for
the current stream of the tensors' device).  Workspaces, and the outputs of
the allocating forms, are allocated per call from torch's allocator in that
stream's pool, so calls on different streams and captured graphs never share
one.  The tensors' device need not be the current one.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import fa
from .fa import FA_OK, FAError

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong
_Z = ctypes.c_size_t
_F = ctypes.c_float
# every function declared in include/fa_gb300_serve.h, with its ctypes signature
SIGNATURES = {
    "fa_fwd_packed": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _L, _L, _L, _I, _F, _P, _Z, _P]),
    "fa_fwd_packed_workspace": (_I, [_P, _I, _I, _I, _I, _I, _I, _P]),
    "fa_kv4_store": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _L, _L, _F, _F, _P, _P]),
    "fa_kv4_load": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _F, _P, _P]),
    "fa_kv4_attention": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _L, _F, _F, _F, _P, _P, _Z,
                              _P]),
    "fa_kv4_attention_workspace": (_I, [_I, _I, _I, _I, _I, _I, _I, _P]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The CUDA library of ``fa.lib()`` with this module's signatures set."""
    global _lib
    handle = fa.lib()
    if _lib is not handle:
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _checked(rc: int) -> None:
    if rc != FA_OK:
        raise FAError(rc)


class _Target:
    """The device and stream of one call: ``with _Target(...) as handle`` makes them current."""

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise ValueError("tensors must be on a CUDA device")
        self.device, self.other = device, None
        if stream is None:
            self.stream = torch.cuda.current_stream(device)
            self.context = (contextlib.nullcontext() if device.index == torch.cuda.current_device()
                            else torch.cuda.device(device))
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                          else torch.cuda.default_stream(device))
            if stream.device != device:
                raise ValueError(f"stream must be on {device}, got {stream.device}")
            caller = torch.cuda.current_stream(device)
            self.stream, self.context = stream, torch.cuda.stream(stream)
            if caller != stream:
                self.other = caller

    def __enter__(self) -> int:
        self.context.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        return self.context.__exit__(*exc)

    def uses(self, *tensors) -> None:
        """Keeps the tensors' memory from being reused before this call's work is done."""
        if self.other is not None:
            for t in tensors:
                t.record_stream(self.stream)

    def gives(self, *tensors):
        """Outputs allocated in the call's stream, for use in the caller's."""
        if self.other is not None:
            for t in tensors:
                t.record_stream(self.other)
        return tensors


def _check_tokens(name, t, heads, d, device, dtype=torch.bfloat16, tokens=None) -> int:
    """Checks a [T, heads, d] tensor whose tokens may be strided; returns the token stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d or (tokens is not None and t.shape[0] != tokens):
        want = ("T" if tokens is None else tokens, heads, d)
        raise ValueError(f"{name} must have shape {want}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.shape[0] <= 1:  # one token's stride says nothing
        if t.shape[0] == 1 and not t[0].is_contiguous():
            raise ValueError(f"{name} must have the heads of a token contiguous")
        return heads * d
    if (heads > 1 and t.stride(1) != d) or t.stride(2) != 1:
        raise ValueError(f"{name} must have the heads of a token contiguous")
    return t.stride(0)


def _scale(scale, d) -> float:
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def _lengths(seq_lens):
    lens = [int(n) for n in (seq_lens.tolist() if isinstance(seq_lens, torch.Tensor) else seq_lens)]
    if any(n < 0 or n > 1 << 30 for n in lens):
        raise ValueError("sequence lengths must lie between 0 and 2^30")
    return (ctypes.c_int * max(1, len(lens)))(*lens), len(lens), sum(lens)


def _packed_shapes(q, k):
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor):
        raise TypeError("q and k must be torch.Tensors")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [T, Hq, d] and k [T, Hkv, d]")
    return q.shape[0], q.shape[1], k.shape[1], q.shape[2]


def fa_fwd_packed(q, k, v, o, lse, seq_lens, causal: bool = True, scale: float | None = None,
                  stream=None) -> None:
    """Attention over packed prompts into caller-owned O and LSE.

    q: bf16 [T, Hq, d]; k, v: bf16 [T, Hkv, d], each with the heads of a token
    contiguous and any token stride (views of a fused projection's output);
    o: bf16 [T, Hq, d] and lse: fp32 [Hq, T], contiguous.  ``seq_lens``: the
    sequences' lengths, known on the host (ints, or a CPU tensor); sequence i
    follows the ones before it.  Query head h reads KV head h // (Hq // Hkv).
    Rows of tokens behind the last sequence are left as they were.
    """
    T, Hq, Hkv, d = _packed_shapes(q, k)
    dev = q.device
    strides = [_check_tokens("q", q, Hq, d, dev), _check_tokens("k", k, Hkv, d, dev, tokens=T),
               _check_tokens("v", v, Hkv, d, dev, tokens=T)]
    fa._check("o", o, torch.bfloat16, (T, Hq, d), dev)
    fa._check("lse", lse, torch.float32, (Hq, T), dev)
    lens, n, total = _lengths(seq_lens)
    if total > T:
        raise ValueError(f"the sequences hold {total} tokens, the tensors {T}")
    c = lib()
    target = _Target(dev, stream)
    need = ctypes.c_size_t(0)
    with target as handle:
        _checked(c.fa_fwd_packed_workspace(lens, n, T, Hq, Hkv, d, int(bool(causal)), ctypes.byref(need)))
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev) if need.value else None
        _checked(c.fa_fwd_packed(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), lens, n, T,
                                 Hq, Hkv, d, *strides, int(bool(causal)), _scale(scale, d),
                                 None if ws is None else ws.data_ptr(), need.value, handle))
    target.uses(q, k, v, o, lse)


def attention_packed(q, k, v, seq_lens, causal: bool = True, scale: float | None = None, stream=None):
    """Allocating form of fa_fwd_packed: returns (O, LSE).

    Rows of tokens behind the last sequence hold nothing of use.
    """
    T, Hq, _, d = _packed_shapes(q, k)
    target = _Target(q.device, stream)
    with target:
        o = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=q.device)
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    fa_fwd_packed(q, k, v, o, lse, seq_lens, causal=causal, scale=scale, stream=stream)
    return target.gives(o, lse)


# ---------------------------------------------------------------------------
# The paged 4-bit cache
# ---------------------------------------------------------------------------
BAD_PAGE = 1      # bits of an `errors` word
BAD_POSITION = 2


def kv4_row_bytes(d: int) -> int:
    """Bytes one token of one KV head takes: codes and scales of its key and value."""
    if d not in (64, 128):
        raise ValueError("d must be 64 or 128")
    return d + d // 8


def kv4_cache(num_pages: int, n_kv_heads: int, d: int, page_size: int = 64, device="cuda"):
    """An empty cache (all zeros: every token reads as 0): uint8 [pages, KV heads, page_size * kv4_row_bytes(d)]."""
    return torch.zeros((num_pages, n_kv_heads, page_size * kv4_row_bytes(d)), dtype=torch.uint8, device=device)


class _Cache:
    """A cache with its tables, checked: the arguments its entry points share."""

    def __init__(self, cache, page_table, seq_lens, d, errors):
        if not isinstance(cache, torch.Tensor) or cache.dim() != 3 or cache.dtype != torch.uint8:
            raise TypeError("cache must be a uint8 tensor [pages, KV heads, bytes]")
        if not cache.is_contiguous():
            raise ValueError("cache must be contiguous")
        self.device = cache.device
        self.pages, self.heads, page_bytes = cache.shape
        self.page_size, rest = divmod(page_bytes, kv4_row_bytes(d))
        if rest:
            raise ValueError(f"a page of {page_bytes} bytes does not hold whole tokens of d = {d}")
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be an int32 tensor [sequences, pages]")
        self.n, self.max_pages = page_table.shape
        fa._check("page_table", page_table, torch.int32, page_table.shape, self.device)
        fa._check("seq_lens", seq_lens, torch.int32, (self.n,), self.device)
        if errors is not None:
            fa._check("errors", errors, torch.int32, (1,), self.device)
        self.tensors = [t for t in (cache, page_table, seq_lens, errors) if t is not None]
        self.errors = None if errors is None else errors.data_ptr()


def kv4_store(cache, k, v, page_table, seq_lens, cu_seqlens, k_scale: float = 1.0, v_scale: float = 1.0,
              errors=None, stream=None) -> None:
    """Quantises new keys and values to 4 bits into the pages of their sequences.

    k, v: bf16 [T, KV heads, d], any token stride; sequence i brings tokens
    cu_seqlens[i] .. cu_seqlens[i+1] - 1, which become the last ones of the
    seq_lens[i] tokens it has with them.  page_table: int32 [sequences, pages];
    seq_lens, cu_seqlens: int32, all on the GPU.  ``k_scale`` and ``v_scale``
    are powers of two, the same for every use of the cache.  ``errors``: an
    int32 tensor of one element in which BAD_PAGE and BAD_POSITION are set for
    tokens that were skipped.
    """
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a bf16 tensor [T, KV heads, d]")
    T, heads, d = k.shape
    c = _Cache(cache, page_table, seq_lens, d, errors)
    strides = [_check_tokens("k", k, c.heads, d, c.device), _check_tokens("v", v, c.heads, d, c.device, tokens=T)]
    fa._check("cu_seqlens", cu_seqlens, torch.int32, (c.n + 1,), c.device)
    target = _Target(c.device, stream)
    with target as handle:
        _checked(lib().fa_kv4_store(k.data_ptr(), v.data_ptr(), cache.data_ptr(), page_table.data_ptr(),
                                    seq_lens.data_ptr(), cu_seqlens.data_ptr(), T, c.n, c.max_pages, c.pages,
                                    c.page_size, c.heads, d, *strides, float(k_scale), float(v_scale), c.errors,
                                    handle))
    target.uses(k, v, cu_seqlens, *c.tensors)


def fa_kv4_load(cache, page_table, seq_lens, cu_seqlens, k, v, k_scale: float = 1.0, v_scale: float = 1.0,
                errors=None, stream=None) -> None:
    """Reads cached keys and values back into caller-owned bf16 k and v [T, KV heads, d], contiguous.

    The tokens are those kv4_store with the same tables writes.  Rows of k and
    v outside all sequences are left as they were; a token whose page or
    position is refused is loaded as zeros.
    """
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a bf16 tensor [T, KV heads, d]")
    T, _, d = k.shape
    c = _Cache(cache, page_table, seq_lens, d, errors)
    fa._check("k", k, torch.bfloat16, (T, c.heads, d), c.device)
    fa._check("v", v, torch.bfloat16, (T, c.heads, d), c.device)
    fa._check("cu_seqlens", cu_seqlens, torch.int32, (c.n + 1,), c.device)
    target = _Target(c.device, stream)
    with target as handle:
        _checked(lib().fa_kv4_load(cache.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
                                   cu_seqlens.data_ptr(), k.data_ptr(), v.data_ptr(), T, c.n, c.max_pages, c.pages,
                                   c.page_size, c.heads, d, float(k_scale), float(v_scale), c.errors, handle))
    target.uses(k, v, cu_seqlens, *c.tensors)


def kv4_load(cache, page_table, seq_lens, cu_seqlens, n_tokens: int, d: int, k_scale: float = 1.0,
             v_scale: float = 1.0, errors=None, stream=None):
    """Allocating form of fa_kv4_load: returns (k, v), bf16 [n_tokens, KV heads, d].

    Rows outside all sequences hold nothing of use.
    """
    if not isinstance(cache, torch.Tensor) or cache.dim() != 3:
        raise TypeError("cache must be a uint8 tensor [pages, KV heads, bytes]")
    target = _Target(cache.device, stream)
    with target:
        k = torch.empty((n_tokens, cache.shape[1], d), dtype=torch.bfloat16, device=cache.device)
        v = torch.empty_like(k)
    fa_kv4_load(cache, page_table, seq_lens, cu_seqlens, k, v, k_scale=k_scale, v_scale=v_scale, errors=errors,
                stream=stream)
    return target.gives(k, v)


def fa_kv4_attention(q, cache, page_table, seq_lens, o, lse, n_queries: int = 1, scale: float | None = None,
                     k_scale: float = 1.0, v_scale: float = 1.0, errors=None, stream=None) -> None:
    """Attention of each sequence's n_queries newest tokens over its cached keys and values, into caller-owned O, LSE.

    q: bf16 [sequences * n_queries, Hq, d], any token stride, a sequence's
    tokens together and in order; they stand at the last n_queries of its
    seq_lens[i] positions, store their own keys and values first.  Each sees
    the positions up to its own; one that sees none gets O = 0, LSE = -inf.
    o: bf16 like q, lse: fp32 [Hq, sequences * n_queries], contiguous.
    """
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a bf16 tensor [T, Hq, d]")
    T, Hq, d = q.shape
    c = _Cache(cache, page_table, seq_lens, d, errors)
    if n_queries < 1:
        raise ValueError("n_queries must be at least 1")
    stride = _check_tokens("q", q, Hq, d, c.device, tokens=c.n * n_queries)
    fa._check("o", o, torch.bfloat16, (T, Hq, d), c.device)
    fa._check("lse", lse, torch.float32, (Hq, T), c.device)
    target = _Target(c.device, stream)
    need = ctypes.c_size_t(0)
    handle_lib = lib()
    with target as handle:
        _checked(handle_lib.fa_kv4_attention_workspace(c.n, n_queries, Hq, c.heads, d, c.max_pages, c.page_size,
                                                       ctypes.byref(need)))
        ws = torch.empty(need.value, dtype=torch.uint8, device=c.device) if need.value else None
        _checked(handle_lib.fa_kv4_attention(q.data_ptr(), cache.data_ptr(), page_table.data_ptr(),
                                             seq_lens.data_ptr(), o.data_ptr(), lse.data_ptr(), c.n, n_queries, Hq,
                                             c.heads, d, c.max_pages, c.pages, c.page_size, stride, _scale(scale, d),
                                             float(k_scale), float(v_scale), c.errors,
                                             None if ws is None else ws.data_ptr(), need.value, handle))
    target.uses(q, o, lse, *c.tensors)


def kv4_attention(q, cache, page_table, seq_lens, n_queries: int = 1, scale: float | None = None,
                  k_scale: float = 1.0, v_scale: float = 1.0, errors=None, stream=None):
    """Allocating form of fa_kv4_attention: returns (O, LSE)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a bf16 tensor [T, Hq, d]")
    target = _Target(q.device, stream)
    with target:
        o = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    fa_kv4_attention(q, cache, page_table, seq_lens, o, lse, n_queries=n_queries, scale=scale, k_scale=k_scale,
                     v_scale=v_scale, errors=errors, stream=stream)
    return target.gives(o, lse)
