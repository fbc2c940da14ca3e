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

import ctypes
import functools
import math
import operator

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


# what torch.cuda.current_stream and current_device ask, without the objects they make
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


class _Target:
    """The device and stream of one call: ``with _Target(...) as handle`` makes them current.

    Without a stream the call runs on the device's current one, where the usual
    case, tensors on the current device, needs no change of either.
    """

    __slots__ = ("context", "handle", "stream", "other")

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise ValueError("tensors must be on a CUDA device")
        self.context = self.stream = self.other = None
        if stream is None:
            index = device.index
            self.handle = _raw_stream(index)
            if _current_device() != index:
                self.context = torch.cuda.device(device)
            return
        if not isinstance(stream, torch.cuda.Stream):
            stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                      else torch.cuda.default_stream(device))
        if stream.device != device:
            raise ValueError(f"stream must be on {device}, got {stream.device}")
        caller = torch.cuda.current_stream(device)
        self.handle, self.context = stream.cuda_stream, torch.cuda.stream(stream)
        if caller != stream:
            self.stream, self.other = stream, caller

    def __enter__(self) -> int:
        if self.context is not None:
            self.context.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.context is not None:
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


def _check(name, t, dtype, shape, device) -> None:
    """fa._check, with the usual case decided in one expression."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device.index
            and t.is_contiguous()):
        fa._check(name, t, dtype, shape, device)


def _check_tokens(name, t, heads, d, device, tokens) -> int:
    """Checks a bf16 [T, heads, d] tensor whose tokens may be strided; returns the token stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != (tokens, heads, d):
        raise ValueError(f"{name} must have shape {(tokens, heads, d)}, got {tuple(t.shape)}")
    if t.get_device() != device.index and t.device != device:  # (a CPU tensor's are -1 and None)
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    token, head, element = t.stride()
    if tokens == 0:
        return heads * d
    if (heads > 1 and head != d) or element != 1:
        raise ValueError(f"{name} must have the heads of a token contiguous")
    return token if tokens > 1 else heads * d  # one token's stride says nothing


def _lengths(seq_lens, T):
    """The lengths as a C array, and their number; checked here, since ctypes would wrap what an int does not hold."""
    lens = [operator.index(x) for x in (seq_lens.tolist() if isinstance(seq_lens, torch.Tensor) else seq_lens)]
    n, total = len(lens), sum(lens)
    if n and min(lens) < 0:
        raise ValueError("sequence lengths must not be negative")
    if total > T:
        raise ValueError(f"the sequences hold {total} tokens, the tensors {T}")
    return (_I * n)(*lens), n


def _packed(q, k, v, o, lse, seq_lens, causal, scale, stream):
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor):
        raise TypeError("q and k must be torch.Tensors")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [T, Hq, d] and k [T, Hkv, d]")
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    dev = q.device
    target = _Target(dev, stream) if dev.type == "cuda" else None
    strides = (_check_tokens("q", q, Hq, d, dev, T), _check_tokens("k", k, Hkv, d, dev, T),
               _check_tokens("v", v, Hkv, d, dev, T))
    lens, n = _lengths(seq_lens, T)
    if o is not None:
        _check("o", o, torch.bfloat16, (T, Hq, d), dev)
        _check("lse", lse, torch.float32, (Hq, T), dev)
    if target is None:
        raise ValueError("tensors must be on a CUDA device")
    c = lib()
    causal = 1 if causal else 0
    with target as handle:
        if o is None:
            o = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=dev)
            lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
        args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), lens, n, T, Hq, Hkv, d, *strides,
                causal, 1.0 / math.sqrt(d) if scale is None else scale)
        # most calls split no item and need no workspace; the others are told so, with nothing launched
        rc = c.fa_fwd_packed(*args, None, 0, handle)
        if rc == fa.FA_ERR_SCRATCH:
            need = _Z(0)
            _checked(c.fa_fwd_packed_workspace(lens, n, T, Hq, Hkv, d, causal, ctypes.byref(need)))
            ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
            rc = c.fa_fwd_packed(*args, ws.data_ptr(), need.value, handle)
        if rc != FA_OK:
            raise FAError(rc)
    target.uses(q, k, v)
    return target, o, lse


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
    if o is None or lse is None:
        raise TypeError("o and lse must be torch.Tensors")
    target, _, _ = _packed(q, k, v, o, lse, seq_lens, causal, scale, stream)
    target.uses(o, lse)


def attention_packed(q, k, v, seq_lens, causal: bool = True, scale: float | None = None, stream=None):
    """Allocating form of fa_fwd_packed: returns (O, LSE).

    Rows of tokens behind the last sequence hold nothing of use.
    """
    target, o, lse = _packed(q, k, v, None, None, seq_lens, causal, scale, stream)
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

    __slots__ = ("device", "pages", "heads", "page_size", "n", "max_pages", "tensors", "errors")

    def __init__(self, cache, page_table, seq_lens, d, errors):
        if not isinstance(cache, torch.Tensor) or cache.dim() != 3 or cache.dtype is not torch.uint8:
            raise TypeError("cache must be a uint8 tensor [pages, KV heads, bytes]")
        if not cache.is_contiguous():
            raise ValueError("cache must be contiguous")
        dev = self.device = cache.device
        self.pages, self.heads, page_bytes = cache.shape
        self.page_size, rest = divmod(page_bytes, kv4_row_bytes(d))
        if rest:
            raise ValueError(f"a page of {page_bytes} bytes does not hold whole tokens of d = {d}")
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be an int32 tensor [sequences, pages]")
        self.n, self.max_pages = page_table.shape
        _check("page_table", page_table, torch.int32, page_table.shape, dev)
        _check("seq_lens", seq_lens, torch.int32, (self.n,), dev)
        if errors is None:
            self.tensors, self.errors = (cache, page_table, seq_lens), None
        else:
            _check("errors", errors, torch.int32, (1,), dev)
            self.tensors, self.errors = (cache, page_table, seq_lens, errors), errors.data_ptr()


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
    strides = _check_tokens("k", k, c.heads, d, c.device, T), _check_tokens("v", v, c.heads, d, c.device, T)
    _check("cu_seqlens", cu_seqlens, torch.int32, (c.n + 1,), c.device)
    target = _Target(c.device, stream)
    with target as handle:
        _checked(lib().fa_kv4_store(k.data_ptr(), v.data_ptr(), cache.data_ptr(), page_table.data_ptr(),
                                    seq_lens.data_ptr(), cu_seqlens.data_ptr(), T, c.n, c.max_pages, c.pages,
                                    c.page_size, c.heads, d, *strides, k_scale, v_scale, c.errors,
                                    handle))
    target.uses(k, v, cu_seqlens, *c.tensors)


def _load(cache, page_table, seq_lens, cu_seqlens, k, v, n_tokens, d, k_scale, v_scale, errors, stream):
    c = _Cache(cache, page_table, seq_lens, d, errors)
    dev, shape = c.device, (n_tokens, c.heads, d)
    _check("cu_seqlens", cu_seqlens, torch.int32, (c.n + 1,), dev)
    if k is not None:
        _check("k", k, torch.bfloat16, shape, dev)
        _check("v", v, torch.bfloat16, shape, dev)
    target = _Target(dev, stream)
    with target as handle:
        if k is None:
            k = torch.empty(shape, dtype=torch.bfloat16, device=dev)
            v = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        _checked(lib().fa_kv4_load(cache.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
                                   cu_seqlens.data_ptr(), k.data_ptr(), v.data_ptr(), n_tokens, c.n, c.max_pages,
                                   c.pages, c.page_size, c.heads, d, k_scale, v_scale, c.errors, handle))
    target.uses(cu_seqlens, *c.tensors)
    return target, k, v


def fa_kv4_load(cache, page_table, seq_lens, cu_seqlens, k, v, k_scale: float = 1.0, v_scale: float = 1.0,
                errors=None, stream=None) -> None:
    """Reads cached keys and values back into caller-owned bf16 k and v [T, KV heads, d], contiguous.

    The tokens are those kv4_store with the same tables writes.  Rows of k and
    v outside all sequences are left as they were; a token whose page or
    position is refused is loaded as zeros.
    """
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a bf16 tensor [T, KV heads, d]")
    target, _, _ = _load(cache, page_table, seq_lens, cu_seqlens, k, v, k.shape[0], k.shape[2], k_scale, v_scale, errors,
                         stream)
    target.uses(k, v)


def kv4_load(cache, page_table, seq_lens, cu_seqlens, n_tokens: int, d: int, k_scale: float = 1.0,
             v_scale: float = 1.0, errors=None, stream=None):
    """Allocating form of fa_kv4_load: returns (k, v), bf16 [n_tokens, KV heads, d].

    Rows outside all sequences hold nothing of use.
    """
    target, k, v = _load(cache, page_table, seq_lens, cu_seqlens, None, None, n_tokens, d, k_scale, v_scale, errors,
                         stream)
    return target.gives(k, v)


@functools.lru_cache(maxsize=1024)
def _attention_workspace(device_index, n, n_queries, Hq, heads, d, max_pages, page_size) -> int:
    """fa_kv4_attention_workspace for these sizes (on the current device, which device_index names)."""
    need = _Z(0)
    _checked(lib().fa_kv4_attention_workspace(n, n_queries, Hq, heads, d, max_pages, page_size, ctypes.byref(need)))
    return need.value


def _kv4_attention(q, cache, page_table, seq_lens, o, lse, n_queries, scale, k_scale, v_scale, errors, stream):
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a bf16 tensor [T, Hq, d]")
    T, Hq, d = q.shape
    c = _Cache(cache, page_table, seq_lens, d, errors)
    dev = c.device
    if n_queries < 1:
        raise ValueError("n_queries must be at least 1")
    stride = _check_tokens("q", q, Hq, d, dev, c.n * n_queries)
    if o is not None:
        _check("o", o, torch.bfloat16, (T, Hq, d), dev)
        _check("lse", lse, torch.float32, (Hq, T), dev)
    target = _Target(dev, stream)
    with target as handle:
        if o is None:
            o = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=dev)
            lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
        need = _attention_workspace(dev.index, c.n, n_queries, Hq, c.heads, d, c.max_pages, c.page_size)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _checked(lib().fa_kv4_attention(q.data_ptr(), cache.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
                                        o.data_ptr(), lse.data_ptr(), c.n, n_queries, Hq, c.heads, d, c.max_pages,
                                        c.pages, c.page_size, stride, 1.0 / math.sqrt(d) if scale is None else scale,
                                        k_scale, v_scale, c.errors, None if ws is None else ws.data_ptr(), need, handle))
    target.uses(q, *c.tensors)
    return target, o, lse


def fa_kv4_attention(q, cache, page_table, seq_lens, o, lse, n_queries: int = 1, scale: float | None = None,
                     k_scale: float = 1.0, v_scale: float = 1.0, errors=None, stream=None) -> None:
    """Attention of each sequence's n_queries newest tokens over its cached keys and values, into caller-owned O, LSE.

    q: bf16 [sequences * n_queries, Hq, d], any token stride, a sequence's
    tokens together and in order; they stand at the last n_queries of its
    seq_lens[i] positions, store their own keys and values first.  Each sees
    the positions up to its own; one that sees none gets O = 0, LSE = -inf.
    o: bf16 like q, lse: fp32 [Hq, sequences * n_queries], contiguous.
    """
    if o is None or lse is None:
        raise TypeError("o and lse must be torch.Tensors")
    target, _, _ = _kv4_attention(q, cache, page_table, seq_lens, o, lse, n_queries, scale, k_scale, v_scale, errors,
                                  stream)
    target.uses(o, lse)


def kv4_attention(q, cache, page_table, seq_lens, n_queries: int = 1, scale: float | None = None,
                  k_scale: float = 1.0, v_scale: float = 1.0, errors=None, stream=None):
    """Allocating form of fa_kv4_attention: returns (O, LSE)."""
    target, o, lse = _kv4_attention(q, cache, page_table, seq_lens, None, None, n_queries, scale, k_scale, v_scale,
                                    errors, stream)
    return target.gives(o, lse)
