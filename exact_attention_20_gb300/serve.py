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
