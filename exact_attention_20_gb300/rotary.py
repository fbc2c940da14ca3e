"""ctypes binding of rotary positions in libfa_gb300.so (include/fa_gb300_rotary.h).

Turning queries and keys by their positions, forward and backward, and
appending new keys and values to the paged 4-bit cache with the turn on the
way.  As in ``serve``, this module checks tensor metadata and passes raw
pointers; streams, devices and errors are as there.  A ``Rope`` is made once per
model (``rope``) and kept; it holds the pairs' speeds as 64-bit fractions of a
turn per position, so far positions lose nothing.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import NamedTuple

import torch

from . import fa, serve
from .fa import FA_OK, FAError
from .serve import _Cache, _check, _check_tokens, _Target

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong
_F = ctypes.c_float
# every function declared in include/fa_gb300_rotary.h, with its ctypes signature
SIGNATURES = {
    "fa_rotate": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _L, _P]),
    "fa_kv4_append": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _L, _L,
                           _L, _F, _F, _P, _P]),
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


class Rope(NamedTuple):
    """How a model turns its heads: the first 2 * len(turns) elements, as pairs."""

    turns: torch.Tensor        # int64 [rot_dim / 2], on the GPU: 2^-64 of a turn per position
    interleaved: bool = False  # pairs (2i, 2i + 1); else (i, i + rot_dim / 2)
    magnitude: float = 1.0     # multiplies cos and sin


# 2^128 / (2 pi), from 2 pi to 39 digits
_TURN = (1 << 128) * 10 ** 38 // 628318530717958647692528676655900576839


def turns(frequencies, device="cuda") -> torch.Tensor:
    """Radians per position (Python floats) as the int64 fractions of a turn that a Rope holds."""
    out = []
    for f in frequencies:
        num, den = float(f).as_integer_ratio()
        x = (num * _TURN // den >> 64) & ((1 << 64) - 1)  # whole turns a position drop out
        out.append(x - (1 << 64) if x >> 63 else x)
    return torch.tensor(out, dtype=torch.int64, device=device)


def frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                original_length: int = 4096, slow: float = 1.0, fast: float = 32.0) -> list[float]:
    """Radians per position of each pair: base ** (-2 i / rot_dim), for contexts ``factor`` times as long by ``scaling``.

    None: as they are.  "linear": all divided by factor.  "base": with a base
    grown so that the slowest pair is divided by factor and the fastest stays.
    "parts": a pair that turns less than ``slow`` times in original_length
    positions is divided by factor, one that turns more than ``fast`` times
    stays, those between go from one to the other.
    """
    if rot_dim % 16 or not 16 <= rot_dim <= 128:
        raise ValueError("rot_dim must be a multiple of 16 up to 128")
    if not (base > 1 and factor >= 1 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError("base must be above 1 and factor at least 1")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "base":
        base *= factor ** (rot_dim / (rot_dim - 2))
    out = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling == "linear":
        return [f / factor for f in out]
    if scaling == "parts":
        if not (original_length > 0 and 0 <= slow < fast):
            raise ValueError("original_length must be positive, and slow below fast")
        share = [min(1.0, max(0.0, (fast - original_length * f / (2 * math.pi)) / (fast - slow))) for f in out]
        return [f * (1.0 - s) + f / factor * s for f, s in zip(out, share)]
    return out


def rope(rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str | None = None,
         factor: float = 1.0, magnitude: float | None = None, device="cuda", **parts) -> Rope:
    """A Rope for ``frequencies(rot_dim, base, scaling, factor, **parts)``.

    ``magnitude``: 1 but for "parts", where it is 1 + 0.1 ln factor, which
    evens out the scores' spread over the longer context.
    """
    f = frequencies(rot_dim, base, scaling, factor, **parts)
    if magnitude is None:
        magnitude = 1.0 + 0.1 * math.log(factor) if scaling == "parts" else 1.0
    return Rope(turns(f, device), interleaved, magnitude)


def _rope(r, d, device) -> int:
    """Checks a Rope; returns rot_dim."""
    if not isinstance(r, Rope):
        raise TypeError("rope must be a Rope")
    t = r.turns
    if isinstance(t, torch.Tensor) and t.dim() == 1:
        rot = 2 * t.shape[0]
        if rot % 16 == 0 and 16 <= rot <= d:
            _check("rope.turns", t, torch.int64, t.shape, device)
            return rot
    raise ValueError(f"rope.turns must be int64 [rot_dim / 2] for a multiple of 16 elements, at most {d}")


def _strides(name, x, shape, device):
    """Checks a bf16 [B, H, N, d] or [T, H, d] tensor; its (batch, token, head) strides."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    if x.get_device() != device.index and x.device != device:  # (a CPU tensor's are -1 and None)
        raise ValueError(f"{name} must be on {device}, got {x.device}")
    s = x.stride()
    if s[-1] != 1 and x.numel():
        raise ValueError(f"{name} must have a head's elements contiguous")
    return (s[0], s[2], s[1]) if len(s) == 4 else (0, s[0], s[1])


@functools.lru_cache(maxsize=1024)
def _stride_array(*strides):
    """The strides as the C array that fa_rotate reads."""
    return (_L * 12)(*strides)


def _rotate(q, k, q_out, k_out, r, positions, backward, stream):
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dev, shape = q.device, q.shape
    if len(shape) == 4:
        B, hq, N, d = shape
    elif len(shape) == 3:
        B, (N, hq, d) = 1, shape
    else:
        raise ValueError("q must be [B, H, N, d] or [T, H, d]")
    dense = len(shape) == 4
    rot = _rope(r, d, dev)
    strides = _strides("q", q, shape, dev)
    hk = 0
    if k is None:
        strides += (0, 0, 0)
    else:
        if not isinstance(k, torch.Tensor) or k.dim() != len(shape):
            raise ValueError("k must have as many dimensions as q")
        hk = k.shape[1]
        kshape = (B, hk, N, d) if dense else (N, hk, d)
        strides += _strides("k", k, kshape, dev)
    position_stride = 0
    if positions is not None:
        # one row for every batch entry, or a row each
        if dense and isinstance(positions, torch.Tensor) and positions.dim() == 2:
            _check("positions", positions, torch.int32, (B, N), dev)
            position_stride = N
        else:
            _check("positions", positions, torch.int32, (N,), dev)
    if q_out is not None:
        strides += _strides("q_out", q_out, shape, dev)
        strides += _strides("k_out", k_out, kshape, dev) if k is not None else (0, 0, 0)
    else:
        strides += (hq * N * d, d, N * d, hk * N * d, d, N * d) if dense else (0, hq * d, d, 0, hk * d, d)
    target = _Target(dev, stream)
    with target as handle:
        if q_out is None:
            q_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
            if k is not None:
                k_out = torch.empty(kshape, dtype=torch.bfloat16, device=dev)
        rc = lib().fa_rotate(q.data_ptr(), k.data_ptr() if hk else None, q_out.data_ptr(), k_out.data_ptr() if hk else None,
                             None if positions is None else positions.data_ptr(), r.turns.data_ptr(), B, N, hq, hk, d, rot,
                             1 if r.interleaved else 0, r.magnitude, backward, _stride_array(*strides), position_stride, handle)
        if rc != FA_OK:
            raise FAError(rc)
    if target.other is not None:
        target.uses(*(t for t in (q, k, positions, r.turns) if t is not None))
    return target, q_out, k_out


def fa_rotate(q, k, q_out, k_out, rope: Rope, positions=None, backward: bool = False, stream=None) -> None:
    """Turns q and k by their tokens' positions, into caller-owned tensors (q and k themselves, to turn in place).

    q: bf16 [B, Hq, N, d] or [T, Hq, d]; k: the same with its own number of
    heads, or None (with k_out None).  Any strides that are multiples of 8 (a
    head's elements contiguous): views of a fused projection's output are fine.
    positions: int32 [N] (or [T]), or [B, N]; None: 0, 1, 2, ...  ``backward``
    turns the other way: gradients of the inputs from those of the outputs.
    """
    if q_out is None or (k is None) != (k_out is None):
        raise TypeError("q_out, and k_out where there is a k, must be torch.Tensors")
    target, _, _ = _rotate(q, k, q_out, k_out, rope, positions, 1 if backward else 0, stream)
    target.uses(q_out, *(() if k is None else (k_out,)))


def _gives(target, q, k):
    return target.gives(q, k) if k is not None else target.gives(q)[0]


def rotate(q, k, rope: Rope, positions=None, stream=None):
    """Allocating form of fa_rotate: returns (q, k) turned, contiguous; q alone where k is None."""
    return _gives(*_rotate(q, k, None, None, rope, positions, 0, stream))


def rotate_backward(dq, dk, rope: Rope, positions=None, stream=None):
    """Gradients of rotate's inputs from those of its outputs (same rope and positions): (dq, dk), or dq alone."""
    return _gives(*_rotate(dq, dk, None, None, rope, positions, 1, stream))


def _append(cache, q, k, v, r, page_table, seq_lens, cu_seqlens, q_out, k_out, want_k, positions, k_scale, v_scale, errors,
            stream):
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a bf16 tensor [T, KV heads, d]")
    T, _, d = k.shape
    c = _Cache(cache, page_table, seq_lens, d, errors)
    dev = c.device
    rot = _rope(r, d, dev)
    ks, vs = _check_tokens("k", k, c.heads, d, dev, T), _check_tokens("v", v, c.heads, d, dev, T)
    hq = qs = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be a bf16 tensor [T, Hq, d]")
        hq = q.shape[1]
        qs = _check_tokens("q", q, hq, d, dev, T)
    _check("cu_seqlens", cu_seqlens, torch.int32, (c.n + 1,), dev)
    if positions is not None:
        _check("positions", positions, torch.int32, (T,), dev)
    if q_out is not None:
        _check("q_out", q_out, torch.bfloat16, (T, hq, d), dev)
    if k_out is not None:
        _check("k_out", k_out, torch.bfloat16, (T, c.heads, d), dev)
    target = _Target(dev, stream)
    with target as handle:
        if q is not None and q_out is None:
            q_out = torch.empty((T, hq, d), dtype=torch.bfloat16, device=dev)
        if want_k and k_out is None:
            k_out = torch.empty((T, c.heads, d), dtype=torch.bfloat16, device=dev)
        rc = lib().fa_kv4_append(None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                 None if q is None else q_out.data_ptr(), None if k_out is None else k_out.data_ptr(),
                                 cache.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens.data_ptr(),
                                 None if positions is None else positions.data_ptr(), r.turns.data_ptr(), T, c.n,
                                 c.max_pages, c.pages, c.page_size, hq, c.heads, d, rot, 1 if r.interleaved else 0,
                                 r.magnitude, qs, ks, vs, k_scale, v_scale, c.errors, handle)
        if rc != FA_OK:
            raise FAError(rc)
    if target.other is not None:
        target.uses(k, v, cu_seqlens, r.turns, *c.tensors, *(t for t in (q, positions) if t is not None))
    return target, q_out, k_out


def fa_kv4_append(cache, q, k, v, rope: Rope, page_table, seq_lens, cu_seqlens, q_out, k_out=None, positions=None,
                  k_scale: float = 1.0, v_scale: float = 1.0, errors=None, stream=None) -> None:
    """Turns new queries and keys and stores keys and values in 4 bits, with the turned q (and k) into caller-owned tensors.

    q: bf16 [T, Hq, d], or None (with q_out None); k, v: bf16 [T, KV heads, d],
    any token stride.  q_out, and k_out where it is wanted: bf16, contiguous.
    positions: int32 [T], the positions to turn by; None: each token's place in
    its sequence.  The cache's arguments are those of ``serve.kv4_store``.  Rows
    of q_out and k_out of tokens outside all sequences are left as they were.
    """
    if (q is None) != (q_out is None):
        raise TypeError("q and q_out must both be torch.Tensors, or None")
    target, _, _ = _append(cache, q, k, v, rope, page_table, seq_lens, cu_seqlens, q_out, k_out, False, positions, k_scale,
                           v_scale, errors, stream)
    target.uses(*(t for t in (q_out, k_out) if t is not None))


def kv4_append(cache, q, k, v, rope: Rope, page_table, seq_lens, cu_seqlens, positions=None, return_k: bool = False,
               k_scale: float = 1.0, v_scale: float = 1.0, errors=None, stream=None):
    """Allocating form of fa_kv4_append: returns the turned q, or with return_k (q, k); q is None where none was given.

    Rows of tokens outside all sequences hold nothing of use.
    """
    target, q_out, k_out = _append(cache, q, k, v, rope, page_table, seq_lens, cu_seqlens, None, None, return_k, positions,
                                   k_scale, v_scale, errors, stream)
    if target.other is not None:
        target.gives(*(t for t in (q_out, k_out) if t is not None))
    return (q_out, k_out) if return_k else q_out
