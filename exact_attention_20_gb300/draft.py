"""ctypes binding of drafted tokens in libfa_gb300.so (include/fa_gb300_draft.h).

A step of speculative decoding over the paged 4-bit cache: the drafted tree's
keys and values are appended (``rotary.kv4_append`` or ``serve.kv4_store``),
its nodes attend to the context and their own line (``kv4_tree_attention``), the
target's logits decide what is kept (``verify_tree``), and the kept nodes move
together in the cache (``kv4_keep``).  As in ``serve``, this module checks tensor
metadata and passes raw pointers; streams, workspaces, devices and errors are
as there.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import fa
from .fa import FA_OK, FAError
from .serve import BAD_PAGE, BAD_POSITION, _Cache, _check, _check_tokens, _checked, _Target  # noqa: F401

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong
_Z = ctypes.c_size_t
_F = ctypes.c_float
# every function declared in include/fa_gb300_draft.h, with its ctypes signature
SIGNATURES = {
    "fa_kv4_tree_attention": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _L, _F, _F, _F, _P, _P, _Z,
                                   _P]),
    "fa_kv4_tree_attention_workspace": (_I, [_I, _I, _I, _I, _I, _I, _I, _P]),
    "fa_verify_tree": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _L, _L, _F, _P]),
    "fa_kv4_keep": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P]),
}
BAD_TREE = 4   # a bit of an `errors` word, beside serve's
MAX_NODES = 64

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


def _nodes(name, t, n, device) -> int:
    """Checks an int32 [sequences, nodes] tensor; returns the number of nodes."""
    shape = t.shape if isinstance(t, torch.Tensor) else ()
    if len(shape) != 2:
        raise ValueError(f"{name} must be an int32 tensor [sequences, nodes]")
    nodes = shape[1]
    if not 1 <= nodes <= MAX_NODES:
        raise ValueError(f"a tree has 1 to {MAX_NODES} places for nodes, got {nodes}")
    _check(name, t, torch.int32, (n, nodes), device)
    return nodes


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=1024)
def _attention_workspace(device_index, n, nodes, Hq, heads, d, max_pages, page_size) -> int:
    """fa_kv4_tree_attention_workspace for these sizes (on the current device, which device_index names)."""
    need = _Z(0)
    _checked(lib().fa_kv4_tree_attention_workspace(n, nodes, Hq, heads, d, max_pages, page_size, ctypes.byref(need)))
    return need.value


def _tree_attention(q, cache, page_table, seq_lens, parents, o, lse, scale, k_scale, v_scale, errors, stream):
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a bf16 tensor [sequences * nodes, Hq, d]")
    T, Hq, d = q.shape
    c = _Cache(cache, page_table, seq_lens, d, errors)
    dev = c.device
    nodes = _nodes("parents", parents, c.n, dev)
    stride = _check_tokens("q", q, Hq, d, dev, c.n * nodes)
    if o is not None:
        _check("o", o, torch.bfloat16, (T, Hq, d), dev)
        _check("lse", lse, torch.float32, (Hq, T), dev)
    target = _Target(dev, stream)
    with target as handle:
        if o is None:
            o = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=dev)
            lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
        need = _attention_workspace(dev.index, c.n, nodes, Hq, c.heads, d, c.max_pages, c.page_size)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        rc = lib().fa_kv4_tree_attention(
            q.data_ptr(), cache.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), parents.data_ptr(), o.data_ptr(),
            lse.data_ptr(), c.n, nodes, Hq, c.heads, d, c.max_pages, c.pages, c.page_size, stride,
            1.0 / math.sqrt(d) if scale is None else scale, k_scale, v_scale, c.errors, None if ws is None else ws.data_ptr(),
            need, handle)
        if rc != FA_OK:
            raise FAError(rc)
    if target.other is not None:
        target.uses(q, parents, *c.tensors)
    return target, o, lse


def fa_kv4_tree_attention(q, cache, page_table, seq_lens, parents, o, lse, scale: float | None = None,
                          k_scale: float = 1.0, v_scale: float = 1.0, errors=None, stream=None) -> None:
    """Attention of a tree of drafted tokens over the cache that holds them, into caller-owned O, LSE.

    parents: int32 [sequences, nodes], up to 64 nodes: node i's parent is a node
    before it, -1 the context; any other value: no node here.  The nodes' keys
    and values are the last ``nodes`` of seq_lens[i] positions.  q: bf16
    [sequences * nodes, Hq, d], any token stride; node i sees the context and
    its line down to itself.  A place without a node gets O = 0, LSE = -inf.
    o: bf16 like q, lse: fp32 [Hq, sequences * nodes], contiguous.  Small trees
    over short contexts are quickest with a page_table not much wider than the
    longest sequence: how a call is divided goes by its width.
    """
    if o is None or lse is None:
        raise TypeError("o and lse must be torch.Tensors")
    target, _, _ = _tree_attention(q, cache, page_table, seq_lens, parents, o, lse, scale, k_scale, v_scale, errors, stream)
    target.uses(o, lse)


def kv4_tree_attention(q, cache, page_table, seq_lens, parents, scale: float | None = None, k_scale: float = 1.0,
                       v_scale: float = 1.0, errors=None, stream=None):
    """Allocating form of fa_kv4_tree_attention: returns (O, LSE)."""
    target, o, lse = _tree_attention(q, cache, page_table, seq_lens, parents, None, None, scale, k_scale, v_scale, errors,
                                     stream)
    return target.gives(o, lse)


# ---------------------------------------------------------------------------
# Verification
# ---------------------------------------------------------------------------
def _rows(name, t, dtypes, n, nodes, V, device):
    """Checks [n, nodes, V] or [n * nodes, V] rows of contiguous elements, evenly spaced; (V, row stride)."""
    shape = t.shape if isinstance(t, torch.Tensor) else ()
    if len(shape) not in (2, 3):
        raise ValueError(f"{name} must be [sequences, nodes, V] or [sequences * nodes, V]")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    V = shape[-1] if V is None else V
    if shape != ((n, nodes, V) if len(shape) == 3 else (n * nodes, V)):
        raise ValueError(f"{name} must have rows of {V} for {n} x {nodes} nodes, got {tuple(shape)}")
    if t.get_device() != device.index and t.device != device:  # (a CPU tensor's are -1 and None)
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    s = t.stride()
    row = s[-2] if nodes > 1 or len(s) == 2 else s[0]
    if V > 1 and s[-1] != 1 or len(s) == 3 and n > 1 and s[0] != nodes * row:
        raise ValueError(f"{name} must have contiguous rows, evenly spaced")
    return V, row if n * nodes > 1 else V


def _verify(logits, tokens, parents, uniforms, draft_probs, path, n_kept, next_token, temperature, stream):
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    dev = logits.device
    if not isinstance(tokens, torch.Tensor) or tokens.dim() != 2:
        raise ValueError("tokens must be an int32 tensor [sequences, nodes]")
    n = tokens.shape[0]
    nodes = _nodes("tokens", tokens, n, dev)
    V, stride = _rows("logits", logits, (torch.bfloat16, torch.float32), n, nodes, None, dev)
    _check("parents", parents, torch.int32, (n, nodes), dev)
    _check("uniforms", uniforms, torch.float32, (n, nodes), dev)
    draft_stride = 0
    if draft_probs is not None:
        _, draft_stride = _rows("draft_probs", draft_probs, (torch.float32,), n, nodes, V, dev)
    if path is not None:
        _check("path", path, torch.int32, (n, nodes), dev)
        _check("n_kept", n_kept, torch.int32, (n,), dev)
        _check("next_token", next_token, torch.int32, (n,), dev)
    target = _Target(dev, stream)
    with target as handle:
        if path is None:
            path = torch.empty((n, nodes), dtype=torch.int32, device=dev)
            n_kept = torch.empty(n, dtype=torch.int32, device=dev)
            next_token = torch.empty(n, dtype=torch.int32, device=dev)
        rc = lib().fa_verify_tree(
            logits.data_ptr(), 1 if logits.dtype is torch.float32 else 0, tokens.data_ptr(), parents.data_ptr(),
            uniforms.data_ptr(), None if draft_probs is None else draft_probs.data_ptr(), path.data_ptr(), n_kept.data_ptr(),
            next_token.data_ptr(), n, nodes, V, stride, draft_stride, temperature, handle)
        if rc != FA_OK:
            raise FAError(rc)
    if target.other is not None:
        target.uses(*(t for t in (logits, tokens, parents, uniforms, draft_probs) if t is not None))
    return target, path, n_kept, next_token


def fa_verify_tree(logits, tokens, parents, uniforms, path, n_kept, next_token, draft_probs=None,
                   temperature: float = 1.0, stream=None) -> None:
    """Which drafted tokens the target keeps, and the token after them, into caller-owned path, n_kept and next_token.

    logits: bf16 or fp32 [sequences, nodes, V] (or [sequences * nodes, V]), rows
    evenly spaced: the target's after each node; V up to 262144.  tokens,
    parents: int32 [sequences, nodes]; node 0, with parent -1, is the context's
    last token, decided already.  uniforms: fp32 [sequences, nodes] from [0, 1):
    node j's decides on it, node 0's draws the next token.  draft_probs: fp32
    like logits, row i what node i's children were drawn from; None: children
    are given, not drawn.  temperature, of all sequences: 0 is the likeliest token alone.
    path: int32 [sequences, nodes], the kept nodes and then -1; n_kept (node 0
    counts) and next_token: int32 [sequences].  What comes out is distributed as
    the target's own samples, whatever the draft.
    """
    if path is None or n_kept is None or next_token is None:
        raise TypeError("path, n_kept and next_token must be torch.Tensors")
    target, *_ = _verify(logits, tokens, parents, uniforms, draft_probs, path, n_kept, next_token, temperature, stream)
    target.uses(path, n_kept, next_token)


def verify_tree(logits, tokens, parents, uniforms, draft_probs=None, temperature: float = 1.0, stream=None):
    """Allocating form of fa_verify_tree: returns (path, n_kept, next_token)."""
    target, *out = _verify(logits, tokens, parents, uniforms, draft_probs, None, None, None, temperature, stream)
    return target.gives(*out)


# ---------------------------------------------------------------------------
# Keeping
# ---------------------------------------------------------------------------
def _keep(cache, page_table, seq_lens, path, n_kept, new_lens, d, errors, stream):
    c = _Cache(cache, page_table, seq_lens, d, errors)
    dev = c.device
    nodes = _nodes("path", path, c.n, dev)
    _check("n_kept", n_kept, torch.int32, (c.n,), dev)
    if new_lens is not None:
        _check("new_lens", new_lens, torch.int32, (c.n,), dev)
    target = _Target(dev, stream)
    with target as handle:
        if new_lens is None:
            new_lens = torch.empty(c.n, dtype=torch.int32, device=dev)
        rc = lib().fa_kv4_keep(cache.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), path.data_ptr(),
                               n_kept.data_ptr(), new_lens.data_ptr(), c.n, nodes, c.max_pages, c.pages, c.page_size,
                               c.heads, d, c.errors, handle)
        if rc != FA_OK:
            raise FAError(rc)
    if target.other is not None:
        target.uses(path, n_kept, *c.tensors)
    return target, new_lens


def fa_kv4_keep(cache, page_table, seq_lens, path, n_kept, new_lens, d: int, errors=None, stream=None) -> None:
    """Moves the kept nodes' keys and values to the first places of their tree, with the new lengths into new_lens.

    path: int32 [sequences, nodes], n_kept: int32 [sequences], as verify_tree
    gives them; seq_lens counts the tree's places, new_lens (int32 [sequences],
    not seq_lens itself) those kept.
    """
    if new_lens is None:
        raise TypeError("new_lens must be a torch.Tensor")
    target, _ = _keep(cache, page_table, seq_lens, path, n_kept, new_lens, d, errors, stream)
    target.uses(new_lens)


def kv4_keep(cache, page_table, seq_lens, path, n_kept, d: int, errors=None, stream=None):
    """Allocating form of fa_kv4_keep: returns the new lengths."""
    target, new_lens = _keep(cache, page_table, seq_lens, path, n_kept, None, d, errors, stream)
    return target.gives(new_lens)[0]
