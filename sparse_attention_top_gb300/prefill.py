"""From the prompt to the cache: norms and rotation of queries and keys with the
cache write in the same pass, attention over packed prompts, and caches held in 4
bits with attention over them.

Bindings of ``gbtopk_rotate_and_cache``, ``gbtopk_rotate_and_cache_int4``,
``gbtopk_cache_read_int4``, ``gbtopk_tree_attention_int4``,
``gbtopk_selected_attention_int4`` and ``gbtopk_prompt_attention`` (``include/gbtopk.h``, which states the formulas and
the rows of a 4-bit cache).  Slots are those of the decode step's calls.  A
4-bit cache is a uint8 tensor [num_slots, kv_heads, int4_row_bytes(head_dim)]
whose slot and head strides are multiples of 16 bytes.  (For attention over it
their greatest common divisor is a row or more, as in any view of a contiguous
tensor whose last axis is the row.)
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

import sparse_attention_top_gb300 as _gb

from .decode import (_F32, _HALF, _I32, _I64, _PAGE_RULE, _PAGES, _QUERY, MAX_PAGE_SIZE, _attention_bytes, _dense, _f, _i32,
                     _i64, _maybe, _outputs, _query, _refuse, _requests, _scratch, _sz, _table, _vp)

__all__ = ["rotate_and_cache", "rotate_and_cache_int4", "read_cache_int4", "CachedRows", "int4_row_bytes", "int4_parts",
           "tree_attention_int4", "selected_attention_int4", "prompt_attention", "gbtopk_prompt_workspace_bytes"]

_TOKENS = [_vp, ctypes.c_int, _i64, _i64, _i64] + [_vp, _i64, _i64] * 2 + [_i32] * 3 + [_vp, _vp, _i32, ctypes.c_int] \
    + [_vp, _vp, ctypes.c_int, _f] + [_vp, _i64, _i64] + [_vp]
_SIGNATURES = {
    "gbtopk_rotate_and_cache": _TOKENS + [_vp, _i64, _i64] * 2 + [_i64, _vp],
    "gbtopk_rotate_and_cache_int4": _TOKENS + [_vp, _i64, _i64, _i64, _f, _f, _vp],
    "gbtopk_tree_attention_int4": _QUERY + [_vp, _i64, _i64, _i64, _f, _f] + _PAGES + [_f, _vp, _vp, _vp, _sz, _vp],
    "gbtopk_selected_attention_int4": _QUERY + [_vp, _i64, _i64, _i64, _f, _f] + [_vp, _i64, _i64]
    + [_f, _vp, _vp, _vp, _sz, _vp],
    "gbtopk_prompt_attention": _QUERY + [_vp, _i64, _i64] * 2 + [_i64, _vp, _vp, _i32, _f, _vp, _vp, _vp, _sz, _vp],
    "gbtopk_cache_read_int4": [_vp, _i64, _i64, _i64, _i32, _i32, _vp, _i64, _f, _f, ctypes.c_int, _vp, _vp, _vp],
}
_calls = None


def _lib():
    global _calls
    if _calls is None:
        lib = _gb.load_library()
        for name, args in _SIGNATURES.items():
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = args
        lib.gbtopk_int4_row_bytes.restype = _i64
        lib.gbtopk_int4_row_bytes.argtypes = [_i32]
        lib.gbtopk_prompt_workspace_bytes.restype = _sz
        lib.gbtopk_prompt_workspace_bytes.argtypes = [_i64, _i32, _i32, _i32, _i32]
        _calls = lib
    return _calls


@functools.lru_cache(maxsize=None)
def int4_row_bytes(head_dim: int) -> int:
    """Bytes of a row of a 4-bit cache: a head's key and value in one slot."""
    n = int(_lib().gbtopk_int4_row_bytes(head_dim)) if 0 < head_dim < 1 << 31 else 0
    if n == 0:
        raise ValueError("head_dim of a 4-bit cache must be a multiple of 16 up to 256")
    return n


def _inner(t) -> bool:
    return t.stride(-1) == 1 or t.shape[-1] < 2


def _heads(q, k, v, same_rows: bool):
    """[rows, heads, dim] queries with keys and values of one shape."""
    if not (isinstance(q, torch.Tensor) and q.is_cuda and q.dim() == 3 and q.dtype in _HALF and _inner(q)):
        _gb._require_cuda(q, "q")
        raise ValueError("q must be a 3-D bf16/fp16 tensor [rows, q_heads, head_dim], inner stride 1")
    for t, name in ((k, "k"), (v, "v")):
        if not (isinstance(t, torch.Tensor) and t.dtype is q.dtype and t.device == q.device and t.dim() == 3 and _inner(t)):
            raise ValueError(f"{name} must be a 3-D {q.dtype} tensor on {q.device}, inner stride 1")
    rows, heads, dim = q.shape
    if not (k.shape == v.shape and k.shape[2] == dim and k.shape[1] >= 1 and heads % k.shape[1] == 0
            and (k.shape[0] == rows or not same_rows)):
        raise ValueError("k and v must be [rows, kv_heads, head_dim] of one shape, q_heads a multiple of kv_heads")
    return rows, heads, k.shape[1], dim


def _tokens(q, k, v, positions, slots, inv_freq, q_weight, k_weight, eps, interleaved, q_out):
    """The arguments that both writes share, up to `slots`, and q_out."""
    try:
        shape, kshape, dt, dev = q.shape, k.shape, q.dtype, q.device
        rows, heads, dim = shape
        kv = kshape[1]
        qs, ks, vs = q.stride(), k.stride(), v.stride()
        if q_out is None:
            q_out, os = torch.empty(shape, dtype=dt, device=dev), (heads * dim, dim, 1)
        else:
            os = q_out.stride()
        freqs = 0 if inv_freq is None else inv_freq.shape[0]
        w = k_weight if q_weight is None else q_weight
        wtype = dt if w is None else w.dtype
        fine = (dt in _HALF and q.is_cuda and k.dtype is dt and v.dtype is dt and k.device == dev and v.device == dev
                and kshape == v.shape and kshape[0] == rows and kshape[2] == dim and kv >= 1 and heads % kv == 0
                and (dim < 2 or qs[2] == ks[2] == vs[2] == os[2] == 1)
                and q_out.shape == shape and q_out.dtype is dt and q_out.device == dev
                and (freqs == 0 or (inv_freq.dtype is _F32 and inv_freq.device == dev and inv_freq.dim() == 1 and inv_freq.is_contiguous()
                                    and positions.dtype is _I32 and positions.device == dev and positions.shape == (rows,)
                                    and positions.is_contiguous()))
                and freqs % 8 == 0 and 2 * freqs <= dim
                and slots.dtype is _I32 and slots.device == dev and slots.shape == (rows,) and slots.is_contiguous()
                and (w is None or ((wtype is dt or wtype is _F32) and _maybe(q_weight, dev, wtype, (dim,))
                                   and _maybe(k_weight, dev, wtype, (dim,)))) and eps >= 0)
    except (AttributeError, IndexError, ValueError, TypeError):
        fine = False
    if not fine:
        _refuse_tokens(q, k, v, positions, slots, inv_freq, q_weight, k_weight, eps, q_out)
    return (q.data_ptr(), _gb._DTYPES[dt], rows, qs[0], qs[1], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
            heads, kv, dim, None if freqs == 0 else positions.data_ptr(), None if freqs == 0 else inv_freq.data_ptr(), freqs,
            1 if interleaved else 0, None if q_weight is None else q_weight.data_ptr(),
            None if k_weight is None else k_weight.data_ptr(), _gb._DTYPES[wtype], eps, q_out.data_ptr(), os[0], os[1],
            slots.data_ptr()), q_out, kv, dim


def _refuse_tokens(q, k, v, positions, slots, inv_freq, q_weight, k_weight, eps, q_out):
    rows, heads, kv, dim = _heads(q, k, v, True)
    dev = q.device
    freqs = 0 if inv_freq is None else inv_freq.numel() if isinstance(inv_freq, torch.Tensor) else -1
    weights = [w for w in (q_weight, k_weight) if w is not None]
    wtype = weights[0].dtype if weights and isinstance(weights[0], torch.Tensor) else q.dtype
    _refuse((freqs == 0 or _dense(inv_freq, dev, _F32, (freqs,)), "inv_freq must be contiguous fp32 [num_freqs]"),
            (freqs == 0 or _dense(positions, dev, _I32, (rows,)), "positions must be contiguous int32 [rows]"),
            (freqs % 8 == 0 and 0 <= 2 * freqs <= dim, "inv_freq must have a multiple of 8 entries, at most head_dim / 2"),
            (_dense(slots, dev, _I32, (rows,)), "slots must be contiguous int32 [rows]"),
            (wtype in (_F32, q.dtype) and all(_dense(w, dev, wtype, (dim,)) for w in weights),
             "the norm weights must be contiguous [head_dim], both fp32 or both of q's type"),
            (eps >= 0, "eps must not be negative"),
            (False, "q_out must be a tensor like q, inner stride 1"))


def rotate_and_cache(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: Optional[torch.Tensor],
                     slots: torch.Tensor, inv_freq: Optional[torch.Tensor], k_cache: torch.Tensor,
                     v_cache: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                     q_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Norms and rotates queries and keys and writes keys and values into the
    caches, in one pass; returns the queries.

    ``q`` [tokens, q_heads, head_dim], ``k`` / ``v`` [tokens, kv_heads,
    head_dim] bf16/fp16 with any strides that are multiples of 8 elements (the
    parts of one projection's output will do); ``positions`` and ``slots``
    int32 [tokens], a token with slot < 0 writes no key and value, the other
    slots all differ; ``inv_freq`` fp32, radians a position of each rotated
    pair (elements i and i + len(inv_freq), or neighbours with
    ``interleaved``), None for no rotation; ``q_weight`` / ``k_weight``
    [head_dim] of ``q``'s type or fp32, None for no norm; caches as for
    ``tree_attention``.  ``q_out`` may be ``q``."""
    args, q_out, kv, dim = _tokens(q, k, v, positions, slots, inv_freq, q_weight, k_weight, eps, interleaved, q_out)
    dev, dt = q.device, q.dtype
    try:
        n = k_cache.shape[0]
        ks, vs = k_cache.stride(), v_cache.stride()
        fine = (k_cache.dtype is dt and v_cache.dtype is dt and k_cache.device == dev and v_cache.device == dev
                and k_cache.shape == (n, kv, dim) and v_cache.shape == (n, kv, dim) and (dim < 2 or ks[2] == vs[2] == 1))
    except (AttributeError, IndexError):
        fine = False
    if not fine:
        raise ValueError("the caches must be [num_slots, kv_heads, head_dim] of q's type and one shape, inner stride 1")
    status = (_calls or _lib()).gbtopk_rotate_and_cache(
        *args, k_cache.data_ptr(), ks[0], ks[1], v_cache.data_ptr(), vs[0], vs[1], n, _gb._stream_handle(dev))
    if status < 0:
        _gb._check(status)
    return q_out


def _int4(cache, dev, kv: Optional[int], dim: int):
    """Slots, heads and strides (bytes) of a 4-bit cache."""
    row = int4_row_bytes(dim)
    try:
        shape, strides = cache.shape, cache.stride()
        if cache.dtype is torch.uint8 and cache.device == dev and shape[2] == row and strides[2] == 1 \
                and len(shape) == 3 and (shape[1] == kv if kv is not None else shape[1] >= 1):
            return shape[0], shape[1], strides
    except (AttributeError, IndexError):
        pass
    raise ValueError(f"cache must be a uint8 tensor [num_slots, kv_heads, int4_row_bytes({dim})] on {dev}, inner stride 1")


def rotate_and_cache_int4(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: Optional[torch.Tensor],
                          slots: torch.Tensor, inv_freq: Optional[torch.Tensor], cache: torch.Tensor,
                          q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                          eps: float = 1e-6, interleaved: bool = False, k_scale: float = 1.0, v_scale: float = 1.0,
                          q_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``rotate_and_cache`` into a 4-bit cache (``head_dim`` a multiple of 16;
    attention over it wants rows on lines of one pitch, see the module).
    ``k_scale`` / ``v_scale``: powers of two, the unit of the cache's scales
    (whose own range, 2^-9 to 448, as a rule needs no other than 1)."""
    args, q_out, kv, dim = _tokens(q, k, v, positions, slots, inv_freq, q_weight, k_weight, eps, interleaved, q_out)
    n, _, cs = _int4(cache, q.device, kv, dim)
    status = (_calls or _lib()).gbtopk_rotate_and_cache_int4(
        *args, cache.data_ptr(), cs[0], cs[1], n, k_scale, v_scale, _gb._stream_handle(q.device))
    if status < 0:
        _gb._check(status)
    return q_out


def int4_parts(cache: torch.Tensor):
    """A 4-bit cache as ``evict_cache`` takes it: two views of its rows, of one
    shape, in place of keys and values.  They overlap where half a row is no
    multiple of 16 bytes; what lies in both is moved twice, to the same place."""
    if not (isinstance(cache, torch.Tensor) and cache.dtype is torch.uint8 and cache.dim() == 3 and cache.shape[2] % 16 == 0
            and cache.stride(2) == 1 and cache.shape[2] > 0):
        raise ValueError("cache must be a 4-bit cache: uint8 [num_slots, kv_heads, row bytes], inner stride 1")
    words = cache.view(torch.int32)
    n = words.shape[2]
    half = (n // 4 + 1) // 2 * 4
    return words[:, :, :half], words[:, :, n - half:]


class CachedRows(NamedTuple):
    k: torch.Tensor   # [n, kv_heads, head_dim]
    v: torch.Tensor


def read_cache_int4(cache: torch.Tensor, slots: torch.Tensor, head_dim: int, dtype: torch.dtype = torch.bfloat16,
                    k_scale: float = 1.0, v_scale: float = 1.0, k_out: Optional[torch.Tensor] = None,
                    v_out: Optional[torch.Tensor] = None) -> CachedRows:
    """Keys and values of the listed slots (int32 [n]) of a 4-bit cache, zeros
    for slots that do not exist."""
    _gb._require_cuda(cache, "cache")
    dev = cache.device
    n, kv, cs = _int4(cache, dev, None, head_dim)
    listed = slots.numel() if isinstance(slots, torch.Tensor) else -1
    shape = (listed, kv, head_dim)
    if not (_dense(slots, dev, _I32, (listed,)) and dtype in _HALF and (k_out is None or _dense(k_out, dev, dtype, shape))
            and (v_out is None or _dense(v_out, dev, dtype, shape))):
        _refuse((_dense(slots, dev, _I32, (listed,)), "slots must be contiguous int32 [n]"),
                (dtype in _HALF, "dtype must be bf16 or fp16"),
                (False, "k_out and v_out must be contiguous [n, kv_heads, head_dim] of dtype"))
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=dev)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dtype, device=dev)
    status = (_calls or _lib()).gbtopk_cache_read_int4(
        cache.data_ptr(), cs[0], cs[1], n, kv, head_dim, slots.data_ptr(), listed, k_scale, v_scale, _gb._DTYPES[dtype],
        k_out.data_ptr(), v_out.data_ptr(), _gb._stream_handle(dev))
    if status < 0:
        _gb._check(status)
    return CachedRows(k_out, v_out)


def tree_attention_int4(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                        page_size: int = 1, next_n: int = 1, tree_mask: Optional[torch.Tensor] = None,
                        scale: Optional[float] = None, k_scale: float = 1.0, v_scale: float = 1.0,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        return_lse: bool = False, workspace: Optional[torch.Tensor] = None):
    """``tree_attention`` over a 4-bit cache; ``k_scale`` / ``v_scale`` as it
    was written with, everything else as there."""
    shape, dev, qs = _query(q)
    rows, heads, dim = shape
    requests = _requests(rows, next_n)
    slots, kv, cs = _int4(cache, dev, None, dim)
    if not (heads % kv == 0 and 1 <= page_size <= MAX_PAGE_SIZE and _table(page_table, dev, requests)
            and _dense(seq_lens, dev, _I32, (requests,)) and _maybe(tree_mask, dev, _I64, (rows,))):
        _refuse((heads % kv == 0, "q_heads must be a multiple of kv_heads"),
                (1 <= page_size <= MAX_PAGE_SIZE, _PAGE_RULE),
                (_table(page_table, dev, requests), "page_table must be int32 [num_requests, pt_cols], inner stride 1"),
                (_dense(seq_lens, dev, _I32, (requests,)), "seq_lens must be contiguous int32 [num_requests]"),
                (False, "tree_mask must be contiguous int64 [num_rows]"))
    out, lse = _outputs(q, shape, dev, out, lse, return_lse)
    lib = _calls or _lib()
    stream = _gb._stream_handle(dev)
    with _gb._LOCKS[dev.index, stream]:
        ws, ws_bytes = _scratch(workspace, dev, stream, _attention_bytes(rows, heads, kv, dim))
        status = lib.gbtopk_tree_attention_int4(
            q.data_ptr(), _gb._DTYPES[q.dtype], rows, qs[0], qs[1], heads, kv, dim, cache.data_ptr(), cs[0], cs[1], slots,
            k_scale, v_scale, page_table.data_ptr(), page_table.shape[1], page_table.stride(0), page_size,
            seq_lens.data_ptr(), next_n, None if tree_mask is None else tree_mask.data_ptr(),
            dim ** -0.5 if scale is None else scale, out.data_ptr(), None if lse is None else lse.data_ptr(), ws,
            ws_bytes, stream)
    if status < 0:
        _gb._check(status)
    return out if lse is None else (out, lse)


def selected_attention_int4(q: torch.Tensor, cache: torch.Tensor, indices: torch.Tensor, scale: Optional[float] = None,
                            k_scale: float = 1.0, v_scale: float = 1.0, out: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                            workspace: Optional[torch.Tensor] = None):
    """``selected_attention`` over a 4-bit cache."""
    shape, dev, qs = _query(q)
    rows, heads, dim = shape
    slots, kv, cs = _int4(cache, dev, None, dim)
    if not (heads % kv == 0 and _table(indices, dev, rows)):
        _refuse((heads % kv == 0, "q_heads must be a multiple of kv_heads"),
                (False, "indices must be int32 [num_rows, top_k], inner stride 1"))
    out, lse = _outputs(q, shape, dev, out, lse, return_lse)
    lib = _calls or _lib()
    stream = _gb._stream_handle(dev)
    with _gb._LOCKS[dev.index, stream]:
        ws, ws_bytes = _scratch(workspace, dev, stream, _attention_bytes(rows, heads, kv, dim))
        status = lib.gbtopk_selected_attention_int4(
            q.data_ptr(), _gb._DTYPES[q.dtype], rows, qs[0], qs[1], heads, kv, dim, cache.data_ptr(), cs[0], cs[1], slots,
            k_scale, v_scale, indices.data_ptr(), indices.shape[1], indices.stride(0),
            dim ** -0.5 if scale is None else scale, out.data_ptr(), None if lse is None else lse.data_ptr(), ws,
            ws_bytes, stream)
    if status < 0:
        _gb._check(status)
    return out if lse is None else (out, lse)


def gbtopk_prompt_workspace_bytes(num_rows: int, num_seqs: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(_lib().gbtopk_prompt_workspace_bytes(num_rows, num_seqs, q_heads, kv_heads, head_dim))


# (packed prompts have another number of rows in nearly every call)
_prompt_bytes = functools.lru_cache(maxsize=256)(gbtopk_prompt_workspace_bytes)


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     cu_seqlens_k: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     return_lse: bool = False, workspace: Optional[torch.Tensor] = None):
    """Causal attention over packed sequences: rows ``cu_seqlens[i] ..
    cu_seqlens[i + 1]`` of ``q`` [rows, q_heads, head_dim] over the keys and
    values of the same offsets, or of ``cu_seqlens_k``, aligned at their ends
    (a chunk of a prompt behind its earlier context; rows that see nothing are
    zero with ``lse`` -inf).  int32 offsets that ascend, on the device: a
    captured call follows them.  Rows behind the last sequence are left as they were in
    ``out`` and ``lse`` (undefined where those are made here).  Everything else
    as for ``tree_attention``."""
    rows, heads, kv, dim = _heads(q, k, v, False)
    dev, shape = q.device, q.shape
    n = cu_seqlens.numel() if isinstance(cu_seqlens, torch.Tensor) else 0
    if not (n >= 1 and _dense(cu_seqlens, dev, _I32, (n,)) and _maybe(cu_seqlens_k, dev, _I32, (n,))):
        _refuse((n >= 1 and _dense(cu_seqlens, dev, _I32, (n,)), "cu_seqlens must be contiguous int32 [num_seqs + 1]"),
                (False, "cu_seqlens_k must be contiguous int32 [num_seqs + 1]"))
    out, lse = _outputs(q, shape, dev, out, lse, return_lse)
    lib = _calls or _lib()
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    stream = _gb._stream_handle(dev)
    with _gb._LOCKS[dev.index, stream]:
        ws, ws_bytes = _scratch(workspace, dev, stream, _prompt_bytes(rows, n - 1, heads, kv, dim))
        status = lib.gbtopk_prompt_attention(
            q.data_ptr(), _gb._DTYPES[q.dtype], rows, qs[0], qs[1], heads, kv, dim, k.data_ptr(), ks[0], ks[1], v.data_ptr(),
            vs[0], vs[1], k.shape[0], cu_seqlens.data_ptr(), None if cu_seqlens_k is None else cu_seqlens_k.data_ptr(), n - 1,
            dim ** -0.5 if scale is None else scale, out.data_ptr(), None if lse is None else lse.data_ptr(), ws, ws_bytes,
            stream)
    if status < 0:
        _gb._check(status)
    return out if lse is None else (out, lse)
