"""The decode step after the selection: attention over a paged cache, the
weight each cached position accumulates, eviction by it, and the verification
of drafted tokens.

Bindings of ``gbtopk_tree_attention``, ``gbtopk_selected_attention``,
``gbtopk_cache_weights``, ``gbtopk_cache_evict`` and ``gbtopk_verify_drafts``
(``include/gbtopk.h``, which states the formulas).  Rows, lengths and slots
follow the top-k calls: row ``r`` is drafted token ``r % next_n`` of request
``r // next_n``, ``seq_lens`` counts the drafted tokens, and position ``p`` of
a request lies in slot ``page_table[i, p // page_size] * page_size +
p % page_size`` - the numbers ``top_k_page_table_transform`` returns.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

import sparse_attention_top_gb300 as _gb

__all__ = [
    "tree_attention", "selected_attention", "accumulate_cache_weights", "evict_cache",
    "verify_drafts", "Verified", "Evicted", "MAX_NEXT_N", "MAX_HEAD_DIM",
    "gbtopk_attention_workspace_bytes", "gbtopk_verify_workspace_bytes",
]

MAX_NEXT_N = 64
MAX_HEAD_DIM = 256

_i32, _i64, _vp, _sz, _f = (ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                            ctypes.c_float)
_QUERY = [_vp, ctypes.c_int, _i64, _i64, _i64, _i32, _i32, _i32]
_PAGES = [_vp, _i64, _i64, _i32, _vp, _i32, _vp]   # page table, lengths, next_n, tree mask
_SIGNATURES = {
    "gbtopk_tree_attention": _QUERY + [_vp, _i64, _i64] * 2 + [_i64] + _PAGES
    + [_f, _vp, _vp, _vp, _sz, _vp],
    "gbtopk_selected_attention": _QUERY + [_vp, _i64, _i64] * 2 + [_i64, _vp, _i64, _i64]
    + [_f, _vp, _vp, _vp, _sz, _vp],
    "gbtopk_cache_weights": _QUERY + [_vp, _i64, _i64, _i64, _vp] + _PAGES
    + [_vp, _f, _vp, _i32, _i64, _vp, _sz, _vp],
    "gbtopk_cache_evict": [_vp, _i64, _i32, _i64, _vp, _i32, _vp, _i32, _i32] + [_vp, _i64, _i64] * 2
    + [_i64, _i32, _i32, _i32] + [_vp, _i64, _i64] * 2 + [_i32, _vp, _vp, _vp, _vp],
    "gbtopk_verify_drafts": [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp, _i32, _vp, _vp, _vp]
    + [_vp] * 4 + [_vp, _sz, _vp],
}
_calls = None


def _lib():
    global _calls
    if _calls is None:
        lib = _gb.load_library()
        for name, args in _SIGNATURES.items():
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = args
        lib.gbtopk_attention_workspace_bytes.restype = _sz
        lib.gbtopk_attention_workspace_bytes.argtypes = [_i64, _i32, _i32, _i32]
        lib.gbtopk_verify_workspace_bytes.restype = _sz
        lib.gbtopk_verify_workspace_bytes.argtypes = [_i64, _i64, _i32]
        _calls = lib
    return _calls


def gbtopk_attention_workspace_bytes(num_rows: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(_lib().gbtopk_attention_workspace_bytes(num_rows, q_heads, kv_heads, head_dim))


def gbtopk_verify_workspace_bytes(num_rows: int, vocab: int, next_n: int) -> int:
    return int(_lib().gbtopk_verify_workspace_bytes(num_rows, vocab, next_n))


def _tensor(t, name: str, device, dtype, shape=None, contiguous: bool = True):
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _query(q):
    _gb._require_cuda(q, "q")
    if q.dim() != 3 or q.dtype not in (torch.bfloat16, torch.float16) or (q.shape[2] > 1 and q.stride(2) != 1):
        raise ValueError("q must be a 3-D bf16/fp16 tensor [num_rows, q_heads, head_dim], inner stride 1")


def _cache(t, name: str, q, like=None):
    if not isinstance(t, torch.Tensor) or t.device != q.device or t.dtype != q.dtype:
        raise ValueError(f"{name} must be a {q.dtype} tensor on {q.device}")
    if t.dim() != 3 or t.shape[2] != q.shape[2] or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name} must be [num_slots, kv_heads, head_dim] with inner stride 1")
    if like is not None and t.shape != like.shape:
        raise ValueError("k_cache and v_cache must have one shape")
    if t.shape[1] < 1 or q.shape[1] % t.shape[1] != 0:
        raise ValueError("q_heads must be a multiple of kv_heads")


def _table(t, name: str, device, requests: int):
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.int32 or t.dim() != 2 \
            or t.shape[0] != requests or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be an int32 [num_requests, pt_cols] tensor on {device}, inner stride 1")


def _requests(rows: int, next_n: int) -> int:
    if next_n < 1 or next_n > MAX_NEXT_N or rows % next_n != 0:
        raise ValueError(f"num_rows must be a multiple of next_n, next_n in [1, {MAX_NEXT_N}]")
    return rows // next_n


def _outputs(q, out, lse, return_lse: bool):
    rows, heads, _ = q.shape
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _tensor(out, "out", q.device, q.dtype, tuple(q.shape))
    if lse is not None:
        _tensor(lse, "lse", q.device, torch.float32, (rows, heads))
    elif return_lse:
        lse = torch.empty((rows, heads), dtype=torch.float32, device=q.device)
    return out, lse


def _scratch(workspace, device, nbytes: int):
    if workspace is None:
        return _gb._workspace(device, nbytes)
    _gb._require_cuda(workspace, "workspace")
    return workspace


def _ws_args(ws):
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _strides(t):
    return t.data_ptr(), t.stride(0), t.stride(1)


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   page_table: torch.Tensor, seq_lens: torch.Tensor, page_size: int = 1,
                   next_n: int = 1, tree_mask: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                   workspace: Optional[torch.Tensor] = None):
    """Attention of each request's ``next_n`` newest tokens over its cache.

    ``q`` [num_rows, q_heads, head_dim] bf16/fp16; ``k_cache`` / ``v_cache``
    [num_slots, kv_heads, head_dim] of the same type (any slot and head
    strides that are multiples of 8 elements); ``page_table`` int32
    [num_rows // next_n, pt_cols]; ``seq_lens`` int32, the drafted tokens
    counted.  A row sees the whole context and the drafted tokens whose bit
    is set in its ``tree_mask`` (int64 [num_rows]; None: tokens 0 .. t).
    ``scale`` defaults to ``head_dim ** -0.5``.  Returns ``out`` (like ``q``),
    or ``(out, lse)`` with ``return_lse`` or a given ``lse``; a row that sees
    nothing is zero with ``lse`` -inf."""
    _query(q)
    rows, heads, dim = q.shape
    requests = _requests(rows, next_n)
    _cache(k_cache, "k_cache", q)
    _cache(v_cache, "v_cache", q, k_cache)
    _table(page_table, "page_table", q.device, requests)
    _tensor(seq_lens, "seq_lens", q.device, torch.int32, (requests,))
    if tree_mask is not None:
        _tensor(tree_mask, "tree_mask", q.device, torch.int64, (rows,))
    out, lse = _outputs(q, out, lse, return_lse)
    kv = k_cache.shape[1]
    lib = _lib()
    ws = _scratch(workspace, q.device, lib.gbtopk_attention_workspace_bytes(rows, heads, kv, dim))
    _gb._check(lib.gbtopk_tree_attention(
        q.data_ptr(), _gb._DTYPES[q.dtype], rows, q.stride(0), q.stride(1), heads, kv, dim,
        *_strides(k_cache), *_strides(v_cache), k_cache.shape[0], page_table.data_ptr(),
        page_table.shape[1], page_table.stride(0), page_size, seq_lens.data_ptr(), next_n,
        _gb._ptr(tree_mask), dim ** -0.5 if scale is None else scale, out.data_ptr(), _gb._ptr(lse),
        *_ws_args(ws), _gb._stream_handle(q.device)))
    return out if lse is None else (out, lse)


def selected_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       indices: torch.Tensor, scale: Optional[float] = None,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       return_lse: bool = False, workspace: Optional[torch.Tensor] = None):
    """Attention of each row over its own list of cache slots.

    ``indices`` int32 [num_rows, top_k], as ``top_k_page_table_transform``
    returns them: entries < 0 or beyond the cache are skipped.  Everything
    else as for ``tree_attention``."""
    _query(q)
    rows, heads, dim = q.shape
    _cache(k_cache, "k_cache", q)
    _cache(v_cache, "v_cache", q, k_cache)
    _table(indices, "indices", q.device, rows)
    out, lse = _outputs(q, out, lse, return_lse)
    kv = k_cache.shape[1]
    lib = _lib()
    ws = _scratch(workspace, q.device, lib.gbtopk_attention_workspace_bytes(rows, heads, kv, dim))
    _gb._check(lib.gbtopk_selected_attention(
        q.data_ptr(), _gb._DTYPES[q.dtype], rows, q.stride(0), q.stride(1), heads, kv, dim,
        *_strides(k_cache), *_strides(v_cache), k_cache.shape[0], indices.data_ptr(),
        indices.shape[1], indices.stride(0), dim ** -0.5 if scale is None else scale,
        out.data_ptr(), _gb._ptr(lse), *_ws_args(ws), _gb._stream_handle(q.device)))
    return out if lse is None else (out, lse)


def accumulate_cache_weights(q: torch.Tensor, k_cache: torch.Tensor, lse: torch.Tensor,
                             page_table: torch.Tensor, seq_lens: torch.Tensor,
                             weights: torch.Tensor, page_size: int = 1, next_n: int = 1,
                             tree_mask: Optional[torch.Tensor] = None,
                             accept_mask: Optional[torch.Tensor] = None,
                             scale: Optional[float] = None,
                             workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Adds to ``weights`` (fp32 [num_requests, 1 or kv_heads, width], in
    place) the probability that the rows of ``q`` gave each position, from
    ``tree_attention``'s ``lse``: all rows, or those whose bit is set in
    ``accept_mask`` (int64 [num_requests], ``verify_drafts``'s).  Returns
    ``weights``."""
    _query(q)
    rows, heads, dim = q.shape
    requests = _requests(rows, next_n)
    _cache(k_cache, "k_cache", q)
    _table(page_table, "page_table", q.device, requests)
    _tensor(seq_lens, "seq_lens", q.device, torch.int32, (requests,))
    _tensor(lse, "lse", q.device, torch.float32, (rows, heads))
    kv = k_cache.shape[1]
    _tensor(weights, "weights", q.device, torch.float32)
    if weights.dim() != 3 or weights.shape[0] != requests or weights.shape[1] not in (1, kv):
        raise ValueError("weights must be [num_requests, 1 or kv_heads, width]")
    if tree_mask is not None:
        _tensor(tree_mask, "tree_mask", q.device, torch.int64, (rows,))
    if accept_mask is not None:
        _tensor(accept_mask, "accept_mask", q.device, torch.int64, (requests,))
    lib = _lib()
    ws = _scratch(workspace, q.device, lib.gbtopk_attention_workspace_bytes(rows, heads, kv, dim))
    _gb._check(lib.gbtopk_cache_weights(
        q.data_ptr(), _gb._DTYPES[q.dtype], rows, q.stride(0), q.stride(1), heads, kv, dim,
        *_strides(k_cache), k_cache.shape[0], lse.data_ptr(), page_table.data_ptr(),
        page_table.shape[1], page_table.stride(0), page_size, seq_lens.data_ptr(), next_n,
        _gb._ptr(tree_mask), _gb._ptr(accept_mask), dim ** -0.5 if scale is None else scale,
        weights.data_ptr(), weights.shape[1], weights.shape[2], *_ws_args(ws),
        _gb._stream_handle(q.device)))
    return weights


class Evicted(NamedTuple):
    kept: torch.Tensor       # int32 [num_requests, weight_heads, budget], -1 padded
    new_lens: torch.Tensor   # int32 [num_requests]
    weights: torch.Tensor    # fp32, the kept positions' weights, zeros behind them


def evict_cache(weights: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                page_table: torch.Tensor, seq_lens: torch.Tensor, out_page_table: torch.Tensor,
                budget: int, recent: int = 0, page_size: int = 1, next_n: int = 1,
                accept_mask: Optional[torch.Tensor] = None,
                out_weights: Optional[torch.Tensor] = None) -> Evicted:
    """Keeps at most ``budget`` positions of each request and packs their
    keys and values, in order, into the pages of ``out_page_table`` (pages of
    the same caches that ``page_table`` does not list).

    The last ``recent`` survivors stay, and those of the others with the most
    weight (ties: the lowest position).  With ``accept_mask`` (int64
    [num_requests]) only the drafted tokens whose bit is set survive, of the
    last ``next_n`` positions.  ``weights`` fp32 [num_requests, 1 or kv_heads,
    width]: one choice for all heads, or one for each.  Caches of 2- or 4-byte
    elements."""
    _gb._require_cuda(weights, "weights")
    dev = weights.device
    _tensor(weights, "weights", dev, torch.float32)
    if weights.dim() != 3:
        raise ValueError("weights must be [num_requests, 1 or kv_heads, width]")
    requests, wheads, width = weights.shape
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor) or t.device != dev or t.dim() != 3 \
                or t.element_size() not in (2, 4) or (t.shape[2] > 1 and t.stride(2) != 1):
            raise ValueError(f"{name} must be [num_slots, kv_heads, head_dim] of 2- or 4-byte elements "
                             f"on {dev}, inner stride 1")
    if k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must have one shape and type")
    if wheads not in (1, k_cache.shape[1]):
        raise ValueError("weights must be [num_requests, 1 or kv_heads, width]")
    _table(page_table, "page_table", dev, requests)
    _table(out_page_table, "out_page_table", dev, requests)
    _tensor(seq_lens, "seq_lens", dev, torch.int32, (requests,))
    if accept_mask is not None:
        _tensor(accept_mask, "accept_mask", dev, torch.int64, (requests,))
    if budget < 1 or recent < 0 or page_size < 1 or out_page_table.shape[1] * page_size < budget:
        raise ValueError("budget >= 1, recent >= 0 and room for budget positions in out_page_table are required")
    if out_weights is None:
        out_weights = torch.empty_like(weights)
    else:
        _tensor(out_weights, "out_weights", dev, torch.float32, tuple(weights.shape))
    kept = torch.empty((requests, wheads, budget), dtype=torch.int32, device=dev)
    new_lens = torch.empty((requests,), dtype=torch.int32, device=dev)
    _gb._check(_lib().gbtopk_cache_evict(
        weights.data_ptr(), requests, wheads, width, seq_lens.data_ptr(), next_n,
        _gb._ptr(accept_mask), budget, recent, *_strides(k_cache), *_strides(v_cache),
        k_cache.shape[0], k_cache.shape[1], k_cache.shape[2], k_cache.element_size(),
        page_table.data_ptr(), page_table.shape[1], page_table.stride(0),
        out_page_table.data_ptr(), out_page_table.shape[1], out_page_table.stride(0), page_size,
        kept.data_ptr(), new_lens.data_ptr(), out_weights.data_ptr(), _gb._stream_handle(dev)))
    return Evicted(kept, new_lens, out_weights)


class Verified(NamedTuple):
    accepted: torch.Tensor     # int32 [num_requests]: drafted tokens accepted
    path: torch.Tensor         # int32 [num_requests, next_n]: accepted nodes from the root, -1 padded
    next_token: torch.Tensor   # int32 [num_requests]
    accept_mask: torch.Tensor  # int64 [num_requests]: the path as bits


def verify_drafts(logits: torch.Tensor, tokens: torch.Tensor, uniforms: torch.Tensor,
                  noise: torch.Tensor, next_n: int = 1, tree_mask: Optional[torch.Tensor] = None,
                  temperature: Optional[torch.Tensor] = None,
                  draft_probs: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> Verified:
    """Verifies each request's drafted tokens against the target's logits and
    draws the token that follows the accepted path.

    ``logits`` [num_rows, vocab] fp32/bf16/fp16, row n of a request the
    target's after node n (node 0: the last token already decided); ``tokens``
    int32 [num_rows]; ``uniforms`` fp32 [num_rows] in [0, 1); ``noise`` fp32
    [num_requests, vocab], standard exponential; ``tree_mask`` int64
    [num_rows] or None (a chain); ``temperature`` fp32 [num_requests] or None
    (1), <= 0 greedy; ``draft_probs`` fp32 [num_rows, vocab], what each node's
    child was drawn from (chains), or None for drafts that were chosen and not
    drawn."""
    _gb._require_cuda(logits, "logits")
    dev = logits.device
    if logits.dim() != 2 or logits.dtype not in _gb._DTYPES or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a 2-D fp32/bf16/fp16 tensor with inner stride 1")
    rows, vocab = logits.shape
    requests = _requests(rows, next_n)
    _tensor(tokens, "tokens", dev, torch.int32, (rows,))
    _tensor(uniforms, "uniforms", dev, torch.float32, (rows,))
    _tensor(noise, "noise", dev, torch.float32, (requests, vocab))
    if tree_mask is not None:
        _tensor(tree_mask, "tree_mask", dev, torch.int64, (rows,))
    if temperature is not None:
        _tensor(temperature, "temperature", dev, torch.float32, (requests,))
    if draft_probs is not None:
        if tree_mask is not None:
            raise ValueError("draft_probs needs a chain of drafts (tree_mask None)")
        _tensor(draft_probs, "draft_probs", dev, torch.float32, (rows, vocab))
    accepted = torch.empty((requests,), dtype=torch.int32, device=dev)
    path = torch.empty((requests, next_n), dtype=torch.int32, device=dev)
    next_token = torch.empty((requests,), dtype=torch.int32, device=dev)
    accept_mask = torch.empty((requests,), dtype=torch.int64, device=dev)
    lib = _lib()
    ws = _scratch(workspace, dev, lib.gbtopk_verify_workspace_bytes(rows, vocab, next_n))
    _gb._check(lib.gbtopk_verify_drafts(
        logits.data_ptr(), _gb._DTYPES[logits.dtype], rows, vocab, logits.stride(0),
        tokens.data_ptr(), uniforms.data_ptr(), noise.data_ptr(), next_n, _gb._ptr(tree_mask),
        _gb._ptr(temperature), _gb._ptr(draft_probs), accepted.data_ptr(), path.data_ptr(),
        next_token.data_ptr(), accept_mask.data_ptr(), *_ws_args(ws), _gb._stream_handle(dev)))
    return Verified(accepted, path, next_token, accept_mask)
