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
import functools
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
MAX_PAGE_SIZE = 1 << 30

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


# Each call tests its arguments in one expression of cheap attribute reads (a
# call's host time is what a small batch waits for); only where that fails does
# _refuse look for the reason.

_HALF = (torch.bfloat16, torch.float16)
_F32, _I32, _I64 = torch.float32, torch.int32, torch.int64


def _refuse(*rules):
    for ok, message in rules:
        if not ok:
            raise ValueError(message)
    raise ValueError("invalid arguments")


def _dense(t, dev, dtype, shape) -> bool:
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.shape == shape \
        and t.is_contiguous()


def _maybe(t, dev, dtype, shape) -> bool:
    return t is None or _dense(t, dev, dtype, shape)


def _table(t, dev, rows) -> bool:
    """An int32 matrix of `rows` rows with inner stride 1."""
    return isinstance(t, torch.Tensor) and t.dtype is _I32 and t.device == dev and t.dim() == 2 \
        and t.shape[0] == rows and (t.stride(1) == 1 or t.shape[1] < 2)


def _query(q):
    """(rows, heads, dim), device, strides of the queries."""
    if not (isinstance(q, torch.Tensor) and q.is_cuda and q.dim() == 3 and q.dtype in _HALF):
        _gb._require_cuda(q, "q")
        raise ValueError("q must be a 3-D bf16/fp16 tensor [num_rows, q_heads, head_dim]")
    strides = q.stride()
    if strides[2] != 1 and q.shape[2] > 1:
        raise ValueError("q must have inner stride 1")
    return q.shape, q.device, strides


def _cache(t, q, dev, dim):
    """(slots, kv heads) and strides of a cache for `q`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is q.dtype and t.device == dev and t.dim() == 3):
        raise ValueError(f"the caches must be 3-D {q.dtype} tensors on {dev}")
    slots, heads, d = t.shape
    strides = t.stride()
    if d != dim or (strides[2] != 1 and d > 1) or heads < 1 or q.shape[1] % heads != 0:
        raise ValueError("the caches must be [num_slots, kv_heads, head_dim] with inner stride 1, q_heads a "
                         "multiple of kv_heads")
    return slots, heads, strides


# (numbers beyond the C types would reach the library cut off)
_PAGE_RULE = f"page_size must be in [1, {MAX_PAGE_SIZE}]"


def _requests(rows: int, next_n: int) -> int:
    if next_n < 1 or next_n > MAX_NEXT_N or rows % next_n != 0:
        raise ValueError(f"num_rows must be a multiple of next_n, next_n in [1, {MAX_NEXT_N}]")
    return rows // next_n


def _outputs(q, shape, dev, out, lse, return_lse: bool):
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=dev)
    elif not _dense(out, dev, q.dtype, shape):
        raise ValueError("out must be a contiguous tensor like q")
    if lse is None:
        if return_lse:
            lse = torch.empty(shape[:2], dtype=_F32, device=dev)
    elif not _dense(lse, dev, _F32, shape[:2]):
        raise ValueError("lse must be a contiguous fp32 [num_rows, q_heads] tensor on q's device")
    return out, lse


_attention_bytes = functools.lru_cache(maxsize=None)(gbtopk_attention_workspace_bytes)
_verify_bytes = functools.lru_cache(maxsize=None)(gbtopk_verify_workspace_bytes)


def _scratch(workspace, dev, stream, nbytes: int):
    """Address and size of the caller's workspace, or of the stream's (under
    the stream's lock)."""
    if workspace is None:
        workspace = _gb._WS.get((dev.index, stream))
        if workspace is None or workspace.numel() < nbytes:
            workspace = _gb._workspace(dev, nbytes)
        return workspace.data_ptr(), workspace.numel()
    _gb._check_workspace(workspace, dev)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


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
    nothing is zero with ``lse`` -inf.

    Probabilities are rounded to ``q``'s type for their product with the
    values (relative error up to 2^-8 in bf16 and 2^-11 in fp16 each; scores
    and sums are fp32): the output is off by 1.2 to 1.4 times its own rounding.
    fp16 loses probabilities below about 2^-24 of the largest among the
    neighbouring 128 positions."""
    shape, dev, qs = _query(q)
    rows, heads, dim = shape
    requests = _requests(rows, next_n)
    slots, kv, ks = _cache(k_cache, q, dev, dim)
    vslots, vkv, vs = _cache(v_cache, q, dev, dim)
    if not (slots == vslots and kv == vkv and 1 <= page_size <= MAX_PAGE_SIZE and _table(page_table, dev, requests)
            and _dense(seq_lens, dev, _I32, (requests,)) and _maybe(tree_mask, dev, _I64, (rows,))):
        _refuse((slots == vslots and kv == vkv, "k_cache and v_cache must have one shape"),
                (1 <= page_size <= MAX_PAGE_SIZE, _PAGE_RULE),
                (_table(page_table, dev, requests), "page_table must be int32 [num_requests, pt_cols], inner stride 1"),
                (_dense(seq_lens, dev, _I32, (requests,)), "seq_lens must be contiguous int32 [num_requests]"),
                (False, "tree_mask must be contiguous int64 [num_rows]"))
    out, lse = _outputs(q, shape, dev, out, lse, return_lse)
    lib = _calls or _lib()
    stream = _gb._stream_handle(dev)
    with _gb._LOCKS[dev.index, stream]:
        ws, ws_bytes = _scratch(workspace, dev, stream, _attention_bytes(rows, heads, kv, dim))
        status = lib.gbtopk_tree_attention(
            q.data_ptr(), _gb._DTYPES[q.dtype], rows, qs[0], qs[1], heads, kv, dim, k_cache.data_ptr(), ks[0], ks[1],
            v_cache.data_ptr(), vs[0], vs[1], slots, page_table.data_ptr(), page_table.shape[1], page_table.stride(0),
            page_size, seq_lens.data_ptr(), next_n, None if tree_mask is None else tree_mask.data_ptr(),
            dim ** -0.5 if scale is None else scale, out.data_ptr(), None if lse is None else lse.data_ptr(), ws,
            ws_bytes, stream)
    if status < 0:
        _gb._check(status)
    return out if lse is None else (out, lse)


def selected_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       indices: torch.Tensor, scale: Optional[float] = None,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       return_lse: bool = False, workspace: Optional[torch.Tensor] = None):
    """Attention of each row over its own list of cache slots.

    ``indices`` int32 [num_rows, top_k], as ``top_k_page_table_transform``
    returns them: entries < 0 or beyond the cache are skipped.  Everything
    else as for ``tree_attention``."""
    shape, dev, qs = _query(q)
    rows, heads, dim = shape
    slots, kv, ks = _cache(k_cache, q, dev, dim)
    vslots, vkv, vs = _cache(v_cache, q, dev, dim)
    if not (slots == vslots and kv == vkv and _table(indices, dev, rows)):
        _refuse((slots == vslots and kv == vkv, "k_cache and v_cache must have one shape"),
                (False, "indices must be int32 [num_rows, top_k], inner stride 1"))
    out, lse = _outputs(q, shape, dev, out, lse, return_lse)
    lib = _calls or _lib()
    stream = _gb._stream_handle(dev)
    with _gb._LOCKS[dev.index, stream]:
        ws, ws_bytes = _scratch(workspace, dev, stream, _attention_bytes(rows, heads, kv, dim))
        status = lib.gbtopk_selected_attention(
            q.data_ptr(), _gb._DTYPES[q.dtype], rows, qs[0], qs[1], heads, kv, dim, k_cache.data_ptr(), ks[0], ks[1],
            v_cache.data_ptr(), vs[0], vs[1], slots, indices.data_ptr(), indices.shape[1], indices.stride(0),
            dim ** -0.5 if scale is None else scale, out.data_ptr(), None if lse is None else lse.data_ptr(), ws,
            ws_bytes, stream)
    if status < 0:
        _gb._check(status)
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
    shape, dev, qs = _query(q)
    rows, heads, dim = shape
    requests = _requests(rows, next_n)
    slots, kv, ks = _cache(k_cache, q, dev, dim)
    wshape = weights.shape if isinstance(weights, torch.Tensor) and weights.dim() == 3 else (-1, -1, -1)
    fits = wshape[0] == requests and wshape[1] in (1, kv) and _dense(weights, dev, _F32, wshape)
    if not (fits and 1 <= page_size <= MAX_PAGE_SIZE and _table(page_table, dev, requests)
            and _dense(seq_lens, dev, _I32, (requests,)) and _dense(lse, dev, _F32, shape[:2])
            and _maybe(tree_mask, dev, _I64, (rows,)) and _maybe(accept_mask, dev, _I64, (requests,))):
        _refuse((fits, "weights must be contiguous fp32 [num_requests, 1 or kv_heads, width]"),
                (1 <= page_size <= MAX_PAGE_SIZE, _PAGE_RULE),
                (_table(page_table, dev, requests), "page_table must be int32 [num_requests, pt_cols], inner stride 1"),
                (_dense(seq_lens, dev, _I32, (requests,)), "seq_lens must be contiguous int32 [num_requests]"),
                (_dense(lse, dev, _F32, shape[:2]), "lse must be contiguous fp32 [num_rows, q_heads]"),
                (_maybe(tree_mask, dev, _I64, (rows,)), "tree_mask must be contiguous int64 [num_rows]"),
                (False, "accept_mask must be contiguous int64 [num_requests]"))
    lib = _calls or _lib()
    stream = _gb._stream_handle(dev)
    with _gb._LOCKS[dev.index, stream]:
        ws, ws_bytes = _scratch(workspace, dev, stream, _attention_bytes(rows, heads, kv, dim))
        status = lib.gbtopk_cache_weights(
            q.data_ptr(), _gb._DTYPES[q.dtype], rows, qs[0], qs[1], heads, kv, dim, k_cache.data_ptr(), ks[0], ks[1], slots,
            lse.data_ptr(), page_table.data_ptr(), page_table.shape[1], page_table.stride(0), page_size,
            seq_lens.data_ptr(), next_n, None if tree_mask is None else tree_mask.data_ptr(),
            None if accept_mask is None else accept_mask.data_ptr(), dim ** -0.5 if scale is None else scale,
            weights.data_ptr(), wshape[1], wshape[2], ws, ws_bytes, stream)
    if status < 0:
        _gb._check(status)
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
    if weights.dtype is not _F32 or weights.dim() != 3 or not weights.is_contiguous():
        raise ValueError("weights must be contiguous fp32 [num_requests, 1 or kv_heads, width]")
    wshape = weights.shape
    requests, wheads, width = wshape
    for t in (k_cache, v_cache):
        if not (isinstance(t, torch.Tensor) and t.device == dev and t.dim() == 3 and t.element_size() in (2, 4)
                and (t.stride(2) == 1 or t.shape[2] < 2)):
            raise ValueError(f"the caches must be [num_slots, kv_heads, head_dim] of 2- or 4-byte elements on {dev}, "
                             "inner stride 1")
    slots, kv, dim = k_cache.shape
    one = k_cache.shape == v_cache.shape and k_cache.dtype is v_cache.dtype
    if not (one and wheads in (1, kv) and _table(page_table, dev, requests) and _table(out_page_table, dev, requests)
            and _dense(seq_lens, dev, _I32, (requests,)) and _maybe(accept_mask, dev, _I64, (requests,))
            and 1 <= budget < 1 << 31 and 0 <= recent < 1 << 31 and 1 <= page_size <= MAX_PAGE_SIZE
            and 1 <= next_n <= MAX_NEXT_N and out_page_table.shape[1] * page_size >= budget
            and _maybe(out_weights, dev, _F32, wshape)):
        _refuse((one, "k_cache and v_cache must have one shape and type"),
                (wheads in (1, kv), "weights must be [num_requests, 1 or kv_heads, width]"),
                (_table(page_table, dev, requests), "page_table must be int32 [num_requests, pt_cols], inner stride 1"),
                (_table(out_page_table, dev, requests), "out_page_table must be int32 [num_requests, cols], inner stride 1"),
                (_dense(seq_lens, dev, _I32, (requests,)), "seq_lens must be contiguous int32 [num_requests]"),
                (_maybe(accept_mask, dev, _I64, (requests,)), "accept_mask must be contiguous int64 [num_requests]"),
                (_maybe(out_weights, dev, _F32, wshape), "out_weights must be contiguous fp32 like weights"),
                (1 <= page_size <= MAX_PAGE_SIZE, _PAGE_RULE),
                (1 <= next_n <= MAX_NEXT_N, f"next_n must be in [1, {MAX_NEXT_N}]"),
                (False, "budget in [1, 2**31), recent in [0, 2**31) and room for budget positions in out_page_table are "
                        "required"))
    if out_weights is None:
        out_weights = torch.empty(wshape, dtype=_F32, device=dev)
    kept = torch.empty((requests, wheads, budget), dtype=_I32, device=dev)
    new_lens = torch.empty((requests,), dtype=_I32, device=dev)
    ks, vs = k_cache.stride(), v_cache.stride()
    status = (_calls or _lib()).gbtopk_cache_evict(
        weights.data_ptr(), requests, wheads, width, seq_lens.data_ptr(), next_n,
        None if accept_mask is None else accept_mask.data_ptr(), budget, recent, k_cache.data_ptr(), ks[0], ks[1],
        v_cache.data_ptr(), vs[0], vs[1], slots, kv, dim, k_cache.element_size(), page_table.data_ptr(),
        page_table.shape[1], page_table.stride(0), out_page_table.data_ptr(), out_page_table.shape[1],
        out_page_table.stride(0), page_size, kept.data_ptr(), new_lens.data_ptr(), out_weights.data_ptr(),
        _gb._stream_handle(dev))
    if status < 0:
        _gb._check(status)
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
    if not (_dense(tokens, dev, _I32, (rows,)) and _dense(uniforms, dev, _F32, (rows,))
            and _dense(noise, dev, _F32, (requests, vocab)) and _maybe(tree_mask, dev, _I64, (rows,))
            and _maybe(temperature, dev, _F32, (requests,)) and _maybe(draft_probs, dev, _F32, (rows, vocab))
            and (draft_probs is None or tree_mask is None)):
        _refuse((_dense(tokens, dev, _I32, (rows,)), "tokens must be contiguous int32 [num_rows]"),
                (_dense(uniforms, dev, _F32, (rows,)), "uniforms must be contiguous fp32 [num_rows]"),
                (_dense(noise, dev, _F32, (requests, vocab)), "noise must be contiguous fp32 [num_requests, vocab]"),
                (_maybe(tree_mask, dev, _I64, (rows,)), "tree_mask must be contiguous int64 [num_rows]"),
                (_maybe(temperature, dev, _F32, (requests,)), "temperature must be contiguous fp32 [num_requests]"),
                (draft_probs is None or tree_mask is None, "draft_probs needs a chain of drafts (tree_mask None)"),
                (False, "draft_probs must be contiguous fp32 [num_rows, vocab]"))
    accepted = torch.empty((requests,), dtype=_I32, device=dev)
    path = torch.empty((requests, next_n), dtype=_I32, device=dev)
    next_token = torch.empty((requests,), dtype=_I32, device=dev)
    accept_mask = torch.empty((requests,), dtype=_I64, device=dev)
    lib = _calls or _lib()
    stream = _gb._stream_handle(dev)
    with _gb._LOCKS[dev.index, stream]:
        ws, ws_bytes = _scratch(workspace, dev, stream, _verify_bytes(rows, vocab, next_n))
        status = lib.gbtopk_verify_drafts(
            logits.data_ptr(), _gb._DTYPES[logits.dtype], rows, vocab, logits.stride(0), tokens.data_ptr(),
            uniforms.data_ptr(), noise.data_ptr(), next_n, None if tree_mask is None else tree_mask.data_ptr(),
            None if temperature is None else temperature.data_ptr(),
            None if draft_probs is None else draft_probs.data_ptr(),
            accepted.data_ptr(), path.data_ptr(), next_token.data_ptr(), accept_mask.data_ptr(), ws, ws_bytes, stream)
    if status < 0:
        _gb._check(status)
    return Verified(accepted, path, next_token, accept_mask)
