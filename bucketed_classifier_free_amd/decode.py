"""Guided decoding of token models: wrappers over the second part of libbcg's
ABI (include/bcg_decode.h), which states every operator's definition.

As in api.py, argument checks and marshalling only; the work runs inside
libbcg on the current torch stream (or ``stream``), and nothing synchronises.
"""
from __future__ import annotations

import ctypes as ct
from dataclasses import dataclass, field

import torch

from . import _lib as L
from .api import _DT, _dev, _ptr, _stream

_KV = {torch.float32: L.BCG_F32, torch.bfloat16: L.BCG_BF16, torch.float8_e4m3fn: L.BCG_E4M3}


def _dense_rows(t, name, dims):
    """A GPU tensor whose dimensions after the first are contiguous; the
    elements between its rows."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a GPU tensor (got {t.device})")
    if t.dim() != dims:
        raise ValueError(f"{name}: expected {dims} dimensions, got {t.dim()}")
    width = 1
    for d in range(dims - 1, 0, -1):
        if t.shape[d] != 1 and t.stride(d) != width:
            raise ValueError(f"{name}: must be contiguous after its first dimension")
        width *= t.shape[d]
    return t.stride(0) if t.shape[0] > 1 else max(width, t.stride(0))


def _i32(t, name, shape=None, allow_none=False):
    return _dev(t, name, torch.int32, shape, allow_none)


def _f32(t, name, shape=None, allow_none=True):
    return _dev(t, name, torch.float32, shape, allow_none)


def _cache_args(k_cache, v_cache, dtype, block_table, kv_len, k_scale, v_scale):
    """Shapes and strides of one layer's pages: (kv_heads, page_size, dim,
    num_pages, k page stride, v page stride, cache type)."""
    ks, vs = _dense_rows(k_cache, "k_cache", 4), _dense_rows(v_cache, "v_cache", 4)
    if k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must have the same shape and dtype")
    if k_cache.dtype not in _KV or (k_cache.dtype != dtype and not (
            k_cache.dtype == torch.float8_e4m3fn and dtype == torch.bfloat16)):
        raise ValueError(f"a cache of {k_cache.dtype} does not go with {dtype}")
    pages, kvh, page, dim = k_cache.shape
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [rows, max_blocks]")
    _i32(block_table, "block_table")
    _i32(kv_len, "kv_len", (block_table.shape[0],))
    _f32(k_scale, "k_scale", (kvh,))
    _f32(v_scale, "v_scale", (kvh,))
    return kvh, page, dim, pages, ks, vs, _KV[k_cache.dtype]


def attention_workspace(tokens: int, q_heads: int, head_dim: int, device=None):
    """A workspace for the attention calls of up to ``tokens`` query rows
    (keep it from call to call; one for each stream)."""
    n = L.lib().attention_workspace_size(int(tokens), int(q_heads), int(head_dim))
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.device("cuda", torch.cuda.current_device()))


def _attention(prompt, q, q_offset, k_cache, v_cache, block_table, kv_len, out, *, workspace, scale, window, sinks,
               k_scale, v_scale, max_len, max_new, lse, stream):
    q_stride = _dense_rows(q, "q", 3)
    if q.dtype not in _DT:
        raise ValueError("q must be float32 or bfloat16")
    tokens, heads, dim = q.shape
    kvh, page, cdim, pages, ks, vs, kvt = _cache_args(k_cache, v_cache, q.dtype, block_table, kv_len, k_scale, v_scale)
    if cdim != dim:
        raise ValueError(f"head_dim {dim} of q, {cdim} of the cache")
    rows, blocks = block_table.shape
    if prompt:
        _i32(q_offset, "q_offset", (rows + 1,))
    elif rows != tokens:
        raise ValueError(f"{tokens} query rows for {rows} rows of the table")
    _dev(out, "out", q.dtype, q.shape)
    _f32(lse, "lse", (tokens, heads))
    _dev(workspace, "workspace", torch.uint8)
    if max_len is None:
        max_len = blocks * page
    a = L.AttnArgs(rows, tokens, heads, kvh, dim, page, blocks, pages, _DT[q.dtype], kvt, int(max_len),
                   int(tokens if max_new is None else max_new), int(window), int(sinks),
                   float(dim ** -0.5 if scale is None else scale), 0, q_stride, ks, vs, _ptr(q), _ptr(k_cache),
                   _ptr(v_cache), _ptr(block_table), _ptr(kv_len), _ptr(q_offset), _ptr(k_scale), _ptr(v_scale),
                   _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel())
    fn = L.lib().prompt_attention if prompt else L.lib().paged_attention
    L.check(fn(ct.byref(a), _stream(stream)))


def paged_attention(q, k_cache, v_cache, block_table, kv_len, out, *, workspace, scale=None, window: int = 0,
                    sinks: int = 0, k_scale=None, v_scale=None, max_len=None, lse=None, stream=None):
    """One new token a row over its pages: q, out [rows, q_heads, head_dim],
    caches [num_pages, kv_heads, page_size, head_dim] (any page stride); see
    include/bcg_decode.h.  ``max_len``: an upper bound of kv_len that the host
    knows (default: the table's width).  ``scale``: default head_dim ** -0.5."""
    _attention(False, q, None, k_cache, v_cache, block_table, kv_len, out, workspace=workspace, scale=scale, window=window,
               sinks=sinks, k_scale=k_scale, v_scale=v_scale, max_len=max_len, max_new=None, lse=lse, stream=stream)


def prompt_attention(q, q_offset, k_cache, v_cache, block_table, kv_len, out, *, workspace, scale=None,
                     window: int = 0, sinks: int = 0, k_scale=None, v_scale=None, max_len=None, max_new=None,
                     lse=None, stream=None):
    """Runs of new tokens over their rows' pages, causally: row r has the
    queries [q_offset[r], q_offset[r+1]) of q [tokens, q_heads, head_dim], the
    last at position kv_len[r] - 1; see include/bcg_decode.h.  ``max_new``: an
    upper bound of a row's new tokens."""
    _attention(True, q, q_offset, k_cache, v_cache, block_table, kv_len, out, workspace=workspace, scale=scale,
               window=window, sinks=sinks, k_scale=k_scale, v_scale=v_scale, max_len=max_len, max_new=max_new, lse=lse,
               stream=stream)


def cache_append(k, v, k_cache, v_cache, block_table, kv_len, *, offset=None, k_scale=None, v_scale=None, stream=None):
    """New keys and values [tokens, kv_heads, head_dim] (any row stride) into
    one layer's pages; ``offset`` as q_offset (None: one token a row)."""
    ks, vs = _dense_rows(k, "k", 3), _dense_rows(v, "v", 3)
    if k.dtype not in _DT or k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must have the same shape, float32 or bfloat16")
    kvh, page, dim, pages, kps, vps, kvt = _cache_args(k_cache, v_cache, k.dtype, block_table, kv_len, k_scale, v_scale)
    if tuple(k.shape[1:]) != (kvh, dim):
        raise ValueError(f"k and v must be [tokens, {kvh}, {dim}]")
    rows, blocks = block_table.shape
    _i32(offset, "offset", (rows + 1,), allow_none=True)
    if offset is None and rows != k.shape[0]:
        raise ValueError(f"{k.shape[0]} tokens for {rows} rows of the table")
    a = L.AppendArgs(rows, k.shape[0], kvh, dim, page, blocks, pages, _DT[k.dtype], kvt, 0, ks, vs, kps, vps, _ptr(k),
                     _ptr(v), _ptr(offset), _ptr(block_table), _ptr(kv_len), _ptr(k_scale), _ptr(v_scale),
                     _ptr(k_cache), _ptr(v_cache))
    L.check(L.lib().cache_append(ct.byref(a), _stream(stream)))


@dataclass
class PagedCache:
    """The pool of a model's pages and its tables.  ``pool`` is
    [planes, num_pages, kv_heads, page_size, head_dim] (planes 2l and 2l + 1:
    the keys and values of layer l); ``table`` [rows, max_blocks] and
    ``length`` [rows] are what the attention calls take, ``refs`` [num_pages]
    counts the references to each page (int32, on the GPU)."""
    pool: torch.Tensor
    table: torch.Tensor
    length: torch.Tensor
    refs: torch.Tensor
    _workspace: torch.Tensor | None = field(default=None, repr=False)

    def __post_init__(self):
        if not isinstance(self.pool, torch.Tensor) or self.pool.dim() != 5:
            raise ValueError("pool must be [planes, num_pages, kv_heads, page_size, head_dim]")
        _dense_rows(self.pool[0], "pool", 4)
        if not isinstance(self.table, torch.Tensor) or self.table.dim() != 2:
            raise ValueError("table must be [rows, max_blocks]")
        _i32(self.table, "table")
        _i32(self.length, "length", (self.table.shape[0],))
        _i32(self.refs, "refs", (self.pool.shape[1],))

    @classmethod
    def empty(cls, layers: int, pages: int, kv_heads: int, page_size: int, head_dim: int, rows: int, max_blocks: int,
              dtype=torch.bfloat16, device="cuda"):
        """A pool without a page in use and tables without a row in use."""
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.zeros((2 * layers, pages, kv_heads, page_size, head_dim), device=device, dtype=dtype),
                   torch.full((rows, max_blocks), -1, **i32), torch.zeros(rows, **i32), torch.zeros(pages, **i32))

    def keys(self, layer: int):
        return self.pool[2 * layer]

    def values(self, layer: int):
        return self.pool[2 * layer + 1]

    def _args(self, n: int):
        p = self.pool
        rows, blocks = self.table.shape
        need = L.lib().cache_workspace_size(rows, p.shape[1], n)
        if self._workspace is None or self._workspace.numel() < need:
            self._workspace = torch.empty(need, dtype=torch.uint8, device=p.device)
        e = p.element_size()
        pstride = p.stride(1) if p.shape[1] > 1 else p[0, 0].numel()
        return L.Cache(p.shape[0], p.shape[1], p.shape[3], rows, blocks, 0, p.stride(0) * e, pstride * e,
                       p[0, 0].numel() * e, _ptr(p), _ptr(self.table), _ptr(self.length), _ptr(self.refs),
                       _ptr(self._workspace), self._workspace.numel())


def _list(t, name, n=None):
    _i32(t, name)
    if t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name}: expected a list of {'int32' if n is None else n} entries")
    return t


def _granted(granted, like):
    return torch.empty_like(like) if granted is None else _list(granted, "granted", like.shape[0])


def cache_extend(cache: PagedCache, rows, count, *, granted=None, stream=None):
    """Rows grow by ``count`` tokens each, taking the pages they need; returns
    ``granted`` (1 where there was room, else 0 and the row as it was)."""
    _list(rows, "rows")
    _list(count, "count", rows.shape[0])
    granted = _granted(granted, rows)
    L.check(L.lib().cache_extend(ct.byref(cache._args(rows.shape[0])), rows.shape[0], _ptr(rows), _ptr(count), _ptr(granted),
                                 _stream(stream)))
    return granted


def cache_fork(cache: PagedCache, src, dst, *, granted=None, stream=None):
    """Empty rows ``dst`` become copies of rows ``src`` (whole pages shared, a
    partly filled last one copied); returns ``granted`` as cache_extend."""
    _list(src, "src")
    _list(dst, "dst", src.shape[0])
    granted = _granted(granted, src)
    L.check(L.lib().cache_fork(ct.byref(cache._args(src.shape[0])), src.shape[0], _ptr(src), _ptr(dst), _ptr(granted),
                               _stream(stream)))
    return granted


def cache_free(cache: PagedCache, rows, *, window: int = 0, sinks: int = 0, stream=None):
    """Rows give their pages back; with ``window`` only those that attention
    with this window and these sinks sees no more."""
    _list(rows, "rows")
    L.check(L.lib().cache_free(ct.byref(cache._args(rows.shape[0])), rows.shape[0], _ptr(rows), int(window), int(sinks),
                               _stream(stream)))


def cache_compact(cache: PagedCache, *, table_out=None, refs_out=None, moved=None, stream=None):
    """Live pages move to the front of the pool; the new tables go to
    ``table_out`` and ``refs_out`` (default: in place), the count of moved
    pages to ``moved`` (int32[1])."""
    table_out = cache.table if table_out is None else _i32(table_out, "table_out", cache.table.shape)
    refs_out = cache.refs if refs_out is None else _i32(refs_out, "refs_out", cache.refs.shape)
    _i32(moved, "moved", (1,), allow_none=True)
    L.check(L.lib().cache_compact(ct.byref(cache._args(0)), _ptr(table_out), _ptr(refs_out), _ptr(moved), _stream(stream)))


def cache_copy(pool, src, dst, *, stream=None):
    """Pages ``src`` to pages ``dst`` in every plane of ``pool`` (as
    PagedCache.pool)."""
    if not isinstance(pool, torch.Tensor) or pool.dim() != 5:
        raise ValueError("pool must be [planes, num_pages, kv_heads, page_size, head_dim]")
    _dense_rows(pool[0], "pool", 4)
    _list(src, "src")
    _list(dst, "dst", src.shape[0])
    e = pool.element_size()
    pstride = pool.stride(1) if pool.shape[1] > 1 else pool[0, 0].numel()
    a = L.Cache(pool.shape[0], pool.shape[1], pool.shape[3], 0, 0, 0, pool.stride(0) * e, pstride * e,
                pool[0, 0].numel() * e, _ptr(pool), None, None, None, None, 0)
    L.check(L.lib().cache_copy(ct.byref(a), src.shape[0], _ptr(src), _ptr(dst), _stream(stream)))


def guided_logits(logits, out, cond_row, uncond_row=None, scale=None, *, history=None, history_len=None, prompt_len=None,
                  repetition=None, presence=None, frequency=None, bias_ids=None, bias=None, temperature=None, mask=None,
                  stream=None):
    """The guided combine of the branches' logits [logit_rows, vocab] (any row
    stride) into out [n, vocab], with penalties of the tokens in ``history``
    [n, max_history], biases [n, num_biases], temperature and a grammar
    ``mask`` (int32 bits, [n, >= ceil(vocab / 32)]); see include/bcg_decode.h."""
    ls, os_ = _dense_rows(logits, "logits", 2), _dense_rows(out, "out", 2)
    if logits.dtype not in _DT or out.dtype not in _DT:
        raise ValueError("logits and out must be float32 or bfloat16")
    n, vocab = out.shape
    if logits.shape[1] != vocab:
        raise ValueError(f"logits of {logits.shape[1]} tokens, out of {vocab}")
    for t, name in ((cond_row, "cond_row"), (uncond_row, "uncond_row"), (history_len, "history_len"), (prompt_len, "prompt_len")):
        _i32(t, name, (n,), allow_none=name != "cond_row")
    for t, name in ((scale, "scale"), (repetition, "repetition"), (presence, "presence"), (frequency, "frequency"),
                    (temperature, "temperature")):
        _f32(t, name, (n,))
    for t, name in ((history, "history"), (bias_ids, "bias_ids"), (mask, "mask")):
        if t is not None and (_i32(t, name).dim() != 2 or t.shape[0] != n):
            raise ValueError(f"{name}: expected {n} rows")
    if bias_ids is not None:
        _f32(bias, "bias", tuple(bias_ids.shape), allow_none=False)
    elif bias is not None:
        raise ValueError("bias without bias_ids")
    a = L.LogitsArgs(n, vocab, logits.shape[0], _DT[logits.dtype], _DT[out.dtype],
                     0 if history is None else history.shape[1], 0 if bias_ids is None else bias_ids.shape[1],
                     0 if mask is None else mask.shape[1], ls, os_, _ptr(logits), _ptr(out), _ptr(cond_row),
                     _ptr(uncond_row), _ptr(scale), _ptr(history), _ptr(history_len), _ptr(prompt_len), _ptr(repetition),
                     _ptr(presence), _ptr(frequency), _ptr(bias_ids), _ptr(bias), _ptr(temperature), _ptr(mask))
    L.check(L.lib().guided_logits(ct.byref(a), _stream(stream)))
