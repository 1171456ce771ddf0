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
from .api import _DT, _dev

_KV = {torch.float32: L.BCG_F32, torch.bfloat16: L.BCG_BF16, torch.float8_e4m3fn: L.BCG_E4M3}
_E4M3 = torch.float8_e4m3fn
_I32, _F32 = torch.int32, torch.float32
_raw_stream = torch._C._cuda_getCurrentRawStream

# One step of a decoding loop makes a handful of these calls for every layer,
# and the smallest of them run for a few microseconds, so the checks are kept
# short: one expression for a tensor that is as it should be (its address comes
# back), and the reason only where it is not.


def _need(t, name, dtype, shape=None):
    """The address of a contiguous GPU tensor of this dtype (and shape)."""
    try:
        if t.is_cuda and t.dtype is dtype and t.is_contiguous() and (shape is None or t.shape == shape):
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, name, dtype, shape)
    raise ValueError(f"{name}: not usable")


def _opt(t, name, dtype, shape=None):
    return None if t is None else _need(t, name, dtype, shape)


def _dense_rows(t, name, dims):
    """A GPU tensor whose dimensions after the first are contiguous: (its
    shape, the elements between its rows, its address)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor (got {t.device})")
    shape, strides = t.shape, t.stride()
    if len(shape) != dims:
        raise ValueError(f"{name}: expected {dims} dimensions, got {len(shape)}")
    width = 1
    for d in range(dims - 1, 0, -1):
        if strides[d] != width and shape[d] != 1:
            raise ValueError(f"{name}: must be contiguous after its first dimension")
        width *= shape[d]
    return shape, strides[0] if shape[0] > 1 or strides[0] > width else width, t.data_ptr()


def _run(fn, args, t, stream):
    # t: a tensor of the call, for the device whose current stream it goes to
    rc = fn(args, _raw_stream(t.get_device()) if stream is None else stream.cuda_stream)
    if rc:
        L.check(rc)


def _cache_args(k_cache, v_cache, dtype, block_table, kv_len, k_scale, v_scale):
    """One layer's pages: (kv_heads, page_size, dim, num_pages, k page stride,
    v page stride, cache type, rows, max_blocks, addresses)."""
    shape, ks, kp = _dense_rows(k_cache, "k_cache", 4)
    vshape, vs, vp = _dense_rows(v_cache, "v_cache", 4)
    kt = k_cache.dtype
    if shape != vshape or v_cache.dtype is not kt:
        raise ValueError("k_cache and v_cache must have the same shape and dtype")
    if kt is not dtype and not (kt is _E4M3 and dtype is torch.bfloat16):
        raise ValueError(f"a cache of {kt} does not go with {dtype}")
    pages, kvh, page, dim = shape
    tp = _need(block_table, "block_table", _I32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [rows, max_blocks]")
    rows, blocks = block_table.shape
    return (kvh, page, dim, pages, ks, vs, _KV[kt], rows, blocks, kp, vp, tp, _need(kv_len, "kv_len", _I32, (rows,)),
            _opt(k_scale, "k_scale", _F32, (kvh,)), _opt(v_scale, "v_scale", _F32, (kvh,)))


def attention_workspace(tokens: int, q_heads: int, head_dim: int, device=None):
    """A workspace for the attention calls of up to ``tokens`` query rows
    (keep it from call to call; one for each stream)."""
    n = L.lib().attention_workspace_size(int(tokens), int(q_heads), int(head_dim))
    return torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda", torch.cuda.current_device()))


def _attention(prompt, q, q_offset, k_cache, v_cache, block_table, kv_len, out, *, workspace, scale, window, sinks,
               k_scale, v_scale, max_len, max_new, lse, stream):
    shape, q_stride, qp = _dense_rows(q, "q", 3)
    qt = _DT.get(q.dtype)
    if qt is None:
        raise ValueError("q must be float32 or bfloat16")
    tokens, heads, dim = shape
    kvh, page, cdim, pages, ks, vs, kvt, rows, blocks, kp, vp, tp, np_, ksp, vsp = _cache_args(
        k_cache, v_cache, q.dtype, block_table, kv_len, k_scale, v_scale)
    if cdim != dim:
        raise ValueError(f"head_dim {dim} of q, {cdim} of the cache")
    if prompt:
        op = _need(q_offset, "q_offset", _I32, (rows + 1,))
    elif rows != tokens:
        raise ValueError(f"{tokens} query rows for {rows} rows of the table")
    else:
        op = None
    a = L.AttnArgs(rows, tokens, heads, kvh, dim, page, blocks, pages, qt, kvt,
                   blocks * page if max_len is None else max_len, tokens if max_new is None else max_new, window, sinks,
                   dim ** -0.5 if scale is None else scale, 0, q_stride, ks, vs, qp, kp, vp, tp, np_, op, ksp, vsp,
                   _need(out, "out", q.dtype, shape), _opt(lse, "lse", _F32, (tokens, heads)),
                   _need(workspace, "workspace", torch.uint8), workspace.numel())
    lib = L.lib()
    _run(lib.prompt_attention if prompt else lib.paged_attention, ct.byref(a), q, stream)


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
    shape, ks, kp = _dense_rows(k, "k", 3)
    vshape, vs, vp = _dense_rows(v, "v", 3)
    t = _DT.get(k.dtype)
    if t is None or v.dtype is not k.dtype or shape != vshape:
        raise ValueError("k and v must have the same shape, float32 or bfloat16")
    kvh, page, dim, pages, kps, vps, kvt, rows, blocks, kcp, vcp, tp, np_, ksp, vsp = _cache_args(
        k_cache, v_cache, k.dtype, block_table, kv_len, k_scale, v_scale)
    tokens = shape[0]
    if shape[1] != kvh or shape[2] != dim:
        raise ValueError(f"k and v must be [tokens, {kvh}, {dim}]")
    if offset is None and rows != tokens:
        raise ValueError(f"{tokens} tokens for {rows} rows of the table")
    a = L.AppendArgs(rows, tokens, kvh, dim, page, blocks, pages, t, kvt, 0, ks, vs, kps, vps, kp, vp,
                     _opt(offset, "offset", _I32, (rows + 1,)), tp, np_, ksp, vsp, kcp, vcp)
    _run(L.lib().cache_append, ct.byref(a), k, stream)


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
        self._pool_args()
        if not isinstance(self.table, torch.Tensor) or self.table.dim() != 2:
            raise ValueError("table must be [rows, max_blocks]")
        self._tables()

    def _pool_args(self):
        return _pool(self.pool)

    def _tables(self):
        rows, blocks = self.table.shape
        return (rows, blocks, _need(self.table, "table", _I32), _need(self.length, "length", _I32, (rows,)),
                _need(self.refs, "refs", _I32, (self.pool.shape[1],)))

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
        planes, pages, page, pstride, stride, size, pp = self._pool_args()
        rows, blocks, tp, lp, rp = self._tables()
        ws = self._workspace
        if ws is None or ws.numel() < 4 * (rows + 3 * pages + 3 * n + 16):  # an upper bound of what is needed
            need = L.lib().cache_workspace_size(rows, pages, n)
            if ws is None or ws.numel() < need:
                ws = self._workspace = torch.empty(need + 4096, dtype=torch.uint8, device=self.pool.device)
        return ct.byref(L.Cache(planes, pages, page, rows, blocks, 0, pstride, stride, size, pp, tp, lp, rp, ws.data_ptr(),
                                ws.numel()))


def _pool(pool):
    """(planes, pages, page_size, bytes between planes, between pages, of a page, address)."""
    if not isinstance(pool, torch.Tensor) or pool.dim() != 5:
        raise ValueError("pool must be [planes, num_pages, kv_heads, page_size, head_dim]")
    if not pool.is_cuda:
        raise ValueError(f"pool: must be a GPU tensor (got {pool.device})")
    planes, pages, heads, page, dim = pool.shape
    s = pool.stride()
    width = heads * page * dim
    if (s[4] != 1 and dim != 1) or (s[3] != dim and page != 1) or (s[2] != page * dim and heads != 1):
        raise ValueError("pool: a page must be contiguous")
    e = pool.element_size()
    return planes, pages, page, s[0] * e, (s[1] if pages > 1 else width) * e, width * e, pool.data_ptr()


def _list(t, name, n=None):
    p = _need(t, name, _I32)
    if t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name}: expected a list of {'int32' if n is None else n} entries")
    return p


def cache_extend(cache: PagedCache, rows, count, *, granted=None, stream=None):
    """Rows grow by ``count`` tokens each, taking the pages they need; returns
    ``granted`` (1 where there was room, else 0 and the row as it was)."""
    rp = _list(rows, "rows")
    n = rows.shape[0]
    granted = torch.empty_like(rows) if granted is None else granted
    _run_list(L.lib().cache_extend, cache, n, rp, _list(count, "count", n), _list(granted, "granted", n), stream=stream)
    return granted


def _run_list(fn, cache, n, *more, stream):
    rc = fn(cache._args(n), n, *more, _raw_stream(cache.pool.get_device()) if stream is None else stream.cuda_stream)
    if rc:
        L.check(rc)


def cache_fork(cache: PagedCache, src, dst, *, granted=None, stream=None):
    """Empty rows ``dst`` become copies of rows ``src`` (whole pages shared, a
    partly filled last one copied); returns ``granted`` as cache_extend."""
    sp = _list(src, "src")
    n = src.shape[0]
    granted = torch.empty_like(src) if granted is None else granted
    _run_list(L.lib().cache_fork, cache, n, sp, _list(dst, "dst", n), _list(granted, "granted", n), stream=stream)
    return granted


def cache_free(cache: PagedCache, rows, *, window: int = 0, sinks: int = 0, stream=None):
    """Rows give their pages back; with ``window`` only those that attention
    with this window and these sinks sees no more."""
    rp = _list(rows, "rows")
    _run_list(L.lib().cache_free, cache, rows.shape[0], rp, window, sinks, stream=stream)


def cache_compact(cache: PagedCache, *, table_out=None, refs_out=None, moved=None, stream=None):
    """Live pages move to the front of the pool; the new tables go to
    ``table_out`` and ``refs_out`` (default: in place), the count of moved
    pages to ``moved`` (int32[1])."""
    tp = _need(cache.table if table_out is None else table_out, "table_out", _I32, cache.table.shape)
    rp = _need(cache.refs if refs_out is None else refs_out, "refs_out", _I32, cache.refs.shape)
    mp = _opt(moved, "moved", _I32, (1,))
    rc = L.lib().cache_compact(cache._args(0), tp, rp, mp, _raw_stream(cache.pool.get_device()) if stream is None
                               else stream.cuda_stream)
    if rc:
        L.check(rc)


def cache_copy(pool, src, dst, *, stream=None):
    """Pages ``src`` to pages ``dst`` in every plane of ``pool`` (as
    PagedCache.pool)."""
    planes, pages, page, pstride, stride, size, pp = _pool(pool)
    sp = _list(src, "src")
    n = src.shape[0]
    a = L.Cache(planes, pages, page, 0, 0, 0, pstride, stride, size, pp, None, None, None, None, 0)
    rc = L.lib().cache_copy(ct.byref(a), n, sp, _list(dst, "dst", n), _raw_stream(pool.get_device()) if stream is None
                            else stream.cuda_stream)
    if rc:
        L.check(rc)


def guided_logits(logits, out, cond_row, uncond_row=None, scale=None, *, history=None, history_len=None, prompt_len=None,
                  repetition=None, presence=None, frequency=None, bias_ids=None, bias=None, temperature=None, mask=None,
                  stream=None):
    """The guided combine of the branches' logits [logit_rows, vocab] (any row
    stride) into out [n, vocab], with penalties of the tokens in ``history``
    [n, max_history], biases [n, num_biases], temperature and a grammar
    ``mask`` (int32 bits, [n, >= ceil(vocab / 32)]); see include/bcg_decode.h."""
    lshape, ls, lp = _dense_rows(logits, "logits", 2)
    oshape, os_, op = _dense_rows(out, "out", 2)
    lt, ot = _DT.get(logits.dtype), _DT.get(out.dtype)
    if lt is None or ot is None:
        raise ValueError("logits and out must be float32 or bfloat16")
    n, vocab = oshape
    if lshape[1] != vocab:
        raise ValueError(f"logits of {lshape[1]} tokens, out of {vocab}")
    hp, hn = _rows_of(history, "history", n)
    ip, biases = _rows_of(bias_ids, "bias_ids", n)
    mp, words = _rows_of(mask, "mask", n)
    if bias_ids is None and bias is not None:
        raise ValueError("bias without bias_ids")
    if bias_ids is not None and bias is None:
        raise ValueError("bias_ids without bias")
    one = (n,)
    a = L.LogitsArgs(n, vocab, lshape[0], lt, ot, hn, biases, words, ls, os_, lp, op, _need(cond_row, "cond_row", _I32, one),
                     _opt(uncond_row, "uncond_row", _I32, one), _opt(scale, "scale", _F32, one), hp,
                     _opt(history_len, "history_len", _I32, one), _opt(prompt_len, "prompt_len", _I32, one),
                     _opt(repetition, "repetition", _F32, one), _opt(presence, "presence", _F32, one),
                     _opt(frequency, "frequency", _F32, one), ip, _opt(bias, "bias", _F32, (n, biases)),
                     _opt(temperature, "temperature", _F32, one), mp)
    _run(L.lib().guided_logits, ct.byref(a), logits, stream)


def _rows_of(t, name, n):
    """(address, width) of an int32 [n, width] tensor; (None, 0) for None."""
    if t is None:
        return None, 0
    p = _need(t, name, _I32)
    if t.dim() != 2 or t.shape[0] != n:
        raise ValueError(f"{name}: expected {n} rows")
    return p, t.shape[1]
