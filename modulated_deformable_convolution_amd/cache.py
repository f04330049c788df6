"""Python binding of libmdcn.so's operators on key/value caches in 4 bits and on the
pages they lie in (include/mdcn.h): new keys and values rounded into their pages, read
back, attended to; sequences forked and freed, pools compacted, pages copied.

A pool is a uint8 tensor [pages, page bytes] (page operators also take several layers
that share a table, [layers, pages, page bytes]), a table int32 [rows, width] with the
pages of each sequence, -1 where there is none, used int32 [rows] the tokens that each
holds, owners int32 [pages] how many entries (and other holds) name a page.  One
step of decoding is

    table, used, owners, missing = fork_pages(pool, table, used, owners, page, None, ones)
    store(cache, pool, k, v, table, used, ends)
    out, lse = attend(attention, cache, q, pool, table, used, ends)

As in attention.py, outputs and workspaces are allocated with torch, calls enqueue work on the
current device, which must be the tensors', on the caller's stream, and return; they raise
MdcnError on bad arguments.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import attention as _a
from . import mdcn as _m
from .attention import (_NO_CONTEXT, _check_current, _check_ints, _check_lse, _check_view,
                        _device_tensors, _fail, _like, _new, _remember, _sig, _stream_of, _strides,
                        _workspace_bytes)
from .mdcn import MDCN_E_ATTR

_i64 = ctypes.c_int64
_page_calls = {}                 # shapes, strides, ... -> what a page operator's checks return


class Cache:
    """Owns an mdcn_cache handle; page_bytes are those of one page."""

    def __init__(self, handle: int, k_heads: int, dim: int, page: int):
        self.handle = handle
        self.k_heads, self.dim, self.page = k_heads, dim, page
        n = _i64()
        _m._check(_m._lib.mdcn_cache_page_bytes(handle, ctypes.byref(n)), "mdcn_cache_page_bytes")
        self.page_bytes = n.value
        self.calls = {}          # shapes, strides, ... -> what _cache_dims returns

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _m is not None and _m._lib is not None:
            _m._lib.mdcn_cache_destroy(h)


def mdcn_cache_create(k_heads: int, dim: int, page: int) -> Cache:
    """Caches of k_heads key and value heads of dim channels in pages of `page` tokens."""
    h = ctypes.c_void_p()
    _m._check(_m.library().mdcn_cache_create(int(k_heads), int(dim), int(page), ctypes.byref(h)),
              "mdcn_cache_create")
    return Cache(h.value, int(k_heads), int(dim), int(page))


# ---------------------------------------------------------------- checks
#
# What a call's checks depend on is its key: shapes, strides, types and devices.  A key that
# passed them before needs only the current device looked at.

def _check_bytes(where, name, pool, like, dims):
    if pool.dtype != torch.uint8 or pool.device != like.device or pool.dim() not in dims:
        _fail(where, "%s must be uint8 [pages, page bytes] on the tensors' device" % name)
    if pool.shape[-1] > 1 and pool.stride(-1) != 1:
        _fail(where, "the bytes of a page of %s must lie together" % name)


def _row_stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _check_table(where, table, like):
    if table.dtype != torch.int32 or table.device != like.device or table.dim() != 2:
        _fail(where, "table must be int32 [rows, width] on the tensors' device")
    if table.shape[1] > 1 and table.stride(1) != 1:
        _fail(where, "the entries of a row of the table must lie together")


def _cache_dims(op, where, pool, table, used, cu, like, tokens, views):
    """(dtype code, ctypes dims) of a call on `tokens` tokens and [tokens, heads, dim] views."""
    _check_bytes(where, "pool", pool, like, (2,))
    if pool.shape[1] != op.page_bytes:
        _fail(where, "a page of pool must hold %d bytes" % op.page_bytes)
    _check_table(where, table, like)
    batch = table.shape[0]
    _check_ints(where, "used", used, like, (batch,))
    _check_ints(where, "cu", cu, like, (batch + 1,))
    vals = [batch, tokens, pool.shape[0], pool.stride(0) if pool.shape[0] > 1 else op.page_bytes,
            table.shape[1], _row_stride(table)]
    for name, t, heads in views:
        if t.dim() != 3:
            _fail(where, "%s must be [tokens, heads, dim]" % name)
        _check_view(where, name, t, like, (tokens, heads, op.dim))
        vals += _strides(t)
    return _m.dtype_code(like.dtype), (_i64 * len(vals))(*vals)


# ---------------------------------------------------------------- keys and values

def store(op: Cache, pool, k, v, table, used, cu, stream=None):
    """Rounds the new keys and values of packed sequences (k, v [tokens, k_heads, dim], cu
    int32 [rows + 1]) into their pages: sequence b's become its last tokens, up to
    used[b] - 1."""
    where = "store"
    key = (_sig(pool), _sig(k), _sig(v), _sig(table), _sig(used), _sig(cu))
    call = op.calls.get(key)
    if call is not None:
        _check_current(where, k.get_device())
    else:
        _device_tensors(where, k, v, pool, table, used, cu)
        call = _remember(op.calls, key, _cache_dims(
            op, where, pool, table, used, cu, k, k.shape[0],
            (("k", k, op.k_heads), ("v", v, op.k_heads))))
    stream, _ = _stream_of(stream, k)
    st = _m._lib.mdcn_cache_store(op.handle, call[0], call[1], k.data_ptr(), v.data_ptr(),
                                  table.data_ptr(), used.data_ptr(), cu.data_ptr(), pool.data_ptr(),
                                  stream)
    if st:
        _m._check(st, where)


def load(op: Cache, pool, table, used, cu, tokens: int, dtype, k=None, v=None, stream=None):
    """The last cu[b + 1] - cu[b] tokens of each sequence as the values that the cache holds for
    them: (k, v), [tokens, k_heads, dim].  Tokens without a page are zeros, and so are those of
    no sequence, but in a k or v that the caller gives they are left as they are."""
    where = "load"
    key = (_sig(pool), _sig(table), _sig(used), _sig(cu), tokens, dtype,
           None if k is None else _sig(k), None if v is None else _sig(v))
    call = op.calls.get(key)
    if call is not None:
        _check_current(where, pool.get_device())
    else:
        _device_tensors(where, pool, table, used, cu)
    stream, ctx = _stream_of(stream, pool)
    with ctx or _NO_CONTEXT:
        if call is None:
            like = _like((tokens, op.k_heads, op.dim), dtype, pool.device)
            views = [_new(like) if t is None else t for t in (k, v)]
            _device_tensors(where, *views)
            if views[0].dtype != dtype:
                _fail(where, "k must be of the dtype asked for")
            call = _remember(op.calls, key, _cache_dims(
                op, where, pool, table, used, cu, views[0], tokens,
                (("k", views[0], op.k_heads), ("v", views[1], op.k_heads))) + (like,))
        fill = (1 if k is None else 0) | (2 if v is None else 0)
        if k is None:
            k = _new(call[2])
        if v is None:
            v = _new(call[2])
    st = _m._lib.mdcn_cache_load(op.handle, call[0], call[1], pool.data_ptr(), table.data_ptr(),
                                 used.data_ptr(), cu.data_ptr(), fill, k.data_ptr(), v.data_ptr(),
                                 stream)
    if st:
        _m._check(st, where)
    return k, v


def attend(att: _a.Attention, op: Cache, q, pool, table, used, cu_q, out=None, lse=None,
           workspace=None, stream=None):
    """attention.attend against the cache: the queries of sequence b (q [q_tokens, q_heads, dim],
    cu_q int32 [rows + 1]) attend to its used[b] tokens.  Returns (out, lse)."""
    where = "attend"
    lib = _m._lib
    key = (att.q_heads, att.k_heads, att.dim, _sig(q), None if out is None else _sig(out),
           _sig(pool), _sig(table), _sig(used), _sig(cu_q))
    call = op.calls.get(key)
    if call is not None:
        _check_current(where, q.get_device())
    else:
        _device_tensors(where, q, pool, table, used, cu_q)
    stream, ctx = _stream_of(stream, q)
    fill = (1 if out is None else 0) | (2 if lse is None else 0)
    with ctx or _NO_CONTEXT:
        if out is None:
            out = torch.empty_like(q)
        if call is None:
            if att.k_heads != op.k_heads or att.dim != op.dim:
                _fail(where, "attention and cache must agree in key heads and dim", MDCN_E_ATTR)
            dims = _cache_dims(op, where, pool, table, used, cu_q, q, q.shape[0],
                               (("q", q, att.q_heads), ("out", out, att.q_heads)))
            n = ctypes.c_size_t()
            _m._check(lib.mdcn_cache_attend_workspace_bytes(att.handle, op.handle, dims[0], dims[1],
                                                            ctypes.byref(n)), where)
            call = _remember(op.calls, key, dims + (
                _like((n.value,), torch.uint8, q.device) if n.value else None,
                _like((att.q_heads, q.shape[0]), torch.float32, q.device)))
        if lse is None:
            lse = _new(call[3])
        else:
            _check_lse(where, att, q, lse)
        if workspace is None and call[2] is not None:
            workspace = _new(call[2])
    st = lib.mdcn_cache_attend(
        att.handle, op.handle, call[0], call[1], q.data_ptr(), pool.data_ptr(), table.data_ptr(),
        used.data_ptr(), cu_q.data_ptr(), fill, out.data_ptr(), lse.data_ptr(),
        None if workspace is None else workspace.data_ptr(), _workspace_bytes(where, workspace, q),
        stream)
    if st:
        _m._check(st, where)
    return out, lse


def describe_attend(att: _a.Attention, op: Cache, dtype, batch: int, q_tokens: int, width: int) -> str:
    """One line on attend's kernels for these sizes (mdcn_describe_cache_attend)."""
    buf = ctypes.create_string_buffer(256)
    dims = (_i64 * 10)(batch, q_tokens, 1, op.page_bytes, width, width, 0, 0, 0, 0)
    _m._check(_m._lib.mdcn_describe_cache_attend(att.handle, op.handle, _m.dtype_code(dtype), dims, buf,
                                                 256), "describe_attend")
    return buf.value.decode()


# ---------------------------------------------------------------- pages

def _pool_dims(where, name, pool, like):
    """layers, pages, page bytes, page stride, layer stride"""
    _check_bytes(where, name, pool, like, (2, 3))
    pages, size = pool.shape[-2:]
    layers = pool.shape[0] if pool.dim() == 3 else 1
    page_stride = pool.stride(-2) if pages > 1 else size
    return [layers, pages, size, page_stride,
            pool.stride(0) if layers > 1 else max(1, pages) * page_stride]


def _contiguous_ints(where, name, t, like, shape):
    _check_ints(where, name, t, like, shape)
    if not t.is_contiguous():
        _fail(where, "%s must be contiguous" % name)


class _Results:
    """The results of a page operator and its workspace.  Where the caller gives none of them they
    are parts of one allocation (2 us a call less than five)."""

    def __init__(self, where, function, dims, like, names, shapes):
        n = ctypes.c_size_t()
        _m._check(function(dims, ctypes.byref(n)), where)
        self.where, self.names, self.shapes = where, names, shapes
        self.sizes = [-(-math.prod(s) // 4) * 4 for s in shapes] + [-(-n.value // 4)]
        self.all = _like((sum(self.sizes),), torch.int32, like.device)
        self.exact = [size == math.prod(s) and len(s) == 1 for size, s in zip(self.sizes, shapes)]

    def make(self, given, workspace, like):
        """(the results, the workspace)"""
        parts = None
        if workspace is None or any(t is None for t in given):
            parts = _new(self.all).split_with_sizes(self.sizes)
        results = []
        for i, t in enumerate(given):
            shape = self.shapes[i]
            if t is not None:
                _contiguous_ints(self.where, self.names[i], t, like, shape)
            elif self.exact[i]:
                t = parts[i]
            else:
                t = parts[i].as_strided(shape, (shape[-1], 1)[-len(shape):])
            results.append(t)
        return results, parts[-1] if workspace is None else workspace


def fork_pages(pool, table, used, owners, page: int, parents=None, new_tokens=None, table_out=None,
               used_out=None, owners_out=None, missing=None, workspace=None, stream=None):
    """New sequences from old ones: row i goes on from row parents[i] (None: from row i; outside
    the table: empty) with room for new_tokens[i] more (None: none).  Full pages are shared, pages
    full in part copied for all children but the first, rows that nobody goes on from give theirs
    up.  Returns (table, used, owners, missing): missing int32 [1] is 0, or how many pages there
    are too few, and then nothing was copied and the old table still holds.  Results that are not
    given are parts of one allocation: clone one that is to be saved or kept by itself."""
    where = "fork_pages"
    lib = _m._lib or _m.library()
    key = (where, None if pool is None else _sig(pool), _sig(table), _sig(used), _sig(owners), page,
           None if parents is None else _sig(parents),
           None if new_tokens is None else _sig(new_tokens))
    call = _page_calls.get(key)
    if call is not None:
        _check_current(where, table.get_device())
    else:
        _device_tensors(where, table, used, owners,
                        *(t for t in (pool, parents, new_tokens) if t is not None))
        if table.dim() != 2 or owners.dim() != 1:
            _fail(where, "table must be [rows, width], owners [pages]")
        rows, width = table.shape
        _contiguous_ints(where, "table", table, table, (rows, width))
        _contiguous_ints(where, "used", used, table, (rows,))
        _contiguous_ints(where, "owners", owners, table, (owners.shape[0],))
        dims = [0, owners.shape[0], 0, 0, 0] if pool is None else _pool_dims(where, "pool", pool, table)
        if dims[1] != owners.shape[0]:
            _fail(where, "owners must have an entry for each page")
        given = parents if parents is not None else new_tokens
        out_rows = rows if given is None else given.shape[0] if given.dim() == 1 else -1
        for name, t in (("parents", parents), ("new_tokens", new_tokens)):
            if t is not None:
                _contiguous_ints(where, name, t, table, (out_rows,))
        dims = (_i64 * 9)(*dims, page, rows, out_rows, width)
        call = _remember(_page_calls, key, (
            dims, _Results(where, lib.mdcn_pages_fork_workspace_bytes, dims, table,
                           ("table_out", "used_out", "owners_out", "missing"),
                           ((out_rows, width), (out_rows,), tuple(owners.shape), (1,)))))
    stream, ctx = _stream_of(stream, table)
    with ctx or _NO_CONTEXT:
        results, workspace = call[1].make((table_out, used_out, owners_out, missing), workspace, table)
    st = lib.mdcn_pages_fork(
        call[0], None if pool is None else pool.data_ptr(), table.data_ptr(), used.data_ptr(),
        owners.data_ptr(), None if parents is None else parents.data_ptr(),
        None if new_tokens is None else new_tokens.data_ptr(), *(t.data_ptr() for t in results),
        workspace.data_ptr(), _workspace_bytes(where, workspace, table), stream)
    if st:
        _m._check(st, where)
    return tuple(results)


def compact_pages(pool, table, owners, table_out=None, owners_out=None, moved=None, workspace=None,
                  stream=None):
    """Moves the n held pages to the numbers 0 .. n - 1.  Returns (table, owners, moved) with
    the new numbers, parts of one allocation as fork_pages' are; moved int32 [pages]: the new
    number of each page, -1 if it is free."""
    where = "compact_pages"
    lib = _m._lib or _m.library()
    key = (where, _sig(pool), _sig(table), _sig(owners))
    call = _page_calls.get(key)
    if call is not None:
        _check_current(where, table.get_device())
    else:
        _device_tensors(where, pool, table, owners)
        if table.dim() != 2:
            _fail(where, "table must be [rows, width]")
        _contiguous_ints(where, "table", table, table, tuple(table.shape))
        dims = _pool_dims(where, "pool", pool, table)
        _contiguous_ints(where, "owners", owners, table, (dims[1],))
        dims = (_i64 * 7)(*dims, *table.shape)
        call = _remember(_page_calls, key, (
            dims, _Results(where, lib.mdcn_pages_compact_workspace_bytes, dims, table,
                           ("table_out", "owners_out", "moved"),
                           (tuple(table.shape), tuple(owners.shape), tuple(owners.shape)))))
    stream, ctx = _stream_of(stream, table)
    with ctx or _NO_CONTEXT:
        results, workspace = call[1].make((table_out, owners_out, moved), workspace, table)
    st = lib.mdcn_pages_compact(
        call[0], pool.data_ptr(), table.data_ptr(), owners.data_ptr(),
        *(t.data_ptr() for t in results), workspace.data_ptr(),
        _workspace_bytes(where, workspace, table), stream)
    if st:
        _m._check(st, where)
    return tuple(results)


def copy_pages(src_pool, dst_pool, src, dst, stream=None):
    """Copies page src[i] of one pool to page dst[i] of another, or of the same one, in every
    layer.  Pairs with a number outside its pool are passed over."""
    where = "copy_pages"
    key = (where, _sig(src_pool), _sig(dst_pool), _sig(src), _sig(dst))
    call = _page_calls.get(key)
    if call is not None:
        _check_current(where, src.get_device())
    else:
        _device_tensors(where, src_pool, dst_pool, src, dst)
        if src.dim() != 1:
            _fail(where, "src and dst must be lists of pages")
        _contiguous_ints(where, "src", src, src, tuple(src.shape))
        _contiguous_ints(where, "dst", dst, src, tuple(src.shape))
        a = _pool_dims(where, "src_pool", src_pool, src)
        b = _pool_dims(where, "dst_pool", dst_pool, src)
        if a[0] != b[0] or a[2] != b[2]:
            _fail(where, "the pools must agree in layers and page bytes")
        call = _remember(_page_calls, key, (_i64 * 9)(a[0], src.shape[0], a[2], a[1], a[3], a[4], b[1],
                                                      b[3], b[4]))
    stream, _ = _stream_of(stream, src)
    st = (_m._lib or _m.library()).mdcn_pages_copy(call, src_pool.data_ptr(), dst_pool.data_ptr(),
                                                   src.data_ptr(), dst.data_ptr(), stream)
    if st:
        _m._check(st, where)
