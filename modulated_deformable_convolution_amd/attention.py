"""Python binding of libmdcn.so's attention operators (include/mdcn.h): rotary
positions with several axes, norms of queries and keys with the rotation in
the same pass, attention over packed sequences and key/value caches, and their
backward passes.

Tensors are [tokens, heads, dim] views of device memory with the channels of a
head together (slices of a projection's output are taken as they are), one
dtype per call.  Outputs and workspaces are allocated with torch, on the stream
the call runs on; every step of the computation runs in the library's HIP
kernels.  Calls enqueue work and return; they raise MdcnError on bad arguments.
"""
from __future__ import annotations

import ctypes

from . import mdcn as _m
from .mdcn import MDCN_E_ATTR, MDCN_E_NULL, MDCN_E_SHAPE, MdcnError

_i64 = ctypes.c_int64
_CACHED_CALLS = 64


class Rotary:
    """Owns an mdcn_rotary handle."""

    def __init__(self, handle: int, dim: int, axes: tuple):
        self.handle, self.dim, self.axes = handle, dim, axes
        self.calls = {}          # (shapes, strides) -> ctypes dims, as mdcn.Op's

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _m is not None and _m._lib is not None:
            _m._lib.mdcn_rotary_destroy(h)


class Attention:
    """Owns an mdcn_attention handle."""

    def __init__(self, handle: int, q_heads: int, k_heads: int, dim: int, causal: bool,
                 scale: float):
        self.handle = handle
        self.q_heads, self.k_heads, self.dim = q_heads, k_heads, dim
        self.causal, self.scale = causal, scale
        self.calls = {}          # (shapes, strides) -> (ctypes dims, workspace bytes)

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _m is not None and _m._lib is not None:
            _m._lib.mdcn_attention_destroy(h)


def mdcn_rotary_create(dim: int, axes, base: float = 10000.0, adjacent: bool = False,
                       round_robin: bool = False, per_axis: bool = False) -> Rotary:
    """axes: the number of channel pairs that each axis turns."""
    lib = _m.library()
    axes = tuple(int(v) for v in axes)
    h = ctypes.c_void_p()
    _m._check(lib.mdcn_rotary_create(int(dim), len(axes), (ctypes.c_int32 * max(1, len(axes)))(*axes),
                                     float(base), int(bool(adjacent)), int(bool(round_robin)),
                                     int(bool(per_axis)), ctypes.byref(h)), "mdcn_rotary_create")
    return Rotary(h.value, int(dim), axes)


def mdcn_attention_create(q_heads: int, k_heads: int, dim: int, causal: bool,
                          scale: float | None = None) -> Attention:
    """scale: of the scores, dim ** -0.5 by default."""
    lib = _m.library()
    if scale is None:
        if int(dim) < 1:
            raise MdcnError(MDCN_E_ATTR, "mdcn_attention_create")
        scale = int(dim) ** -0.5
    h = ctypes.c_void_p()
    _m._check(lib.mdcn_attention_create(int(q_heads), int(k_heads), int(dim), int(bool(causal)),
                                        float(scale), ctypes.byref(h)), "mdcn_attention_create")
    return Attention(h.value, int(q_heads), int(k_heads), int(dim), bool(causal), float(scale))


# ---------------------------------------------------------------- checks

def _fail(where, what, status=MDCN_E_SHAPE):
    raise MdcnError(status, "%s: %s" % (where, what))


def _check_view(where, name, t, like, shape):
    if not t.is_cuda:
        _fail(where, name + " must be a device tensor", MDCN_E_NULL)
    if t.dtype != like.dtype or t.device != like.device:
        _fail(where, "tensors must share one dtype and device")
    if tuple(t.shape) != shape:
        _fail(where, "%s must be of shape %s" % (name, shape))
    if shape[2] > 1 and t.stride(2) != 1:
        _fail(where, "the channels of a head of %s must lie together" % name)


def _device_tensors(where, *tensors):
    for t in tensors:
        if not t.is_cuda:
            _fail(where, "tensors must be device tensors", MDCN_E_NULL)


def _check_ints(where, name, t, like, shape):
    import torch
    if t.dtype != torch.int32 or t.device != like.device or tuple(t.shape) != shape:
        _fail(where, "%s must be int32 of shape %s on the tensors' device" % (name, shape))
    if shape[-1] > 1 and t.stride(-1) != 1:
        _fail(where, "%s must be contiguous" % name)


def _strides(t):
    # a dimension of one element is never stepped over; whatever stride torch
    # gives it must not be refused
    n, h, d = t.shape
    return (t.stride(0) if n > 1 else h * d, t.stride(1) if h > 1 else d)


def _remember(calls, key, value):
    if len(calls) >= _CACHED_CALLS:
        calls.clear()
    calls[key] = value
    return value


def _rotary_dims(op, where, q, k, positions, more):
    """ctypes dims of a call on q, k and further views, checked once per
    combination of shapes and strides."""
    key = (q.dtype, q.shape, q.stride(), k.shape, k.stride(), positions.dtype, positions.shape,
           positions.stride(), q.device, k.device, k.dtype, positions.device,
           tuple((t.dtype, t.device, t.shape, t.stride()) for _, t, _ in more))
    dims = op.calls.get(key)
    if dims is None:
        if q.dim() != 3 or k.dim() != 3:
            _fail(where, "q and k must be [tokens, heads, dim]")
        t = q.shape[0]
        _check_view(where, "q", q, q, (t, q.shape[1], op.dim))
        _check_view(where, "k", k, q, (t, k.shape[1], op.dim))
        _check_ints(where, "positions", positions, q, (len(op.axes), t))
        vals = [t, q.shape[1], k.shape[1], positions.stride(0) if len(op.axes) > 1 else t]
        vals += _strides(q) + _strides(k)
        for name, view, like in more:
            _check_view(where, name, view, q, tuple(like.shape))
            vals += _strides(view)
        dims = _remember(op.calls, key, (_i64 * len(vals))(*vals))
    return dims


def _check_gain(where, op, q, *gains):
    for g in gains:
        if g.dtype != q.dtype or g.device != q.device or tuple(g.shape) != (op.dim,) or \
                (op.dim > 1 and g.stride(0) != 1):
            _fail(where, "gains must hold dim values of the tensors' dtype and device")


# ---------------------------------------------------------------- rotary positions

def _rotate(op, q, k, positions, inverse, q_out, k_out, stream, where):
    import torch
    _device_tensors(where, q, k, positions)
    stream, ctx = _m._alloc_stream(stream, q.device, q_out is None or k_out is None)
    with ctx:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        dims = _rotary_dims(op, where, q, k, positions, (("q_out", q_out, q), ("k_out", k_out, k)))
        _m._check(_m._lib.mdcn_rotate(op.handle, _m.dtype_code(q.dtype), dims, q.data_ptr(),
                                      k.data_ptr(), positions.data_ptr(), inverse,
                                      q_out.data_ptr(), k_out.data_ptr(), stream or None), where)
    return q_out, k_out


def rotate(op: Rotary, q, k, positions, q_out=None, k_out=None, stream=None):
    """Turns the heads of q [tokens, q_heads, dim] and k [tokens, k_heads, dim]
    by the angles of positions (int32 [axes, tokens]).  Returns (q_out, k_out);
    they may be q and k themselves."""
    return _rotate(op, q, k, positions, 0, q_out, k_out, stream, "rotate")


def rotate_backward(op: Rotary, grad_q, grad_k, positions, q_out=None, k_out=None, stream=None):
    """Gradients of rotate's inputs from those of its outputs."""
    return _rotate(op, grad_q, grad_k, positions, 1, q_out, k_out, stream, "rotate_backward")


def norm_rotate(op: Rotary, q, k, positions, q_gain, k_gain, eps: float = 1e-6, q_out=None,
                k_out=None, stream=None):
    """rotate of the RMS norm of each head times a gain [dim]."""
    import torch
    where = "norm_rotate"
    _device_tensors(where, q, k, positions, q_gain, k_gain)
    stream, ctx = _m._alloc_stream(stream, q.device, q_out is None or k_out is None)
    with ctx:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        dims = _rotary_dims(op, where, q, k, positions, (("q_out", q_out, q), ("k_out", k_out, k)))
        _check_gain(where, op, q, q_gain, k_gain)
        _m._check(_m._lib.mdcn_norm_rotate(
            op.handle, _m.dtype_code(q.dtype), dims, q.data_ptr(), k.data_ptr(),
            positions.data_ptr(), q_gain.data_ptr(), k_gain.data_ptr(), eps, q_out.data_ptr(),
            k_out.data_ptr(), stream or None), where)
    return q_out, k_out


def norm_rotate_backward(op: Rotary, q, k, positions, q_gain, k_gain, grad_q_out, grad_k_out,
                         eps: float = 1e-6, workspace=None, stream=None):
    """Gradients of norm_rotate: a dict of q, k, q_gain, k_gain."""
    import torch
    where = "norm_rotate_backward"
    _device_tensors(where, q, k, positions, q_gain, k_gain, grad_q_out, grad_k_out)
    stream, ctx = _m._alloc_stream(stream, q.device, True)
    with ctx:
        g = {"q": torch.empty(q.shape, dtype=q.dtype, device=q.device),
             "k": torch.empty(k.shape, dtype=k.dtype, device=k.device),
             "q_gain": torch.empty(op.dim, dtype=q.dtype, device=q.device),
             "k_gain": torch.empty(op.dim, dtype=q.dtype, device=q.device)}
        dims = _rotary_dims(op, where, q, k, positions,
                            (("grad_q_out", grad_q_out, q), ("grad_k_out", grad_k_out, k),
                             ("grad_q", g["q"], q), ("grad_k", g["k"], k)))
        _check_gain(where, op, q, q_gain, k_gain)
        lib = _m._lib
        if workspace is None:
            n = ctypes.c_size_t()
            _m._check(lib.mdcn_norm_rotate_backward_workspace_bytes(op.handle, q.shape[0],
                                                                    ctypes.byref(n)), where)
            workspace = torch.empty(n.value, dtype=torch.uint8, device=q.device)
        _m._check(lib.mdcn_norm_rotate_backward(
            op.handle, _m.dtype_code(q.dtype), dims, q.data_ptr(), k.data_ptr(),
            positions.data_ptr(), q_gain.data_ptr(), k_gain.data_ptr(), eps,
            grad_q_out.data_ptr(), grad_k_out.data_ptr(), g["q"].data_ptr(), g["k"].data_ptr(),
            g["q_gain"].data_ptr(), g["k_gain"].data_ptr(), workspace.data_ptr(),
            workspace.numel(), stream or None), where)
    return g


# ---------------------------------------------------------------- attention

def _attend_dims(op, where, q, k, v, out, cu_q, cu_k, used_k, grads):
    """(ctypes dims, workspace bytes) of a call, checked once per combination
    of shapes and strides."""
    views = (q, k, v, out) + grads
    ints = (cu_q, cu_k) + (() if used_k is None else (used_k,))
    key = tuple((t.dtype, t.device, t.shape, t.stride()) for t in views + ints)
    call = op.calls.get(key)
    if call is None:
        if q.dim() != 3 or k.dim() != 3:
            _fail(where, "q and k must be [tokens, heads, dim]")
        q_shape = (q.shape[0], op.q_heads, op.dim)
        k_shape = (k.shape[0], op.k_heads, op.dim)
        for name, t, shape in zip(("q", "k", "v", "out", "grad_out", "grad_q", "grad_k", "grad_v"),
                                  views, (q_shape, k_shape, k_shape, q_shape, q_shape, q_shape,
                                          k_shape, k_shape)):
            _check_view(where, name, t, q, shape)
        if cu_q.dim() != 1 or cu_q.shape[0] < 1:
            _fail(where, "cu_q must hold batch + 1 offsets")
        batch = cu_q.shape[0] - 1
        _check_ints(where, "cu_q", cu_q, q, (batch + 1,))
        _check_ints(where, "cu_k", cu_k, q, (batch + 1,))
        if used_k is not None:
            _check_ints(where, "used_k", used_k, q, (batch,))
        vals = [batch, q.shape[0], k.shape[0]]
        for t in views:
            vals += _strides(t)
        dims = (_i64 * len(vals))(*vals)
        n = ctypes.c_size_t()
        lib = _m.library()
        fn = lib.mdcn_attend_backward_workspace_bytes if grads else lib.mdcn_attend_workspace_bytes
        _m._check(fn(op.handle, _m.dtype_code(q.dtype), dims, ctypes.byref(n)), where)
        call = _remember(op.calls, key, (dims, n.value))
    return call


def attend(op: Attention, q, k, v, cu_q, cu_k, used_k=None, out=None, lse=None, workspace=None,
           stream=None):
    """Attention of packed sequences: q [q_tokens, q_heads, dim], k and v
    [k_tokens, k_heads, dim], cu_q and cu_k int32 [batch + 1] offsets of the
    sequences.  used_k (int32 [batch]): the keys that sequence b's part of k and
    v holds so far, for a cache with room.  Returns (out, lse) with lse fp32
    [q_heads, q_tokens]."""
    import torch
    _device_tensors("attend", q, k, v, cu_q, cu_k)
    stream, ctx = _m._alloc_stream(stream, q.device, True)
    with ctx:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty((op.q_heads, q.shape[0]), dtype=torch.float32, device=q.device)
        elif lse.dtype != torch.float32 or lse.device != q.device or not lse.is_contiguous() or \
                tuple(lse.shape) != (op.q_heads, q.shape[0]):
            _fail("attend", "lse must be contiguous fp32 [q_heads, q_tokens]")
        dims, need = _attend_dims(op, "attend", q, k, v, out, cu_q, cu_k, used_k, ())
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        _m._check(_m._lib.mdcn_attend(
            op.handle, _m.dtype_code(q.dtype), dims, q.data_ptr(), k.data_ptr(), v.data_ptr(),
            cu_q.data_ptr(), cu_k.data_ptr(), None if used_k is None else used_k.data_ptr(),
            out.data_ptr(), lse.data_ptr(), None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel(), stream or None), "attend")
    return out, lse


def attend_backward(op: Attention, q, k, v, out, lse, grad_out, cu_q, cu_k, used_k=None,
                    workspace=None, stream=None):
    """Gradients of attend: a dict of q, k, v.  out and lse are the forward's."""
    import torch
    where = "attend_backward"
    _device_tensors(where, q, k, v, out, lse, grad_out, cu_q, cu_k)
    if lse.dtype != torch.float32 or lse.device != q.device or not lse.is_contiguous() or \
            tuple(lse.shape) != (op.q_heads, q.shape[0]):
        _fail(where, "lse must be contiguous fp32 [q_heads, q_tokens]")
    stream, ctx = _m._alloc_stream(stream, q.device, True)
    with ctx:
        g = {"q": torch.empty(q.shape, dtype=q.dtype, device=q.device),
             "k": torch.empty(k.shape, dtype=k.dtype, device=k.device),
             "v": torch.empty(v.shape, dtype=v.dtype, device=v.device)}
        dims, need = _attend_dims(op, where, q, k, v, out, cu_q, cu_k, used_k,
                                  (grad_out, g["q"], g["k"], g["v"]))
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        _m._check(_m._lib.mdcn_attend_backward(
            op.handle, _m.dtype_code(q.dtype), dims, q.data_ptr(), k.data_ptr(), v.data_ptr(),
            out.data_ptr(), lse.data_ptr(), grad_out.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(),
            None if used_k is None else used_k.data_ptr(), g["q"].data_ptr(), g["k"].data_ptr(),
            g["v"].data_ptr(), workspace.data_ptr(), workspace.numel(), stream or None), where)
    return g
