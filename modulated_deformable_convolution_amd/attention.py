"""Python binding of libmdcn.so's attention operators (include/mdcn.h): rotary
positions with several axes, norms of queries and keys with the rotation in
the same pass, attention over packed sequences and key/value caches, and their
backward passes.

Tensors are [tokens, heads, dim] views of device memory with the channels of a
head together (slices of a projection's output are taken as they are), one
dtype per call.  Outputs and workspaces are allocated with torch, on the stream
the call runs on; every step of the computation runs in the library's HIP
kernels.  Calls enqueue work on the current device, which must be the tensors', and
return; they raise MdcnError on bad arguments.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import mdcn as _m
from .mdcn import MDCN_E_ATTR, MDCN_E_NULL, MDCN_E_SHAPE, MdcnError

_i64 = ctypes.c_int64
_CACHED_CALLS = 64
_NO_CONTEXT = contextlib.nullcontext()


def _raw_stream(index):
    """Handle of torch's current stream on a device (0, the default stream, as None)."""
    return torch.cuda.current_stream(index).cuda_stream or None


if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    # the same handle without building a Stream object (a microsecond a call)
    def _raw_stream(index, _get=torch._C._cuda_getCurrentRawStream):  # noqa: F811
        return _get(index) or None


# torch.cuda.current_device without its checks
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _like(shape, dtype, device):
    """A one-element tensor seen as `shape`: torch.empty_like of it is a third of
    torch.empty's host time."""
    return torch.empty((), dtype=dtype, device=device).expand(shape)


def _new(template):
    return torch.empty_like(template, memory_format=torch.contiguous_format)


class Rotary:
    """Owns an mdcn_rotary handle."""

    def __init__(self, handle: int, dim: int, axes: tuple):
        self.handle, self.dim, self.axes = handle, dim, axes
        self.calls = {}          # shapes, strides, ... -> what _rotary_call returns

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
        self.calls = {}          # shapes, strides, ... -> what _attend_call returns

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


def _check_current(where, index):
    if index != _current_device():
        _fail(where, "the tensors' device must be the current one", _m.MDCN_E_DEVICE)


def _device_tensors(where, *tensors):
    for t in tensors:
        if not t.is_cuda:
            _fail(where, "tensors must be device tensors", MDCN_E_NULL)
    _check_current(where, tensors[0].get_device())


def _check_ints(where, name, t, like, shape):
    if t.dtype != torch.int32 or t.device != like.device or tuple(t.shape) != shape:
        _fail(where, "%s must be int32 of shape %s on the tensors' device" % (name, shape))
    if shape[-1] > 1 and t.stride(-1) != 1:
        _fail(where, "%s must be contiguous" % name)


def _workspace_bytes(where, workspace, like):
    if workspace is None:
        return 0
    if workspace.device != like.device or not workspace.is_contiguous():
        _fail(where, "workspace must be contiguous on the tensors' device", _m.MDCN_E_WORKSPACE)
    return workspace.numel() * workspace.element_size()


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


def _sig(t):
    """What a call's checks and dims depend on."""
    return (t.shape, t.stride(), t.dtype, t.device)


def _rotary_call(op, where, q, k, positions, more):
    """(dtype code, ctypes dims) of a call on q, k and further views."""
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
    return _m.dtype_code(q.dtype), (_i64 * len(vals))(*vals)


def _stream_of(stream, t):
    """(handle, context or None) to allocate and launch with; see mdcn._alloc_stream."""
    if stream is None:
        return _raw_stream(t.get_device()), None
    return _m._alloc_stream(stream, t.device, True)


def _check_gain(where, op, q, *gains):
    for g in gains:
        if g.dtype != q.dtype or g.device != q.device or tuple(g.shape) != (op.dim,) or \
                (op.dim > 1 and g.stride(0) != 1):
            _fail(where, "gains must hold dim values of the tensors' dtype and device")


# ---------------------------------------------------------------- rotary positions

def _outputs(stream, q, k, q_out, k_out):
    """(stream handle, q_out, k_out), allocated where not given."""
    stream, ctx = _stream_of(stream, q)
    if q_out is None or k_out is None:
        with ctx or _NO_CONTEXT:
            q_out = torch.empty_like(q) if q_out is None else q_out
            k_out = torch.empty_like(k) if k_out is None else k_out
    return stream, q_out, k_out


def _rotate(op, q, k, positions, inverse, q_out, k_out, stream, where):
    _device_tensors(where, q, k, positions)
    stream, q_out, k_out = _outputs(stream, q, k, q_out, k_out)
    key = (_sig(q), _sig(k), _sig(positions), _sig(q_out), _sig(k_out))
    call = op.calls.get(key)
    if call is None:
        call = _remember(op.calls, key, _rotary_call(
            op, where, q, k, positions, (("q_out", q_out, q), ("k_out", k_out, k))))
    st = _m._lib.mdcn_rotate(op.handle, call[0], call[1], q.data_ptr(), k.data_ptr(),
                             positions.data_ptr(), inverse, q_out.data_ptr(), k_out.data_ptr(),
                             stream)
    if st:
        _m._check(st, where)
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
    where = "norm_rotate"
    _device_tensors(where, q, k, positions, q_gain, k_gain)
    stream, q_out, k_out = _outputs(stream, q, k, q_out, k_out)
    key = (_sig(q), _sig(k), _sig(positions), _sig(q_out), _sig(k_out), _sig(q_gain), _sig(k_gain))
    call = op.calls.get(key)
    if call is None:
        _check_gain(where, op, q, q_gain, k_gain)
        call = _remember(op.calls, key, _rotary_call(
            op, where, q, k, positions, (("q_out", q_out, q), ("k_out", k_out, k))))
    st = _m._lib.mdcn_norm_rotate(op.handle, call[0], call[1], q.data_ptr(), k.data_ptr(),
                                  positions.data_ptr(), q_gain.data_ptr(), k_gain.data_ptr(), eps,
                                  q_out.data_ptr(), k_out.data_ptr(), stream)
    if st:
        _m._check(st, where)
    return q_out, k_out


def norm_rotate_backward(op: Rotary, q, k, positions, q_gain, k_gain, grad_q_out, grad_k_out,
                         eps: float = 1e-6, workspace=None, stream=None):
    """Gradients of norm_rotate: a dict of q, k, q_gain, k_gain."""
    where = "norm_rotate_backward"
    _device_tensors(where, q, k, positions, q_gain, k_gain, grad_q_out, grad_k_out)
    lib = _m._lib
    stream, ctx = _stream_of(stream, q)
    with ctx or _NO_CONTEXT:
        dq, dk = torch.empty_like(q), torch.empty_like(k)
        dq_gain, dk_gain = torch.empty_like(q_gain), torch.empty_like(k_gain)
        key = (_sig(q), _sig(k), _sig(positions), _sig(q_gain), _sig(k_gain), _sig(grad_q_out),
               _sig(grad_k_out), "backward")
        call = op.calls.get(key)
        if call is None:
            _check_gain(where, op, q, q_gain, k_gain)
            call = _rotary_call(op, where, q, k, positions,
                                (("grad_q_out", grad_q_out, q), ("grad_k_out", grad_k_out, k),
                                 ("grad_q", dq, q), ("grad_k", dk, k)))
            n = ctypes.c_size_t()
            _m._check(lib.mdcn_norm_rotate_backward_workspace_bytes(op.handle, q.shape[0],
                                                                    ctypes.byref(n)), where)
            call = _remember(op.calls, key, call + (_like((n.value,), torch.uint8, q.device),))
        if workspace is None:
            workspace = _new(call[2])
    st = lib.mdcn_norm_rotate_backward(
        op.handle, call[0], call[1], q.data_ptr(), k.data_ptr(), positions.data_ptr(),
        q_gain.data_ptr(), k_gain.data_ptr(), eps, grad_q_out.data_ptr(), grad_k_out.data_ptr(),
        dq.data_ptr(), dk.data_ptr(), dq_gain.data_ptr(), dk_gain.data_ptr(),
        workspace.data_ptr(), _workspace_bytes(where, workspace, q), stream)
    if st:
        _m._check(st, where)
    return {"q": dq, "k": dk, "q_gain": dq_gain, "k_gain": dk_gain}


# ---------------------------------------------------------------- attention

def _attend_call(op, where, views, cu_q, cu_k, used_k, grads):
    """(dtype code, ctypes dims, workspace or None, lse) of a call, the last two as
    templates for _new."""
    q, k = views[:2]
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
    code, dims = _m.dtype_code(q.dtype), (_i64 * len(vals))(*vals)
    n = ctypes.c_size_t()
    lib = _m.library()
    fn = lib.mdcn_attend_backward_workspace_bytes if grads else lib.mdcn_attend_workspace_bytes
    _m._check(fn(op.handle, code, dims, ctypes.byref(n)), where)
    return (code, dims, _like((n.value,), torch.uint8, q.device) if n.value else None,
            _like((op.q_heads, q.shape[0]), torch.float32, q.device))


def _check_lse(where, op, q, lse):
    if lse.dtype != torch.float32 or lse.device != q.device or not lse.is_contiguous() or \
            tuple(lse.shape) != (op.q_heads, q.shape[0]):
        _fail(where, "lse must be contiguous fp32 [q_heads, q_tokens]")


def attend(op: Attention, q, k, v, cu_q, cu_k, used_k=None, out=None, lse=None, workspace=None,
           stream=None):
    """Attention of packed sequences: q [q_tokens, q_heads, dim], k and v
    [k_tokens, k_heads, dim], cu_q and cu_k int32 [batch + 1] offsets of the
    sequences.  used_k (int32 [batch]): the keys that sequence b's part of k and
    v holds so far, for a cache with room.  Returns (out, lse) with lse fp32
    [q_heads, q_tokens].  Tokens before the first sequence and after the last get
    zeros and -infinity, like a row that sees no key; in an out or lse that the
    caller gives they are left as they are."""
    _device_tensors("attend", q, k, v, cu_q, cu_k)
    stream, ctx = _stream_of(stream, q)
    fill = (1 if out is None else 0) | (2 if lse is None else 0)
    with ctx or _NO_CONTEXT:
        if out is None:
            out = torch.empty_like(q)
        key = (_sig(q), _sig(k), _sig(v), _sig(out), _sig(cu_q), _sig(cu_k),
               None if used_k is None else _sig(used_k))
        call = op.calls.get(key)
        if call is None:
            call = _remember(op.calls, key, _attend_call(op, "attend", (q, k, v, out), cu_q, cu_k,
                                                         used_k, False))
        if lse is None:
            lse = _new(call[3])
        else:
            _check_lse("attend", op, q, lse)
        if workspace is None and call[2] is not None:
            workspace = _new(call[2])
    st = _m._lib.mdcn_attend_filled(
        op.handle, call[0], call[1], q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(),
        cu_k.data_ptr(), None if used_k is None else used_k.data_ptr(), fill, out.data_ptr(),
        lse.data_ptr(), None if workspace is None else workspace.data_ptr(),
        _workspace_bytes("attend", workspace, q), stream)
    if st:
        _m._check(st, "attend")
    return out, lse


def attend_backward(op: Attention, q, k, v, out, lse, grad_out, cu_q, cu_k, used_k=None,
                    workspace=None, stream=None):
    """Gradients of attend: a dict of q, k, v, with zeros for tokens of no sequence.  out
    and lse are the forward's."""
    where = "attend_backward"
    _device_tensors(where, q, k, v, out, lse, grad_out, cu_q, cu_k)
    _check_lse(where, op, q, lse)
    stream, ctx = _stream_of(stream, q)
    with ctx or _NO_CONTEXT:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        key = (_sig(q), _sig(k), _sig(v), _sig(out), _sig(grad_out), _sig(cu_q), _sig(cu_k),
               None if used_k is None else _sig(used_k), "backward")
        call = op.calls.get(key)
        if call is None:
            call = _remember(op.calls, key, _attend_call(
                op, where, (q, k, v, out, grad_out, dq, dk, dv), cu_q, cu_k, used_k, True))
        if workspace is None:
            workspace = _new(call[2])
    st = _m._lib.mdcn_attend_backward(
        op.handle, call[0], call[1], q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
        lse.data_ptr(), grad_out.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(),
        None if used_k is None else used_k.data_ptr(), dq.data_ptr(), dk.data_ptr(),
        dv.data_ptr(), workspace.data_ptr(), _workspace_bytes(where, workspace, q), stream)
    if st:
        _m._check(st, where)
    return {"q": dq, "k": dk, "v": dv}


# ---------------------------------------------------------------- what a call runs

def describe_rotate(op: Rotary, dtype, tokens: int, q_heads: int, k_heads: int) -> str:
    """One line on the shape of rotate's and norm_rotate's kernels (mdcn_describe_rotate)."""
    buf = ctypes.create_string_buffer(256)
    _m._check(_m._lib.mdcn_describe_rotate(op.handle, _m.dtype_code(dtype),
                                           (_i64 * 3)(tokens, q_heads, k_heads), buf, 256),
              "describe_rotate")
    return buf.value.decode()


def describe_attend(op: Attention, dtype, batch: int, q_tokens: int, k_tokens: int,
                    backward: bool = False) -> str:
    """One line on attend's kernels, or attend_backward's (mdcn_describe_attend)."""
    buf = ctypes.create_string_buffer(256)
    _m._check(_m._lib.mdcn_describe_attend(op.handle, _m.dtype_code(dtype),
                                           (_i64 * 3)(batch, q_tokens, k_tokens), int(backward),
                                           buf, 256), "describe_attend")
    return buf.value.decode()
