"""ctypes binding to libkda.so for the operators around the mixer: the norms with
gate and residual, the token embedding, and softmax cross entropy over the
vocabulary.  As in ``_native``: argument marshalling only; outputs the caller did
not pass are allocated with torch, launches go to the current stream (or
``stream``), and every library error raises ``KDAError``.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native as _k
from ._native import _ACT, _check, _need, _ptr, _stream

ACTS = {"none": 0, "sigmoid": 1, "silu": 2}
_IDS = {torch.int32: 0, torch.int64: 1}


class NormDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("gate_stride", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("width", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("eps", ctypes.c_float)]


class EmbedDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("rows", ctypes.c_int32), ("width", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("id_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class CrossEntropyDesc(ctypes.Structure):
    _fields_ = [("ignore_index", ctypes.c_int64), ("tokens", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("width", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("id_dtype", ctypes.c_int32),
                ("piece", ctypes.c_int32)]


def bind(L):
    """Declare the C signatures of this module's entry points on the loaded library."""
    P, I, Z, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    N, E, C = (ctypes.POINTER(t) for t in (NormDesc, EmbedDesc, CrossEntropyDesc))
    for name, args in (
            ("kda_gated_norm_forward", [N] + [P] * 5),
            ("kda_gated_norm_backward", [N] + [P] * 8 + [Z, P]),
            ("kda_residual_norm_forward", [N] + [P] * 3 + [F] + [P] * 3),
            ("kda_residual_norm_backward", [N] + [P] * 4 + [F] + [P] * 4 + [Z, P]),
            ("kda_embedding_forward", [E] + [P] * 5),
            ("kda_embedding_backward", [E] + [P] * 4 + [Z, P, P]),
            ("kda_linear_ce_forward", [C] + [P] * 7 + [Z, P, P]),
            ("kda_linear_ce_backward", [C] + [P] * 8 + [Z, P, P])):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = ctypes.c_int, args
    for name, args in (("kda_norm_backward_workspace_size", [N]),
                       ("kda_embedding_backward_workspace_size", [E]),
                       ("kda_linear_ce_workspace_size", [C, I])):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = Z, args


def _act(t, name):
    act = _ACT.get(t.dtype)
    if act is None:
        raise ValueError("%s must be float32 or bfloat16" % name)
    return act


def _workspace(workspace, need, dev):
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    return workspace, workspace.numel() * workspace.element_size()


def _status(dev_status, dev):
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32, None, dev)
    return _ptr(dev_status)


# -------------------------------------------------------------------- gated norm

def _rows(t, name, dtype, shape, dev):
    """A ``[T, H, D]`` tensor whose tokens may lie further apart than H * D (a slice
    of a wider projection's output); returns the token stride, 0 where it is H * D."""
    T, H, D = shape
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda or t.device != dev:
        raise ValueError("%s must be a CUDA tensor on %s" % (name, dev))
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
    if t.is_contiguous() or T == 0:
        return 0
    sT, sH, sD = t.stride()
    if (D > 1 and sD != 1) or (H > 1 and sH != D) or (T > 1 and sT < H * D):
        raise ValueError("%s must have contiguous heads and channels" % name)
    return sT if T > 1 else 0


def _gated(x, gate, weight, act, eps):
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [T, H, D] tensor")
    if act not in ACTS:
        raise ValueError("act must be one of %s" % ", ".join(sorted(ACTS)))
    if (gate is None) != (act == "none"):
        raise ValueError("a gate is required unless act is 'none', and not allowed then")
    dev, shape = x.device, tuple(x.shape)
    xs = _rows(x, "x", x.dtype, shape, dev)
    gs = _rows(gate, "gate", x.dtype, shape, dev) if gate is not None else 0
    if weight is not None:
        _need(weight, "weight", torch.float32, shape[2:], dev)
    return NormDesc(shape[0], xs, gs, shape[1], shape[2], _act(x, "x"), ACTS[act], eps)


def gated_norm(x, gate=None, weight=None, *, act="sigmoid", eps=1e-6, out=None, stream=None):
    """RMS norm of a mixer's output per (token, head) with its gate: ``x r weight
    act(gate)`` (see kda_gated_norm_forward in kda.h).  x, gate ``[T, H, D]`` in one
    activation dtype, tokens possibly strided; weight ``[D]`` fp32 or None; act
    "sigmoid", "silu" or "none" (gate None).  Returns out ``[T, H, D]``."""
    desc = _gated(x, gate, weight, act, eps)
    dev = x.device
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    _need(out, "out", x.dtype, x.shape, dev)
    _check("kda_gated_norm_forward",
           _k.lib().kda_gated_norm_forward(desc, _ptr(x), _ptr(gate), _ptr(weight), _ptr(out),
                                           _stream(stream, dev)))
    return out


def gated_norm_backward(d_out, x, gate=None, weight=None, *, act="sigmoid", eps=1e-6,
                        want_d_weight=True, workspace=None, stream=None):
    """Gradients of ``gated_norm`` for the adjoint d_out ``[T, H, D]`` of its output:
    ``(dx, d_gate, d_weight)``, d_gate None without a gate, d_weight fp32 ``[D]`` (see
    kda_gated_norm_backward in kda.h)."""
    desc = _gated(x, gate, weight, act, eps)
    dev = x.device
    _need(d_out, "d_out", x.dtype, x.shape, dev)
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    d_gate = torch.empty(x.shape, dtype=x.dtype, device=dev) if gate is not None else None
    d_weight, ws_len = None, 0
    if want_d_weight:
        d_weight = torch.empty(x.shape[2], dtype=torch.float32, device=dev)
        workspace, ws_len = _workspace(workspace, _k.lib().kda_norm_backward_workspace_size(desc),
                                       dev)
    _check("kda_gated_norm_backward",
           _k.lib().kda_gated_norm_backward(desc, _ptr(d_out), _ptr(x), _ptr(gate), _ptr(weight),
                                            _ptr(dx), _ptr(d_gate), _ptr(d_weight),
                                            _ptr(workspace), ws_len, _stream(stream, dev)))
    return dx, d_gate, d_weight


# ----------------------------------------------------------------- residual norm

def _residual(h, weight, eps, name):
    if not isinstance(h, torch.Tensor) or h.dim() != 2:
        raise ValueError("%s must be a [T, D] tensor" % name)
    _need(h, name, h.dtype)
    if weight is not None:
        _need(weight, "weight", torch.float32, h.shape[1:], h.device)
    return NormDesc(h.shape[0], 0, 0, 1, h.shape[1], _act(h, name), 0, eps)


def residual_norm(h, y=None, weight=None, *, scale=1.0, eps=1e-6, h_out=None, out=None,
                  stream=None):
    """The residual stream's update and the next block's norm: ``h_out = h + scale y``
    and the RMS norm of it times weight (see kda_residual_norm_forward in kda.h).
    h, y ``[T, D]``; without y, h_out is h.  Returns ``(h_out, out)``."""
    desc = _residual(h, weight, eps, "h")
    dev = h.device
    if y is None:
        if h_out is not None:
            raise ValueError("h_out needs y")
        new_h = None
    else:
        _need(y, "y", h.dtype, h.shape, dev)
        new_h = torch.empty(h.shape, dtype=h.dtype, device=dev) if h_out is None else h_out
        _need(new_h, "h_out", h.dtype, h.shape, dev)
    if out is None:
        out = torch.empty(h.shape, dtype=h.dtype, device=dev)
    _need(out, "out", h.dtype, h.shape, dev)
    _check("kda_residual_norm_forward",
           _k.lib().kda_residual_norm_forward(desc, _ptr(h), _ptr(y), _ptr(weight), scale,
                                              _ptr(new_h), _ptr(out), _stream(stream, dev)))
    return (h if y is None else new_h), out


def residual_norm_backward(d_out, h_out, weight=None, d_h_out=None, *, scale=1.0, eps=1e-6,
                           want_dy=True, want_d_weight=True, workspace=None, stream=None):
    """Gradients of ``residual_norm`` from its h_out, for the adjoints d_out of the
    norm and d_h_out (None: zero) of h_out: ``(dh, dy, d_weight)`` (see
    kda_residual_norm_backward in kda.h).  With scale 1, dy is dh itself."""
    desc = _residual(h_out, weight, eps, "h_out")
    dev, like = h_out.device, dict(dtype=h_out.dtype, device=h_out.device)
    _need(d_out, "d_out", h_out.dtype, h_out.shape, dev)
    if d_h_out is not None:
        _need(d_h_out, "d_h_out", h_out.dtype, h_out.shape, dev)
    dh = torch.empty(h_out.shape, **like)
    dy = torch.empty(h_out.shape, **like) if want_dy and scale != 1.0 else None
    d_weight, ws_len = None, 0
    if want_d_weight:
        d_weight = torch.empty(h_out.shape[1], dtype=torch.float32, device=dev)
        workspace, ws_len = _workspace(workspace, _k.lib().kda_norm_backward_workspace_size(desc),
                                       dev)
    _check("kda_residual_norm_backward",
           _k.lib().kda_residual_norm_backward(desc, _ptr(d_out), _ptr(d_h_out), _ptr(h_out),
                                               _ptr(weight), scale, _ptr(dh), _ptr(dy),
                                               _ptr(d_weight), _ptr(workspace), ws_len,
                                               _stream(stream, dev)))
    return dh, (dh if want_dy and scale == 1.0 else dy), d_weight


# --------------------------------------------------------------------- embedding

def _ids(ids, name, dev, count=None):
    if not isinstance(ids, torch.Tensor) or ids.dim() != 1:
        raise ValueError("%s must be a [T] tensor" % name)
    kind = _IDS.get(ids.dtype)
    if kind is None:
        raise ValueError("%s must be int32 or int64" % name)
    _need(ids, name, ids.dtype, None if count is None else (count,), dev)
    return kind


def embedding(table, ids, *, scale=1.0, out=None, dev_status=None, stream=None):
    """``out[t] = scale table[ids[t]]`` (see kda_embedding_forward in kda.h): table
    ``[V, D]``, ids ``[T]`` int32 or int64.  An id outside the table gives a zero row
    and status 1 in dev_status (a device int32)."""
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a [V, D] tensor")
    _need(table, "table")
    dev = table.device
    kind = _ids(ids, "ids", dev)
    T, (V, D) = ids.shape[0], table.shape
    desc = EmbedDesc(T, V, D, _act(table, "table"), kind, scale)
    if out is None:
        out = torch.empty((T, D), dtype=table.dtype, device=dev)
    _need(out, "out", table.dtype, (T, D), dev)
    _check("kda_embedding_forward",
           _k.lib().kda_embedding_forward(desc, _ptr(table), _ptr(ids), _ptr(out),
                                          _status(dev_status, dev), _stream(stream, dev)))
    return out


def embedding_backward(d_out, ids, num_rows, *, scale=1.0, d_table=None, workspace=None,
                       dev_status=None, stream=None):
    """The gradient ``[num_rows, D]`` of ``embedding``'s table for the adjoint d_out
    ``[T, D]``, in d_out's dtype (see kda_embedding_backward in kda.h)."""
    if not isinstance(d_out, torch.Tensor) or d_out.dim() != 2:
        raise ValueError("d_out must be a [T, D] tensor")
    _need(d_out, "d_out")
    dev, (T, D) = d_out.device, d_out.shape
    desc = EmbedDesc(T, num_rows, D, _act(d_out, "d_out"), _ids(ids, "ids", dev, T), scale)
    if d_table is None:
        d_table = torch.empty((num_rows, D), dtype=d_out.dtype, device=dev)
    _need(d_table, "d_table", d_out.dtype, (num_rows, D), dev)
    workspace, ws_len = _workspace(
        workspace, _k.lib().kda_embedding_backward_workspace_size(desc), dev)
    _check("kda_embedding_backward",
           _k.lib().kda_embedding_backward(desc, _ptr(d_out), _ptr(ids), _ptr(d_table),
                                           _ptr(workspace), ws_len, _status(dev_status, dev),
                                           _stream(stream, dev)))
    return d_table


# ----------------------------------------------------------------- cross entropy

def _ce(x, weight, targets, ignore_index, piece):
    for t, name in ((x, "x"), (weight, "weight")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError("%s must be a matrix" % name)
    _need(x, "x")
    dev, (T, D) = x.device, x.shape
    _need(weight, "weight", x.dtype, None, dev)
    if weight.shape[1] != D:
        raise ValueError("weight must have shape [V, %d], got %s" % (D, tuple(weight.shape)))
    return CrossEntropyDesc(ignore_index, T, weight.shape[0], D, _act(x, "x"),
                            _ids(targets, "targets", dev, T), piece)


def linear_cross_entropy(x, weight, targets, *, ignore_index=-100, loss=None, lse=None,
                         workspace=None, dev_status=None, stream=None):
    """Softmax cross entropy of the logits ``x weight^T`` without storing them (see
    kda_linear_ce_forward in kda.h): x ``[T, D]``, weight ``[V, D]``, targets ``[T]``
    int32 or int64.  Returns ``(loss [T], lse [T], mean)`` in fp32, mean over the rows
    whose target is not ignore_index."""
    desc = _ce(x, weight, targets, ignore_index, 0)
    dev, T = x.device, x.shape[0]
    f32 = dict(dtype=torch.float32, device=dev)
    loss = torch.empty(T, **f32) if loss is None else _need(loss, "loss", torch.float32, (T,), dev)
    lse = torch.empty(T, **f32) if lse is None else _need(lse, "lse", torch.float32, (T,), dev)
    mean = torch.empty((), **f32)
    workspace, ws_len = _workspace(workspace, _k.lib().kda_linear_ce_workspace_size(desc, 0), dev)
    _check("kda_linear_ce_forward",
           _k.lib().kda_linear_ce_forward(desc, _ptr(x), _ptr(weight), _ptr(targets), _ptr(loss),
                                          _ptr(lse), _ptr(mean), _ptr(workspace), ws_len,
                                          _status(dev_status, dev), _stream(stream, dev)))
    return loss, lse, mean


def linear_cross_entropy_backward(x, weight, targets, lse, d_loss, *, ignore_index=-100, piece=0,
                                  want_dx=True, want_d_weight=True, workspace=None,
                                  dev_status=None, stream=None):
    """Gradients ``(dx, d_weight)`` of ``linear_cross_entropy`` for the adjoint d_loss
    ``[T]`` fp32 of its per-row loss (see kda_linear_ce_backward in kda.h); ``piece``
    vocabulary columns at a time (0: the library's choice)."""
    desc = _ce(x, weight, targets, ignore_index, piece)
    dev, T = x.device, x.shape[0]
    _need(lse, "lse", torch.float32, (T,), dev)
    _need(d_loss, "d_loss", torch.float32, (T,), dev)
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if want_dx else None
    d_weight = torch.empty(weight.shape, dtype=x.dtype, device=dev) if want_d_weight else None
    workspace, ws_len = _workspace(workspace, _k.lib().kda_linear_ce_workspace_size(desc, 1), dev)
    _check("kda_linear_ce_backward",
           _k.lib().kda_linear_ce_backward(desc, _ptr(x), _ptr(weight), _ptr(targets), _ptr(lse),
                                           _ptr(d_loss), _ptr(dx), _ptr(d_weight),
                                           _ptr(workspace), ws_len, _status(dev_status, dev),
                                           _stream(stream, dev)))
    return dx, d_weight
