"""ctypes binding to libkda.so for the operators around the mixer: the norms with
gate and residual, the token embedding, and softmax cross entropy over the
vocabulary.  As in ``_native``: argument marshalling only; outputs the caller did
not pass are allocated with torch, launches go to the current stream (or
``stream``: the caller makes it wait for the inputs and waits for it before it uses the
outputs; the tensors' memory is kept for both streams), and every library error raises
``KDAError``.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native as _k
from ._native import _ACT, _check

ACTS = {"none": 0, "sigmoid": 1, "silu": 2}
_IDS = {torch.int32: 0, torch.int64: 1}


class NormDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("gate_stride", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("width", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("eps", ctypes.c_float)]


class DropoutDesc(ctypes.Structure):
    _fields_ = [("rng", ctypes.c_void_p), ("p", ctypes.c_double), ("site", ctypes.c_int32)]


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
    N, E, C, K = (ctypes.POINTER(t) for t in (NormDesc, EmbedDesc, CrossEntropyDesc, DropoutDesc))
    for name, args in (
            ("kda_gated_norm_forward", [N] + [P] * 6),
            ("kda_gated_norm_backward", [N] + [P] * 8 + [Z, P, P]),
            ("kda_residual_norm_forward", [N] + [P] * 3 + [F] + [P] * 4),
            ("kda_residual_norm_backward", [N] + [P] * 4 + [F] + [P] * 4 + [Z, P, P]),
            ("kda_residual_norm_dropout_forward", [N, K] + [P] * 3 + [F] + [P] * 4),
            ("kda_residual_norm_dropout_backward", [N, K] + [P] * 4 + [F] + [P] * 4 + [Z, P, P]),
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


# These calls are as short as a decode step's (a few microseconds on the device), so
# the host's part is kept short: one combined test per tensor (_need, and with it
# the precise error, only when that fails), plain integers instead of ctypes
# objects, and the current stream's handle without a Stream object around it.  A call
# with a stream of its own is the same call inside that stream's context.

def _lib():
    return _k._lib or _k.lib()


def _fit(n):
    """n for a 32-bit field, which would keep n's low bits only: the nearest value that it
    holds, which is beyond the library's limits wherever n is."""
    return n if -0x80000000 <= n <= 0x7fffffff else 0x7fffffff if n > 0 else -0x80000000


def _is(t, name, dtype, shape, dev):
    try:
        if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
            return
    except AttributeError:  # no tensor: _need says so
        pass
    _k._need(t, name, dtype, shape, dev)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev.index)


@functools.lru_cache(maxsize=None)
def _several():
    return torch.cuda.device_count() > 1


def _call(dev, name, *args):
    """The entry point on the tensors' device and its current stream (a launch goes to the current
    device, whatever device its tensors and stream are on)."""
    if not _several() or dev.index is None or torch._C._cuda_getDevice() == dev.index:
        rc = getattr(_lib(), name)(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = getattr(_lib(), name)(*args, _stream(dev))
    if rc:
        _check(name, rc)


def _size(dev, name, *args):
    """A workspace's size, which can depend on the device's SMs."""
    if not _several() or dev.index is None or torch._C._cuda_getDevice() == dev.index:
        return getattr(_lib(), name)(*args)
    with torch.cuda.device(dev):
        return getattr(_lib(), name)(*args)


def _first(t, name, dims):
    """Device and act_dtype of the operator's first tensor."""
    try:
        if len(t.shape) == dims and t.is_cuda:
            return t.device, _ACT[t.dtype]
    except (AttributeError, KeyError):
        pass
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError("%s must be a tensor of %d dimensions" % (name, dims))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    raise ValueError("%s must be float32 or bfloat16" % name)


def _workspace(workspace, need, dev):
    if workspace is None:
        return torch.empty(need or 16, dtype=torch.uint8, device=dev), need or 16
    if not isinstance(workspace, torch.Tensor) or workspace.device != dev:
        raise ValueError("workspace must be a tensor on %s" % dev)
    return workspace, workspace.numel() * workspace.element_size()


def _out(out, name, like):
    """A caller's output of the same type and shape as ``like``, or a new one."""
    if out is None:
        if like.is_contiguous():
            return torch.empty_like(like)
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    _is(out, name, like.dtype, like.shape, like.device)
    return out


def _status(dev_status, dev):
    if dev_status is None:
        return None
    _k._need(dev_status, "dev_status", torch.int32, None, dev)
    return dev_status.data_ptr()


# -------------------------------------------------------------------- gated norm

def _rows(t, name, like):
    """A ``[T, H, D]`` tensor like ``like`` whose tokens may lie further apart than H D
    (a slice of a wider projection's output); returns the token stride, 0 for H D."""
    if t is not like:
        try:
            ok = t.dtype is like.dtype and t.shape == like.shape and t.device == like.device
        except AttributeError:
            ok = False
        if not ok:
            if isinstance(t, torch.Tensor) and not t.is_contiguous():
                t = t.contiguous()  # for the error: the stride is not what is wrong
            _k._need(t, name, like.dtype, like.shape, like.device)
    if t.is_contiguous():
        return 0
    (T, H, D), (sT, sH, sD) = t.shape, t.stride()
    if (D > 1 and sD != 1) or (H > 1 and sH != D) or (T > 1 and sT < H * D):
        raise ValueError("%s must have contiguous heads and channels" % name)
    return sT if T > 1 else 0


def _gated(x, gate, weight, act, eps):
    dev, dtype = _first(x, "x", 3)
    kind = ACTS.get(act)
    if kind is None:
        raise ValueError("act must be one of %s" % ", ".join(sorted(ACTS)))
    if (gate is None) != (kind == 0):
        raise ValueError("a gate is required unless act is 'none', and not allowed then")
    T, H, D = x.shape
    if weight is not None:
        _is(weight, "weight", torch.float32, (D,), dev)
    return dev, NormDesc(T, _rows(x, "x", x), 0 if gate is None else _rows(gate, "gate", x),
                         _fit(H), _fit(D), dtype, kind, eps)


def gated_norm(x, gate=None, weight=None, *, act="sigmoid", eps=1e-6, out=None, dev_status=None,
               stream=None):
    """RMS norm of a mixer's output per (token, head) with its gate: ``x r weight
    act(gate)`` (see kda_gated_norm_forward in kda.h).  x, gate ``[T, H, D]`` in one
    activation dtype, tokens possibly strided; weight ``[D]`` fp32 or None; act
    "sigmoid", "silu" or "none" (gate None).  Returns out ``[T, H, D]``."""
    if stream is not None:
        return _k._on(stream, gated_norm, x, gate, weight, act=act, eps=eps, out=out,
                      dev_status=dev_status)
    dev, desc = _gated(x, gate, weight, act, eps)
    out = _out(out, "out", x)
    _call(dev, "kda_gated_norm_forward", desc, x.data_ptr(), _ptr(gate), _ptr(weight),
          out.data_ptr(), _status(dev_status, dev))
    return out


def gated_norm_backward(d_out, x, gate=None, weight=None, *, act="sigmoid", eps=1e-6,
                        want_d_weight=True, workspace=None, dev_status=None, stream=None):
    """Gradients of ``gated_norm`` for the adjoint d_out ``[T, H, D]`` of its output:
    ``(dx, d_gate, d_weight)``, d_gate None without a gate, d_weight fp32 ``[D]`` (see
    kda_gated_norm_backward in kda.h)."""
    if stream is not None:
        return _k._on(stream, gated_norm_backward, d_out, x, gate, weight, act=act, eps=eps,
                      want_d_weight=want_d_weight, workspace=workspace, dev_status=dev_status)
    dev, desc = _gated(x, gate, weight, act, eps)
    _is(d_out, "d_out", x.dtype, x.shape, dev)
    dx = _out(None, "dx", x)
    d_gate = None if gate is None else _out(None, "d_gate", x)
    d_weight, ws_len = None, 0
    if want_d_weight:
        d_weight = torch.empty(x.shape[2], dtype=torch.float32, device=dev)
        workspace, ws_len = _workspace(workspace, _size(dev, "kda_norm_backward_workspace_size", desc), dev)
    _call(dev, "kda_gated_norm_backward", desc, d_out.data_ptr(), x.data_ptr(), _ptr(gate),
          _ptr(weight), dx.data_ptr(), _ptr(d_gate), _ptr(d_weight), _ptr(workspace), ws_len,
          _status(dev_status, dev))
    return dx, d_gate, d_weight


# ----------------------------------------------------------------- residual norm

def _residual(h, weight, eps, name):
    dev, dtype = _first(h, name, 2)
    _is(h, name, h.dtype, h.shape, dev)
    T, D = h.shape
    if weight is not None:
        _is(weight, "weight", torch.float32, (D,), dev)
    return dev, NormDesc(T, 0, 0, 1, _fit(D), dtype, 0, eps)


def _dropout(p, rng, site, dev):
    """The descriptor of a dropout with probability p by the device's (seed, offset)."""
    _is(rng, "rng", torch.int64, (2,), dev)
    return DropoutDesc(rng.data_ptr(), p, _fit(site))


def residual_norm(h, y=None, weight=None, *, scale=1.0, eps=1e-6, dropout=0.0, rng=None, site=0,
                  h_out=None, out=None, dev_status=None, stream=None):
    """The residual stream's update and the next block's norm: ``h_out = h + scale y``
    and the RMS norm of it times weight (see kda_residual_norm_forward in kda.h).
    h, y ``[T, D]``; without y, h_out is h.  With ``dropout`` > 0 y is dropped out first, by
    rng and site as in ``dropout`` (see kda_residual_norm_dropout_forward in kda.h).  Returns
    ``(h_out, out)``."""
    if stream is not None:
        return _k._on(stream, residual_norm, h, y, weight, scale=scale, eps=eps, dropout=dropout,
                      rng=rng, site=site, h_out=h_out, out=out, dev_status=dev_status)
    dev, desc = _residual(h, weight, eps, "h")
    new_h = None
    if y is not None:
        _is(y, "y", h.dtype, h.shape, dev)
        new_h = _out(h_out, "h_out", h)
    elif h_out is not None:
        raise ValueError("h_out needs y")
    out = _out(out, "out", h)
    if dropout:
        if y is None:
            raise ValueError("dropout needs y")
        _call(dev, "kda_residual_norm_dropout_forward", desc, _dropout(dropout, rng, site, dev),
              h.data_ptr(), y.data_ptr(), _ptr(weight), scale, new_h.data_ptr(), out.data_ptr(),
              _status(dev_status, dev))
        return new_h, out
    _call(dev, "kda_residual_norm_forward", desc, h.data_ptr(), _ptr(y), _ptr(weight), scale,
          _ptr(new_h), out.data_ptr(), _status(dev_status, dev))
    return (h if y is None else new_h), out


def residual_norm_backward(d_out, h_out, weight=None, d_h_out=None, *, scale=1.0, eps=1e-6,
                           dropout=0.0, rng=None, site=0, want_dy=True, want_d_weight=True,
                           workspace=None, dev_status=None, stream=None):
    """Gradients of ``residual_norm`` from its h_out, for the adjoints d_out of the
    norm and d_h_out (None: zero) of h_out: ``(dh, dy, d_weight)`` (see
    kda_residual_norm_backward in kda.h).  With scale 1 and no dropout, dy is dh itself.  With
    ``dropout``, rng and site as in the forward call (rng holding what it held then)."""
    if stream is not None:
        return _k._on(stream, residual_norm_backward, d_out, h_out, weight, d_h_out, scale=scale,
                      eps=eps, dropout=dropout, rng=rng, site=site, want_dy=want_dy, want_d_weight=want_d_weight, workspace=workspace,
                      dev_status=dev_status)
    dev, desc = _residual(h_out, weight, eps, "h_out")
    _is(d_out, "d_out", h_out.dtype, h_out.shape, dev)
    if d_h_out is not None:
        _is(d_h_out, "d_h_out", h_out.dtype, h_out.shape, dev)
    dh = _out(None, "dh", h_out)
    dropped = bool(dropout) and want_dy
    dy = _out(None, "dy", h_out) if dropped or (want_dy and scale != 1.0) else None
    d_weight, ws_len = None, 0
    if want_d_weight:
        d_weight = torch.empty(h_out.shape[1], dtype=torch.float32, device=dev)
        workspace, ws_len = _workspace(workspace, _size(dev, "kda_norm_backward_workspace_size", desc), dev)
    if dropped:
        _call(dev, "kda_residual_norm_dropout_backward", desc, _dropout(dropout, rng, site, dev),
              d_out.data_ptr(), _ptr(d_h_out), h_out.data_ptr(), _ptr(weight), scale, dh.data_ptr(),
              dy.data_ptr(), _ptr(d_weight), _ptr(workspace), ws_len, _status(dev_status, dev))
        return dh, dy, d_weight
    _call(dev, "kda_residual_norm_backward", desc, d_out.data_ptr(), _ptr(d_h_out),
          h_out.data_ptr(), _ptr(weight), scale, dh.data_ptr(), _ptr(dy), _ptr(d_weight),
          _ptr(workspace), ws_len, _status(dev_status, dev))
    return dh, (dh if want_dy and scale == 1.0 else dy), d_weight


# --------------------------------------------------------------------- embedding

def _ids(ids, name, dev, count=None):
    try:
        kind = _IDS[ids.dtype]
        if len(ids.shape) != 1:
            raise ValueError("%s must be a [T] tensor" % name)
    except AttributeError:
        raise TypeError("%s must be a torch.Tensor" % name) from None
    except KeyError:
        raise ValueError("%s must be int32 or int64" % name) from None
    _is(ids, name, ids.dtype, ids.shape if count is None else (count,), dev)
    return kind


def embedding(table, ids, *, scale=1.0, out=None, dev_status=None, stream=None):
    """``out[t] = scale table[ids[t]]`` (see kda_embedding_forward in kda.h): table
    ``[V, D]``, ids ``[T]`` int32 or int64.  An id outside the table gives a zero row
    and status 1 in dev_status (a device int32)."""
    if stream is not None:
        return _k._on(stream, embedding, table, ids, scale=scale, out=out, dev_status=dev_status)
    dev, dtype = _first(table, "table", 2)
    _is(table, "table", table.dtype, table.shape, dev)
    kind = _ids(ids, "ids", dev)
    T, (V, D) = ids.shape[0], table.shape
    if out is None:
        out = torch.empty((T, D), dtype=table.dtype, device=dev)
    else:
        _is(out, "out", table.dtype, (T, D), dev)
    _call(dev, "kda_embedding_forward", EmbedDesc(_fit(T), _fit(V), _fit(D), dtype, kind, scale),
          table.data_ptr(), ids.data_ptr(), out.data_ptr(), _status(dev_status, dev))
    return out


def embedding_backward(d_out, ids, num_rows, *, scale=1.0, d_table=None, workspace=None,
                       dev_status=None, stream=None):
    """The gradient ``[num_rows, D]`` of ``embedding``'s table for the adjoint d_out
    ``[T, D]``, in d_out's dtype (see kda_embedding_backward in kda.h)."""
    if stream is not None:
        return _k._on(stream, embedding_backward, d_out, ids, num_rows, scale=scale, d_table=d_table,
                      workspace=workspace, dev_status=dev_status)
    dev, dtype = _first(d_out, "d_out", 2)
    _is(d_out, "d_out", d_out.dtype, d_out.shape, dev)
    T, D = d_out.shape
    desc = EmbedDesc(_fit(T), _fit(num_rows), _fit(D), dtype, _ids(ids, "ids", dev, T), scale)
    if d_table is None:
        d_table = torch.empty((num_rows, D), dtype=d_out.dtype, device=dev)
    else:
        _is(d_table, "d_table", d_out.dtype, (num_rows, D), dev)
    workspace, ws_len = _workspace(workspace, _size(dev, "kda_embedding_backward_workspace_size", desc), dev)
    _call(dev, "kda_embedding_backward", desc, d_out.data_ptr(), ids.data_ptr(), d_table.data_ptr(),
          workspace.data_ptr(), ws_len, _status(dev_status, dev))
    return d_table


# ----------------------------------------------------------------- cross entropy

def _ce(x, weight, targets, ignore_index, piece):
    dev, dtype = _first(x, "x", 2)
    _first(weight, "weight", 2)
    T, D = x.shape
    _is(x, "x", x.dtype, x.shape, dev)
    _is(weight, "weight", x.dtype, (weight.shape[0], D), dev)
    return dev, CrossEntropyDesc(ignore_index, _fit(T), _fit(weight.shape[0]), _fit(D), dtype,
                                 _ids(targets, "targets", dev, T), _fit(piece))


def _vector(t, name, T, dev):
    if t is None:
        return torch.empty(T, dtype=torch.float32, device=dev)
    _is(t, name, torch.float32, (T,), dev)
    return t


def linear_cross_entropy(x, weight, targets, *, ignore_index=-100, loss=None, lse=None,
                         workspace=None, dev_status=None, stream=None):
    """Softmax cross entropy of the logits ``x weight^T`` without storing them (see
    kda_linear_ce_forward in kda.h): x ``[T, D]``, weight ``[V, D]``, targets ``[T]``
    int32 or int64.  Returns ``(loss [T], lse [T], mean)`` in fp32, mean over the rows
    whose target is not ignore_index."""
    if stream is not None:
        return _k._on(stream, linear_cross_entropy, x, weight, targets, ignore_index=ignore_index,
                      loss=loss, lse=lse, workspace=workspace, dev_status=dev_status)
    dev, desc = _ce(x, weight, targets, ignore_index, 0)
    T = x.shape[0]
    loss, lse = _vector(loss, "loss", T, dev), _vector(lse, "lse", T, dev)
    mean = torch.empty((), dtype=torch.float32, device=dev)
    workspace, ws_len = _workspace(workspace, _size(dev, "kda_linear_ce_workspace_size", desc, 0), dev)
    _call(dev, "kda_linear_ce_forward", desc, x.data_ptr(), weight.data_ptr(), targets.data_ptr(),
          loss.data_ptr(), lse.data_ptr(), mean.data_ptr(), workspace.data_ptr(), ws_len,
          _status(dev_status, dev))
    return loss, lse, mean


def linear_cross_entropy_backward(x, weight, targets, lse, d_loss, *, ignore_index=-100, piece=0,
                                  want_dx=True, want_d_weight=True, workspace=None,
                                  dev_status=None, stream=None):
    """Gradients ``(dx, d_weight)`` of ``linear_cross_entropy`` for the adjoint d_loss
    ``[T]`` fp32 of its per-row loss (see kda_linear_ce_backward in kda.h); ``piece``
    vocabulary columns at a time (0: the library's choice)."""
    if stream is not None:
        return _k._on(stream, linear_cross_entropy_backward, x, weight, targets, lse, d_loss,
                      ignore_index=ignore_index, piece=piece, want_dx=want_dx,
                      want_d_weight=want_d_weight, workspace=workspace, dev_status=dev_status)
    dev, desc = _ce(x, weight, targets, ignore_index, piece)
    T = x.shape[0]
    _is(lse, "lse", torch.float32, (T,), dev)
    _is(d_loss, "d_loss", torch.float32, (T,), dev)
    dx = _out(None, "dx", x) if want_dx else None
    d_weight = _out(None, "d_weight", weight) if want_d_weight else None
    workspace, ws_len = _workspace(workspace, _size(dev, "kda_linear_ce_workspace_size", desc, 1), dev)
    _call(dev, "kda_linear_ce_backward", desc, x.data_ptr(), weight.data_ptr(), targets.data_ptr(),
          lse.data_ptr(), d_loss.data_ptr(), _ptr(dx), _ptr(d_weight), workspace.data_ptr(), ws_len,
          _status(dev_status, dev))
    return dx, d_weight
