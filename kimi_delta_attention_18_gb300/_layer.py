"""ctypes binding to libkda.so for a recurrent layer's parts beside the mixer: the gated
linear recurrence, the gated feed-forward block and dropout.  As in ``_lm``: argument
marshalling only; outputs the caller did not pass are allocated with torch, launches go to
the current stream of the tensors' device (or ``stream``: the caller makes it wait for the
inputs and waits for it before it uses the outputs; the tensors' memory is kept for both
streams), and every library error raises ``KDAError``.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native as _k
from ._lm import (DropoutDesc, _call, _dropout, _first, _fit, _is, _lib, _out, _ptr, _size,
                  _status, _workspace)

WRITES = {"add": 0, "mix": 1}
FFN_ACTS = {"sigmoid": 1, "silu": 2, "gelu": 3}


class RecurrenceDesc(ctypes.Structure):
    _fields_ = [("x_stride", ctypes.c_int64), ("g_stride", ctypes.c_int64),
                ("num_seqs", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("channels", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("write", ctypes.c_int32)]


class FFNDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("width", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("act", ctypes.c_int32)]


def bind(L):
    """Declare the C signatures of this module's entry points on the loaded library."""
    P, I, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    R, F = ctypes.POINTER(RecurrenceDesc), ctypes.POINTER(FFNDesc)
    for name, args in (
            ("kda_recurrence_forward", [R] + [P] * 7 + [Z, P, P]),
            ("kda_recurrence_backward", [R] + [P] * 11 + [Z, P, P]),
            ("kda_recurrence_step", [R] + [P] * 6),
            ("kda_selftest_recurrence_timeout", [R] + [P] * 6 + [Z, P, P]),
            ("kda_dropout", [ctypes.POINTER(DropoutDesc), ctypes.c_int64, I, I] + [P] * 3),
            ("kda_gated_ffn_forward", [F] + [P] * 4 + [Z, P, P]),
            ("kda_gated_ffn_backward", [F] + [P] * 6 + [Z, P, P])):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = ctypes.c_int, args
    for name, args in (("kda_recurrence_workspace_size", [R, I]),
                       ("kda_gated_ffn_workspace_size", [F, I])):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = Z, args


# ------------------------------------------------------------ linear recurrence

def _tokens(t, name, dtype, shape, dev):
    """A ``[T, C]`` tensor whose tokens may lie further apart than C (a slice of a wider
    projection's output); returns the token stride, 0 for C."""
    if not isinstance(t, torch.Tensor) or t.is_contiguous():
        _is(t, name, dtype, shape, dev)
        return 0
    if t.dtype is not dtype or t.shape != shape or t.device != dev:
        _k._need(t.contiguous(), name, dtype, shape, dev)
    (T, C), (sT, sC) = t.shape, t.stride()
    if (C > 1 and sC != 1) or (T > 1 and sT < C):
        raise ValueError("%s must have contiguous channels" % name)
    return sT if T > 1 else 0


def _recurrence(x, g, cu_seqlens, write):
    """Device, number of sequences and descriptor of a call over packed tokens."""
    dev, dtype = _first(x, "x", 2)
    kind = WRITES.get(write)
    if kind is None:
        raise ValueError("write must be one of %s" % ", ".join(sorted(WRITES)))
    T, C = x.shape
    xs, gs = _tokens(x, "x", x.dtype, x.shape, dev), _tokens(g, "g", torch.float32, x.shape, dev)
    N = 1
    if cu_seqlens is not None:
        _k._need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a [N + 1] tensor")
        N = cu_seqlens.numel() - 1
    return dev, N, RecurrenceDesc(xs, gs, _fit(N), _fit(T), _fit(C), dtype, kind)


def _state(t, name, N, C, dev, new=False):
    if t is not None:
        _is(t, name, torch.float32, (N, C), dev)
    elif new:
        t = torch.empty((N, C), dtype=torch.float32, device=dev)
    return t


def linear_recurrence(x, g, h0=None, cu_seqlens=None, *, write="add", h=None, h_final=None,
                      want_final_state=True, workspace=None, dev_status=None, stream=None):
    """The gated linear recurrence ``h_t = e^{g_t} h_{t-1} + w_t x_t`` over packed sequences,
    w 1 (write "add") or ``1 - e^{g_t}`` ("mix") (see kda_recurrence_forward in kda.h).
    x ``[T, C]`` (fp32 or bf16) and the log-decay g ``[T, C]`` (fp32), tokens possibly
    strided; h0 ``[N, C]`` fp32 or None; cu_seqlens int32 ``[N+1]`` (None = one sequence).
    Where g is positive, products of e^g over up to 2,048 tokens must stay within fp32.
    Returns ``(h [T, C], h_final [N, C] fp32)``."""
    if stream is not None:
        return _k._on(stream, linear_recurrence, x, g, h0, cu_seqlens, write=write, h=h,
                      h_final=h_final, want_final_state=want_final_state, workspace=workspace,
                      dev_status=dev_status)
    dev, N, desc = _recurrence(x, g, cu_seqlens, write)
    C = x.shape[1]
    _state(h0, "h0", N, C, dev)
    h = _out(h, "h", x)
    h_final = _state(h_final, "h_final", N, C, dev, want_final_state)
    workspace, ws_len = _workspace(workspace, _lib().kda_recurrence_workspace_size(desc, 0), dev)
    _call(dev, "kda_recurrence_forward", desc, x.data_ptr(), g.data_ptr(), _ptr(h0),
          _ptr(cu_seqlens), h.data_ptr(), _ptr(h_final), workspace.data_ptr(), ws_len,
          _status(dev_status, dev))
    return h, h_final


def linear_recurrence_backward(d_h, x, g, h, h0=None, cu_seqlens=None, d_h_final=None, *,
                               write="add", want_d_h0=True, workspace=None, dev_status=None,
                               stream=None):
    """Gradients of ``linear_recurrence`` for the adjoints d_h ``[T, C]`` (x's dtype) of h and
    d_h_final ``[N, C]`` (fp32, None: zero) of h_final, from the forward's h:
    ``(dx, dg, d_h0)``, dx in x's dtype, dg and d_h0 fp32 (see kda_recurrence_backward in
    kda.h)."""
    if stream is not None:
        return _k._on(stream, linear_recurrence_backward, d_h, x, g, h, h0, cu_seqlens, d_h_final,
                      write=write, want_d_h0=want_d_h0, workspace=workspace,
                      dev_status=dev_status)
    dev, N, desc = _recurrence(x, g, cu_seqlens, write)
    C = x.shape[1]
    _is(d_h, "d_h", x.dtype, x.shape, dev)
    _is(h, "h", x.dtype, x.shape, dev)
    _state(h0, "h0", N, C, dev)
    _state(d_h_final, "d_h_final", N, C, dev)
    dx = _out(None, "dx", x)
    dg = torch.empty(x.shape, dtype=torch.float32, device=dev)
    d_h0 = _state(None, "d_h0", N, C, dev, want_d_h0)
    workspace, ws_len = _workspace(workspace, _lib().kda_recurrence_workspace_size(desc, 1), dev)
    _call(dev, "kda_recurrence_backward", desc, d_h.data_ptr(), x.data_ptr(), g.data_ptr(),
          h.data_ptr(), _ptr(h0), _ptr(cu_seqlens), _ptr(d_h_final), dx.data_ptr(), dg.data_ptr(),
          _ptr(d_h0), workspace.data_ptr(), ws_len, _status(dev_status, dev))
    return dx, dg, d_h0


def linear_recurrence_step(x, g, state, *, write="add", state_out=None, h=None, stream=None):
    """One token of each of N sequences (see kda_recurrence_step in kda.h): x ``[N, C]``, g
    ``[N, C]`` fp32, both possibly strided; state ``[N, C]`` fp32, updated in place unless
    state_out is given.  Returns ``(h [N, C], state_out)``."""
    if stream is not None:
        return _k._on(stream, linear_recurrence_step, x, g, state, write=write,
                      state_out=state_out, h=h)
    dev, dtype = _first(x, "x", 2)
    kind = WRITES.get(write)
    if kind is None:
        raise ValueError("write must be one of %s" % ", ".join(sorted(WRITES)))
    N, C = x.shape
    _is(state, "state", torch.float32, x.shape, dev)
    if state_out is None:
        state_out = state
    else:
        _is(state_out, "state_out", torch.float32, x.shape, dev)
    desc = RecurrenceDesc(_tokens(x, "x", x.dtype, x.shape, dev),
                          _tokens(g, "g", torch.float32, x.shape, dev), _fit(N), _fit(N), _fit(C),
                          dtype, kind)
    h = _out(h, "h", x)
    if N > 0:
        _call(dev, "kda_recurrence_step", desc, x.data_ptr(), g.data_ptr(), state.data_ptr(),
              state_out.data_ptr(), h.data_ptr())
    return h, state_out


# ------------------------------------------------------ gated feed-forward block

def _ffn(x, weight, act):
    dev, dtype = _first(x, "x", 2)
    kind = FFN_ACTS.get(act)
    if kind is None:
        raise ValueError("act must be one of %s" % ", ".join(sorted(FFN_ACTS)))
    _first(weight, "weight", 3)
    T, D = x.shape
    F = weight.shape[1]
    _is(x, "x", x.dtype, x.shape, dev)
    _is(weight, "weight", x.dtype, (2, F, D), dev)
    return dev, FFNDesc(_fit(T), _fit(D), _fit(F), dtype, kind)


def gated_ffn(x, weight, *, act="silu", h=None, workspace=None, dev_status=None, stream=None):
    """The gated feed-forward block up to its last projection: ``act(x weight[0]^T) *
    (x weight[1]^T)`` without storing the projections (see kda_gated_ffn_forward in kda.h):
    x ``[T, D]``, weight ``[2, F, D]`` in x's dtype; act "silu", "gelu" or "sigmoid".
    Returns h ``[T, F]``."""
    if stream is not None:
        return _k._on(stream, gated_ffn, x, weight, act=act, h=h, workspace=workspace,
                      dev_status=dev_status)
    dev, desc = _ffn(x, weight, act)
    T, F = x.shape[0], weight.shape[1]
    if h is None:
        h = torch.empty((T, F), dtype=x.dtype, device=dev)
    else:
        _is(h, "h", x.dtype, (T, F), dev)
    workspace, ws_len = _workspace(workspace, _size(dev, "kda_gated_ffn_workspace_size", desc, 0), dev)
    _call(dev, "kda_gated_ffn_forward", desc, x.data_ptr(), weight.data_ptr(), h.data_ptr(),
          workspace.data_ptr(), ws_len, _status(dev_status, dev))
    return h


def gated_ffn_backward(d_h, x, weight, *, act="silu", want_dx=True, want_d_weight=True,
                       workspace=None, dev_status=None, stream=None):
    """Gradients ``(dx [T, D], d_weight [2, F, D])`` of ``gated_ffn`` for the adjoint d_h
    ``[T, F]``, from its inputs alone (see kda_gated_ffn_backward in kda.h)."""
    if stream is not None:
        return _k._on(stream, gated_ffn_backward, d_h, x, weight, act=act, want_dx=want_dx,
                      want_d_weight=want_d_weight, workspace=workspace, dev_status=dev_status)
    dev, desc = _ffn(x, weight, act)
    _is(d_h, "d_h", x.dtype, (x.shape[0], weight.shape[1]), dev)
    dx = _out(None, "dx", x) if want_dx else None
    d_weight = _out(None, "d_weight", weight) if want_d_weight else None
    workspace, ws_len = _workspace(workspace, _size(dev, "kda_gated_ffn_workspace_size", desc, 1), dev)
    _call(dev, "kda_gated_ffn_backward", desc, d_h.data_ptr(), x.data_ptr(), weight.data_ptr(),
          _ptr(dx), _ptr(d_weight), workspace.data_ptr(), ws_len, _status(dev_status, dev))
    return dx, d_weight


# ------------------------------------------------------------------------ dropout

def dropout(x, p, rng, *, site=0, out=None, stream=None):
    """x ``[T, D]`` with each element kept (and divided by 1 - p) or, with probability p, 0;
    the mask comes from a counter and is never stored (see kda_dropout in kda.h).  rng: a
    device int64 tensor (seed, offset) that the kernel reads; ``site`` (0..65535) tells a
    step's dropouts apart.  The gradient is the same call on the output's adjoint, with rng
    holding what it held here.  ``out`` may be x."""
    if stream is not None:
        return _k._on(stream, dropout, x, p, rng, site=site, out=out)
    dev, dtype = _first(x, "x", 2)
    _is(x, "x", x.dtype, x.shape, dev)
    desc = _dropout(p, rng, site, dev)
    out = _out(out, "out", x)
    T, D = x.shape
    _call(dev, "kda_dropout", desc, T, _fit(D), dtype, x.data_ptr(), out.data_ptr())
    return out
