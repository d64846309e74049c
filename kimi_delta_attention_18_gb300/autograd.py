"""The library's operators as differentiable PyTorch operations.

``kda_prefill(q, k, v, g, beta, S0=None, cu_seqlens=None)`` returns
``(o, S_final)``: the forward is kda_prefill_chunked, the backward
kda_prefill_backward (both libkda kernels); gradients flow to q, k, v, g (the
log-decay), beta and S0 for any loss of o and S_final.  The library's gradients
are fp32; they are cast to each input's dtype (BF16 q, k, v get BF16 gradients).

Around the mixer: ``kda_gated_norm`` (x, gate, weight), ``kda_residual_norm`` (h, y,
weight), ``kda_embedding`` (the table) and ``kda_linear_cross_entropy`` (x, weight),
each with its library forward and backward; gradients have their inputs' dtypes
(norm weights fp32).

The gradients are not differentiable themselves: a second derivative through one of
these operations raises an error.

``dev_status`` (a device int32 tensor, zero before the first call) gets the first error
that a kernel of the forward or the backward pass meets: an id or a target outside its
range (KDA_ERR_INVALID_ARG), a bounded wait that gave up (KDA_ERR_TIMEOUT, the results
are incomplete).  Without it such an error goes unnoticed; read it where the program
waits for the device anyway.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lm
from . import _native as _k


class KDAPrefill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, S0, cu_seqlens, num_segments, dev_status):
        out, S_final = _k.prefill_chunked(q, k, v, g, beta, S0, cu_seqlens,
                                          num_segments=num_segments, dev_status=dev_status)
        ctx.save_for_backward(q, k, v, g, beta, S0, cu_seqlens)
        ctx.has_S0, ctx.dev_status = S0 is not None, dev_status
        return out, S_final

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out, d_S_final):
        q, k, v, g, beta, S0, cu_seqlens = ctx.saved_tensors
        if d_out is None:
            d_out = torch.zeros((q.shape[0], q.shape[1], v.shape[2]), dtype=q.dtype,
                                device=q.device)
        d_out = d_out.to(q.dtype).contiguous()
        if d_S_final is not None:
            d_S_final = d_S_final.float().contiguous()
        dq, dk, dv, dg, dbeta, dS0 = _k.prefill_backward(q, k, v, g, beta, S0, cu_seqlens, d_out,
                                                         d_S_final, want_dS0=ctx.has_S0,
                                                         dev_status=ctx.dev_status)
        return (dq.to(q.dtype), dk.to(k.dtype), dv.to(v.dtype), dg, dbeta,
                dS0 if ctx.has_S0 else None, None, None, None)


def kda_prefill(q, k, v, g, beta, S0=None, cu_seqlens=None, *, num_segments=0, dev_status=None):
    """Differentiable one-call prefill (see the module docstring).  Inputs as for
    ``prefill_chunked``; returns ``(o, S_final)``."""
    if cu_seqlens is None:
        cu_seqlens = torch.tensor([0, q.shape[0]], dtype=torch.int32, device=q.device)
    return KDAPrefill.apply(q, k, v, g, beta, S0, cu_seqlens, num_segments, dev_status)


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, weight, act, eps, dev_status):
        ctx.save_for_backward(x, gate, weight)
        ctx.act, ctx.eps, ctx.dev_status = act, eps, dev_status
        return _lm.gated_norm(x, gate, weight, act=act, eps=eps, dev_status=dev_status)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        x, gate, weight = ctx.saved_tensors
        dx, d_gate, d_weight = _lm.gated_norm_backward(
            d_out.contiguous(), x, gate, weight, act=ctx.act, eps=ctx.eps,
            want_d_weight=ctx.needs_input_grad[2], dev_status=ctx.dev_status)
        return dx, d_gate, d_weight, None, None, None


def kda_gated_norm(x, gate=None, weight=None, *, act="sigmoid", eps=1e-6, dev_status=None):
    """Differentiable ``gated_norm``."""
    return GatedNorm.apply(x, gate, weight, act, eps, dev_status)


class ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, y, weight, scale, eps, dev_status):
        h_out, out = _lm.residual_norm(h, y, weight, scale=scale, eps=eps, dev_status=dev_status)
        ctx.save_for_backward(h_out, weight)
        ctx.scale, ctx.eps, ctx.has_y, ctx.dev_status = scale, eps, y is not None, dev_status
        return (h_out, out) if ctx.has_y else out

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        h_out, weight = ctx.saved_tensors
        d_h, d_out = grads if ctx.has_y else (None, grads[0])
        d_out = torch.zeros_like(h_out) if d_out is None else d_out.contiguous()
        dh, dy, d_weight = _lm.residual_norm_backward(
            d_out, h_out, weight, None if d_h is None else d_h.contiguous(), scale=ctx.scale,
            eps=ctx.eps, want_dy=ctx.has_y, want_d_weight=ctx.needs_input_grad[2],
            dev_status=ctx.dev_status)
        return dh, dy, d_weight, None, None, None


def kda_residual_norm(h, y=None, weight=None, *, scale=1.0, eps=1e-6, dev_status=None):
    """Differentiable ``residual_norm``; returns ``(h_out, out)``."""
    if y is None:
        return h, ResidualNorm.apply(h, None, weight, scale, eps, dev_status)
    return ResidualNorm.apply(h, y, weight, scale, eps, dev_status)


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, scale, dev_status):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale, ctx.dev_status = table.shape[0], scale, dev_status
        return _lm.embedding(table, ids, scale=scale, dev_status=dev_status)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        ids, = ctx.saved_tensors
        d_table = _lm.embedding_backward(d_out.contiguous(), ids, ctx.rows, scale=ctx.scale,
                                         dev_status=ctx.dev_status)
        return d_table, None, None, None


def kda_embedding(table, ids, *, scale=1.0, dev_status=None):
    """Differentiable ``embedding``."""
    return Embedding.apply(table, ids, scale, dev_status)


class LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, targets, ignore_index, mean, dev_status):
        loss, lse, total = _lm.linear_cross_entropy(x, weight, targets, ignore_index=ignore_index,
                                                    dev_status=dev_status)
        ctx.save_for_backward(x, weight, targets, lse)
        ctx.ignore_index, ctx.mean, ctx.dev_status = ignore_index, mean, dev_status
        return total if mean else loss

    @staticmethod
    @once_differentiable
    def backward(ctx, d_loss):
        x, weight, targets, lse = ctx.saved_tensors
        if ctx.mean:  # over the rows that have a loss
            kept = (targets != ctx.ignore_index) & (targets >= 0) & (targets < weight.shape[0])
            d_loss = (d_loss / kept.sum().clamp(min=1)).expand(x.shape[0])
        dx, d_weight = _lm.linear_cross_entropy_backward(
            x, weight, targets, lse, d_loss.float().contiguous(), ignore_index=ctx.ignore_index,
            want_dx=ctx.needs_input_grad[0], want_d_weight=ctx.needs_input_grad[1],
            dev_status=ctx.dev_status)
        return dx, d_weight, None, None, None, None


def kda_linear_cross_entropy(x, weight, targets, *, ignore_index=-100, reduction="mean",
                             dev_status=None):
    """Differentiable ``linear_cross_entropy``: the mean loss over the rows whose target
    is not ignore_index, their "sum", or the per-row losses ("none")."""
    if reduction not in ("mean", "sum", "none"):
        raise ValueError("reduction must be mean, sum or none")
    loss = LinearCrossEntropy.apply(x, weight, targets, ignore_index, reduction == "mean",
                                    dev_status)
    return loss.sum() if reduction == "sum" else loss
