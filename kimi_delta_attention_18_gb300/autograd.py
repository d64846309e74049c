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
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lm
from . import _native as _k


class KDAPrefill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, S0, cu_seqlens, num_segments):
        out, S_final = _k.prefill_chunked(q, k, v, g, beta, S0, cu_seqlens,
                                          num_segments=num_segments)
        ctx.save_for_backward(q, k, v, g, beta, S0, cu_seqlens)
        ctx.has_S0 = S0 is not None
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
                                                         d_S_final, want_dS0=ctx.has_S0)
        return (dq.to(q.dtype), dk.to(k.dtype), dv.to(v.dtype), dg, dbeta,
                dS0 if ctx.has_S0 else None, None, None)


def kda_prefill(q, k, v, g, beta, S0=None, cu_seqlens=None, *, num_segments=0):
    """Differentiable one-call prefill (see the module docstring).  Inputs as for
    ``prefill_chunked``; returns ``(o, S_final)``."""
    if cu_seqlens is None:
        cu_seqlens = torch.tensor([0, q.shape[0]], dtype=torch.int32, device=q.device)
    return KDAPrefill.apply(q, k, v, g, beta, S0, cu_seqlens, num_segments)


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, weight, act, eps):
        ctx.save_for_backward(x, gate, weight)
        ctx.act, ctx.eps = act, eps
        return _lm.gated_norm(x, gate, weight, act=act, eps=eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        x, gate, weight = ctx.saved_tensors
        dx, d_gate, d_weight = _lm.gated_norm_backward(
            d_out.contiguous(), x, gate, weight, act=ctx.act, eps=ctx.eps,
            want_d_weight=ctx.needs_input_grad[2])
        return dx, d_gate, d_weight, None, None


def kda_gated_norm(x, gate=None, weight=None, *, act="sigmoid", eps=1e-6):
    """Differentiable ``gated_norm``."""
    return GatedNorm.apply(x, gate, weight, act, eps)


class ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, y, weight, scale, eps):
        h_out, out = _lm.residual_norm(h, y, weight, scale=scale, eps=eps)
        ctx.save_for_backward(h_out, weight)
        ctx.scale, ctx.eps, ctx.has_y = scale, eps, y is not None
        return (h_out, out) if ctx.has_y else out

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        h_out, weight = ctx.saved_tensors
        d_h, d_out = grads if ctx.has_y else (None, grads[0])
        d_out = torch.zeros_like(h_out) if d_out is None else d_out.contiguous()
        dh, dy, d_weight = _lm.residual_norm_backward(
            d_out, h_out, weight, None if d_h is None else d_h.contiguous(), scale=ctx.scale,
            eps=ctx.eps, want_dy=ctx.has_y, want_d_weight=ctx.needs_input_grad[2])
        return dh, dy, d_weight, None, None


def kda_residual_norm(h, y=None, weight=None, *, scale=1.0, eps=1e-6):
    """Differentiable ``residual_norm``; returns ``(h_out, out)``."""
    if y is None:
        return h, ResidualNorm.apply(h, None, weight, scale, eps)
    return ResidualNorm.apply(h, y, weight, scale, eps)


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, scale):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale = table.shape[0], scale
        return _lm.embedding(table, ids, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        ids, = ctx.saved_tensors
        return _lm.embedding_backward(d_out.contiguous(), ids, ctx.rows, scale=ctx.scale), None, None


def kda_embedding(table, ids, *, scale=1.0):
    """Differentiable ``embedding``."""
    return Embedding.apply(table, ids, scale)


class LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, targets, ignore_index, mean):
        loss, lse, total = _lm.linear_cross_entropy(x, weight, targets, ignore_index=ignore_index)
        ctx.save_for_backward(x, weight, targets, lse)
        ctx.ignore_index, ctx.mean = ignore_index, mean
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
            want_dx=ctx.needs_input_grad[0], want_d_weight=ctx.needs_input_grad[1])
        return dx, d_weight, None, None, None


def kda_linear_cross_entropy(x, weight, targets, *, ignore_index=-100, reduction="mean"):
    """Differentiable ``linear_cross_entropy``: the mean loss over the rows whose target
    is not ignore_index, their "sum", or the per-row losses ("none")."""
    if reduction not in ("mean", "sum", "none"):
        raise ValueError("reduction must be mean, sum or none")
    loss = LinearCrossEntropy.apply(x, weight, targets, ignore_index, reduction == "mean")
    return loss.sum() if reduction == "sum" else loss
