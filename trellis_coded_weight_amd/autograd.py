"""Products with coded weights, products in 8-bit blocks and the norm as differentiable functions.

The coded matrix is frozen: gradients go to the activations and to the adapters' matrices.
Activations may have any leading dimensions, [..., cols]; the row arguments (ids, offsets)
count rows in their flattened order.

A weight's levels and within-tile order are its context's: a backward pass needs those of its
forward pass and raises if the context has others by then (weights of different codebooks take a
context each).
"""
from __future__ import annotations

from typing import Optional

import torch

from .binding import Adapters, BlockWeight, CodedWeight, Context


def _rows(x: torch.Tensor) -> torch.Tensor:
    return x.reshape(-1, x.shape[-1])


def _kept(weight: CodedWeight):
    """The weight's tensors, saved so that torch sees if they change before the backward pass."""
    return weight.packed, weight.scale, weight.su, weight.sv


def _same_decoder(context: Context, decoder) -> None:
    if context._decoder() != decoder:
        raise RuntimeError("the context's codebook or within-tile order has changed since the "
                           "forward pass: set it back, or use a context for each codebook")


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, context, weight, offsets):
        ctx.args = context, weight, context._decoder()
        ctx.save_for_backward(offsets, *_kept(weight))
        if offsets is None:
            return context.linear(x, weight)
        return context.grouped_linear(x, weight, offsets)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        context, weight, decoder = ctx.args
        _same_decoder(context, decoder)
        offsets = ctx.saved_tensors[0]
        if offsets is None:
            dx = context.linear(dy, weight, transpose=True)
        else:
            dx = context.grouped_linear(dy, weight, offsets, transpose=True)
        return dx, None, None, None


class _AdapterLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, A, B, context, weight, alpha, ids):
        ctx.args = context, weight, context._decoder()
        ctx.save_for_backward(x, A, B, alpha, ids, *_kept(weight))
        return context.adapter_linear(x, weight, Adapters(A, B, alpha), ids)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        context, weight, decoder = ctx.args
        _same_decoder(context, decoder)
        x, A, B, alpha, ids = ctx.saved_tensors[:5]
        want_x, want_a, want_b = ctx.needs_input_grad[:3]
        dx, dA, dB = context.adapter_linear_backward(
            dy, x, weight, Adapters(A, B, alpha), ids, want_dx=want_x,
            want_adapters=want_a or want_b)
        return dx, dA if want_a else None, dB if want_b else None, None, None, None, None


def coded_linear(context: Context, x: torch.Tensor, weight: CodedWeight) -> torch.Tensor:
    """x [..., cols] -> x W^T [..., rows]."""
    y = _Linear.apply(_rows(x), context, weight, None)
    return y.reshape(x.shape[:-1] + (weight.rows,))


def coded_grouped_linear(context: Context, x: torch.Tensor, weight: CodedWeight,
                         offsets: torch.Tensor) -> torch.Tensor:
    """x [n, cols], sorted by group (expert) -> [n, rows]; offsets int32 [groups + 1]."""
    return _Linear.apply(x, context, weight, offsets)


def coded_adapter_linear(context: Context, x: torch.Tensor, weight: CodedWeight, A: torch.Tensor,
                         B: torch.Tensor, alpha: torch.Tensor, ids: torch.Tensor) -> torch.Tensor:
    """x [..., cols] -> x W^T + alpha_a (x A_a^T) B_a^T; ids int32, the adapter of each row or
    -1.  Differentiable in x, A and B; alpha has no gradient and may not require one."""
    if torch.is_grad_enabled() and alpha.requires_grad:
        raise ValueError("alpha requires a gradient, which is not computed: pass alpha.detach()")
    y = _AdapterLinear.apply(_rows(x), A, B, context, weight, alpha, ids.reshape(-1))
    return y.reshape(x.shape[:-1] + (weight.rows,))


class _BlockLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, context, weight, offsets):
        ctx.args = context, weight
        ctx.save_for_backward(offsets, weight.q, weight.scale)
        if offsets is None:
            return context.block_linear(x, weight)
        return context.block_grouped_linear(x, weight, offsets)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        context, weight = ctx.args
        offsets = ctx.saved_tensors[0]
        if offsets is None:
            dx = context.block_linear(dy, weight, transpose=True)
        else:
            dx = context.block_grouped_linear(dy, weight, offsets, transpose=True)
        return dx, None, None, None


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gain, residual, context, eps):
        ctx.set_materialize_grads(False)
        ctx.args = context, eps
        if residual is None:
            ctx.save_for_backward(x, gain)
            return context.rms_norm(x, gain, eps)
        y, total = context.rms_norm(x, gain, eps, residual=residual)
        ctx.save_for_backward(total, gain)
        return y, total

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, ds=None):
        context, eps = ctx.args
        s, gain = ctx.saved_tensors
        want_x, want_gain, want_residual = ctx.needs_input_grad[:3]
        dx = dgain = None
        if dy is None:
            dx = ds
            dgain = torch.zeros_like(gain) if want_gain else None
        else:
            dx, dgain = context.rms_norm_backward(dy, s, gain, eps, ds=ds,
                                                  want_dx=want_x or want_residual,
                                                  want_dgain=want_gain)
        return (dx if want_x else None, dgain, dx if want_residual else None, None, None)


def block_linear(context: Context, x: torch.Tensor, weight: BlockWeight) -> torch.Tensor:
    """x [..., cols] -> x W^T [..., rows] with W, and x within the call, in 8-bit blocks.  The
    gradient of x is dy W with dy in 8-bit blocks; x's own rounding is passed straight through."""
    y = _BlockLinear.apply(_rows(x), context, weight, None)
    return y.reshape(x.shape[:-1] + (weight.rows,))


def block_grouped_linear(context: Context, x: torch.Tensor, weight: BlockWeight,
                         offsets: torch.Tensor) -> torch.Tensor:
    """x [n, cols], sorted by group (expert) -> [n, rows]; offsets int32 [groups + 1]."""
    return _BlockLinear.apply(x, context, weight, offsets)


def rms_norm(context: Context, x: torch.Tensor, gain: torch.Tensor, eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None):
    """Root-mean-square norm of s = x + residual over the last dimension, times gain: y, or
    (y, s) with a residual.  Differentiable in x, gain and the residual."""
    if residual is None:
        return _RmsNorm.apply(_rows(x), gain, None, context, eps).reshape(x.shape)
    if residual.shape != x.shape:
        raise ValueError("residual must have shape %s, got %s" %
                         (tuple(x.shape), tuple(residual.shape)))
    y, total = _RmsNorm.apply(_rows(x), gain, _rows(residual), context, eps)
    return y.reshape(x.shape), total.reshape(x.shape)
