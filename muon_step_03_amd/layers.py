"""Differentiable layers over the layer operators: ``layer_norm``, ``linear`` and
``expert_linear`` for models whose parameters ``HybridMuonAdamW`` steps.

What they keep for the backward pass is a checkpoint in 8 bits where asked
for: the norm's input, the linear layers' input.  Norm, checkpoints, weight
gradients, the products of experts and all products in 8 bits run in the
library's kernels; the products of ``linear`` in the tensors' own type are
PyTorch's plain matrix products.  All run outside autocast, in the types of
their arguments.  What runs in the library has no forward-mode derivative: a
tangent that reaches it raises.

A backward pass may be captured into a graph when the forward pass it belongs
to is captured with it and no other autograd graph of the same parameters is
alive, as for any PyTorch layer.
"""
from __future__ import annotations

import math
from typing import Optional, Union

import torch
from torch.autograd.function import once_differentiable

from .layer_ops import (ActCheckpoint, checkpoint_save, layernorm_backward, layernorm_forward,
                        weight_grad)
from .linear_ops import Weight8, linear_forward, linear_input_grad, weight_quantize


def _rows(t: torch.Tensor) -> torch.Tensor:
    """[..., cols] as [tokens, cols] with unit column stride; a copy only where
    no view is one."""
    t = t.reshape(-1, t.shape[-1]) if t.ndim != 2 else t
    ok = t.shape[1] <= 1 or t.stride(1) == 1
    return t if ok and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1]) else t.contiguous()


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gain, bias, eps, keep, y_keep):
        rows = _rows(x)
        out = layernorm_forward(rows, gain, bias, eps=eps, x_checkpoint=keep, y_checkpoint=y_keep)
        kept = (rows,) if keep is None else (out.x_checkpoint.q, out.x_checkpoint.scale)
        ctx.save_for_backward(gain, out.mean, out.rstd, *kept)
        ctx.set_materialize_grads(False)      # no zeros for the checkpoint's outputs
        ctx.has_bias = bias is not None
        ctx.shape = x.shape
        y_kept = (None, None) if y_keep is None else (out.y_checkpoint.q, out.y_checkpoint.scale)
        if y_keep is not None:
            ctx.mark_non_differentiable(*y_kept)
        return out.y.view(x.shape), *y_kept

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, _q, _scale):
        if dy is None:
            return (None,) * 6
        gain, mean, rstd, *kept = ctx.saved_tensors
        x = kept[0] if len(kept) == 1 else ActCheckpoint(*kept, ctx.shape[-1])
        dx, dgain, dbias = layernorm_backward(_rows(dy), x, gain, mean, rstd, bias=ctx.has_bias)
        return dx.view(ctx.shape), dgain, dbias, None, None, None


def layer_norm(x, gain, bias=None, *, eps=1e-5, keep: Optional[str] = None,
               y_keep: Optional[str] = None):
    """Layer norm over the last dimension of ``x`` [..., cols].

    keep: "e4m3" or "int8" keeps x for the backward pass in 8 bits, None as it
    is.  y_keep: a format also returns the checkpoint of y, which every
    :func:`linear` that reads y can share: ``y, ck = layer_norm(...)``.
    """
    if not (torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                            for t in (x, gain, bias))):
        keep = None      # no backward pass will read it
    y, q, scale = _LayerNorm.apply(x, gain, bias, float(eps), keep, y_keep)
    return y if y_keep is None else (y, ActCheckpoint(q, scale, x.shape[-1]))


def _product(x, B):
    """x [..., n] times a matrix B: one product of two matrices.  (``x @ B`` is
    one over batches, each with an expanded B, where x's leading dimensions do
    not fold.)"""
    with torch.autocast(device_type=x.device.type, enabled=False):
        rows = x.reshape(math.prod(x.shape[:-1]), x.shape[-1])
        return (rows @ B).view(*x.shape[:-1], B.shape[1])


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, q, scale):
        ctx.save_for_backward(W, q, scale)
        return _product(x, W.t())

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        W, q, scale = ctx.saved_tensors
        dx = dW = None
        if ctx.needs_input_grad[0]:
            dx = _product(dy, W)
        if ctx.needs_input_grad[1]:
            dW = weight_grad(_rows(dy), ActCheckpoint(q, scale, W.shape[1]), dtype=W.dtype)
        return dx, dW, None, None


class _ExpertLinear(torch.autograd.Function):
    """x [tokens, cols] by the experts' weights in x's own type."""

    @staticmethod
    def forward(ctx, x, W, offsets, q, scale):
        ctx.save_for_backward(W, offsets, q, scale)
        return linear_forward(_rows(x), W, offsets=offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        W, offsets, q, scale = ctx.saved_tensors
        dx = dW = None
        dy = _rows(dy)
        if ctx.needs_input_grad[0]:
            dx = linear_input_grad(dy, W, offsets=offsets)
        if ctx.needs_input_grad[1]:
            dW = weight_grad(dy, ActCheckpoint(q, scale, W.shape[2]), offsets=offsets, dtype=W.dtype)
        return dx, dW, None, None, None


class _Linear8(torch.autograd.Function):
    """Both products from 8 bits, dense or per expert; x and W only carry the
    gradients, which pass the rounding as if it were not there."""

    @staticmethod
    def forward(ctx, x, W, offsets, q, scale, wq, wq_t, ws):
        ctx.save_for_backward(offsets, q, scale, wq, wq_t, ws)
        ctx.shape, ctx.dtypes = x.shape, (x.dtype, W.dtype)
        y = linear_forward(ActCheckpoint(q, scale, x.shape[-1]), Weight8(wq, wq_t, ws), offsets=offsets,
                           dtype=x.dtype)
        return y.view(*x.shape[:-1], y.shape[1])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        offsets, q, scale, *w8 = ctx.saved_tensors
        dx = dW = None
        dy = _rows(dy)
        if ctx.needs_input_grad[0]:
            dx = linear_input_grad(checkpoint_save(dy, "e4m3"), Weight8(*w8), offsets=offsets,
                                   dtype=ctx.dtypes[0]).view(ctx.shape)
        if ctx.needs_input_grad[1]:
            dW = weight_grad(dy, ActCheckpoint(q, scale, ctx.shape[-1]), offsets=offsets,
                             dtype=ctx.dtypes[1])
        return dx, dW, *(None,) * 6


def _check_keep(keep, x, products):
    """The checkpoint of x that ``keep`` gives or names."""
    if isinstance(keep, ActCheckpoint):
        if keep.shape != (x.numel() // max(1, x.shape[-1]), x.shape[-1]) or keep.device != x.device:
            raise ValueError(f"keep is {keep}, x has shape {tuple(x.shape)} on {x.device}")
    if products is not None and (keep.format if isinstance(keep, ActCheckpoint) else keep) != "e4m3":
        raise ValueError("products in 8 bits read the checkpoint of x: keep must be e4m3")
    return keep if isinstance(keep, ActCheckpoint) else checkpoint_save(_rows(x.detach()), keep)


def _check_products(products, W):
    """The 8-bit weight that ``products`` gives or asks for."""
    if isinstance(products, Weight8):
        if products.shape != tuple(W.shape) or products.device != W.device:
            raise ValueError(f"products is {products}, W has shape {tuple(W.shape)} on {W.device}")
        return products
    if products != "e4m3":
        raise ValueError(f"products must be None, 'e4m3' or a Weight8, not {products!r}")
    return weight_quantize(W.detach().contiguous())


def _linear8(x, W, offsets, keep, products):
    ck, w8 = _check_keep(keep, x, products), _check_products(products, W)
    return _Linear8.apply(x, W, offsets, ck.q, ck.scale, w8.q, w8.q_t, w8.scale)


def linear(x, W, keep: Union[str, ActCheckpoint] = "e4m3", *,
           products: Union[None, str, Weight8] = None):
    """``x W^T`` for x [..., cols] and a 2-D weight W [rows, cols] of the same
    type, keeping x for the weight gradient in 8 bits: in the format ``keep``,
    or as the checkpoint of x given (one that :func:`layer_norm` returned).

    products: None multiplies x and W as they are.  "e4m3" multiplies the
    checkpoint of x with W in 8 bits (scales for 32 columns and for 128 x 128
    elements), and in the backward pass dy, in 8 bits too, with the same W; a
    :class:`Weight8` of W, made once after each optimizer step, spares the
    micro-batches the quantizing.  With bfloat16 x the sums hold fewer bits than
    float32 (see :func:`linear_forward`), with float32 x they do not."""
    if W.ndim != 2:
        raise ValueError(f"W must be 2-D, it has {W.ndim} dims")
    if x.dtype != W.dtype:
        raise TypeError(f"x has dtype {x.dtype}, W {W.dtype}")
    if x.shape[-1] != W.shape[1]:
        raise ValueError(f"x has {x.shape[-1]} columns, W {W.shape[1]}")
    if products is not None:
        return _linear8(x, W, None, keep, products)
    if not (torch.is_grad_enabled() and W.requires_grad):
        return _product(x, W.t())      # no weight gradient: nothing is kept
    keep = _check_keep(keep, x, None)
    return _Linear.apply(x, W, keep.q, keep.scale)


def expert_linear(x, W, offsets, keep: Union[str, ActCheckpoint] = "e4m3", *,
                  products: Union[None, str, Weight8] = None):
    """``x[t] W[e]^T`` for x [tokens, cols] and the experts' weights W [count,
    rows, cols] of the same type; the tokens [offsets[e], offsets[e + 1]) are
    expert e's (offsets: int64 GPU tensor of count + 1 running totals, read on
    the device only).  Tokens of no expert give zeros and get zero gradients.
    A W that is not contiguous is copied in each call.
    keep, products: as for :func:`linear`."""
    if x.ndim != 2 or W.ndim != 3:
        raise ValueError(f"x must be [tokens, cols] and W [count, rows, cols], not {tuple(x.shape)} "
                         f"and {tuple(W.shape)}")
    if x.dtype != W.dtype:
        raise TypeError(f"x has dtype {x.dtype}, W {W.dtype}")
    if x.shape[1] != W.shape[2]:
        raise ValueError(f"x has {x.shape[1]} columns, W {W.shape[2]}")
    if products is not None:
        return _linear8(x, W, offsets, keep, products)
    W = W.contiguous()
    q = scale = None
    if torch.is_grad_enabled() and W.requires_grad:
        keep = _check_keep(keep, x, None)
        q, scale = keep.q, keep.scale
    return _ExpertLinear.apply(x, W, offsets, q, scale)
