"""Differentiable layers over the layer operators: ``layer_norm`` and
``linear`` for models whose parameters ``HybridMuonAdamW`` steps.

What they keep for the backward pass is a checkpoint in 8 bits where asked
for: the norm's input, the linear layer's input.  Norm, checkpoints and weight
gradients run in the library's kernels; the forward product ``x W^T`` and the
input gradient ``dy W`` are PyTorch's plain matrix products.  Both run outside
autocast, in the types of their arguments.

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


def linear(x, W, keep: Union[str, ActCheckpoint] = "e4m3"):
    """``x W^T`` for x [..., cols] and a 2-D weight W [rows, cols] of the same
    type, keeping x for the weight gradient in 8 bits: in the format ``keep``,
    or as the checkpoint of x given (one that :func:`layer_norm` returned)."""
    if W.ndim != 2:
        raise ValueError(f"W must be 2-D, it has {W.ndim} dims")
    if x.dtype != W.dtype:
        raise TypeError(f"x has dtype {x.dtype}, W {W.dtype}")
    if x.shape[-1] != W.shape[1]:
        raise ValueError(f"x has {x.shape[-1]} columns, W {W.shape[1]}")
    if not (torch.is_grad_enabled() and W.requires_grad):
        return _product(x, W.t())      # no weight gradient: nothing is kept
    if isinstance(keep, ActCheckpoint):
        if keep.shape != (x.numel() // max(1, x.shape[-1]), x.shape[-1]) or keep.device != x.device:
            raise ValueError(f"keep is {keep}, x has shape {tuple(x.shape)} on {x.device}")
    else:
        keep = checkpoint_save(_rows(x.detach()), keep)
    return _Linear.apply(x, W, keep.q, keep.scale)
