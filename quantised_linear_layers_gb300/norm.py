"""Layer norm: over the last axis, in fp32 from bf16 or fp32, rounded once.

``LayerNorm`` is the module, ``layer_norm`` the function behind it; both go through
``ops.layer_norm`` and, with gradients, ``ops.layer_norm_saving`` and
``ops.layer_norm_backward``, which makes the gradients of x, weight and bias from one read
of x and dy.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import ops


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, dtype):
        y, stats = ops.layer_norm_saving(x, weight, bias, eps, dtype=dtype)
        ctx.save_for_backward(x, stats, weight)
        ctx.types = (None if weight is None else weight.dtype, None if bias is None else bias.dtype)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, stats, weight = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        dx, dw, db = ops.layer_norm_backward(dy, x, stats, weight, sums=need_w or need_b)
        return (dx if need_x else None, dw.to(ctx.types[0]) if need_w else None, db.to(ctx.types[1]) if need_b else None,
                None, None)


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, eps: float = 1e-5,
               dtype: torch.dtype | None = None) -> torch.Tensor:
    """(x - mean) / sqrt(var + eps) * weight + bias over the last axis of x (bf16 or
    fp32), of ``dtype`` (default: x's). Differentiable once in x, weight and bias."""
    ops._refuse_forward_mode("layer_norm", x, weight, bias)
    x2 = x.reshape(x.shape[:-1].numel(), x.shape[-1])                  # (no -1: rows may have no columns)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias)):
        y = _LayerNormFn.apply(x2, weight, bias, eps, dtype)
    else:
        y = ops.layer_norm(x2, weight, bias, eps, dtype=dtype)
    return y.reshape(x.shape)


class LayerNorm(torch.nn.Module):
    """nn.LayerNorm over the last axis, with parameters in fp32 (``param_dtype``) whatever
    x is; ``dtype`` is that of the result (default: x's)."""

    def __init__(self, features: int, eps: float = 1e-5, affine: bool = True, bias: bool = True, device=None,
                 dtype: torch.dtype | None = None, param_dtype: torch.dtype = torch.float32):
        super().__init__()
        self.features, self.eps, self.dtype = features, eps, dtype
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=param_dtype)) if affine else None
        self.bias = torch.nn.Parameter(torch.zeros(features, device=device, dtype=param_dtype)) if affine and bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.features:
            raise ValueError(f"expected {self.features} features, got {x.shape[-1]}")
        return layer_norm(x, self.weight, self.bias, self.eps, self.dtype)
