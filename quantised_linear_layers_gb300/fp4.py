"""4-bit linear layers: forward, dgrad and wgrad over microscaled E2M1 casts
and products, for one weight and for experts with ragged loads.

The microscaled formats and layouts are those of include/qlinear.h. As in the
FP8 layer (linear.py), every operand is cast along the axis that its product
sums over:

  fwd    Y  = X  W^T  : X and W cast along the input features
  dgrad  dX = dY W    : dY and W^T cast along the output features
  wgrad  dW = dY^T X  : dY^T and X^T cast along the tokens, fp32 output,
                        optionally accumulated

The tensor core takes 4-bit operands with the summed axis contiguous only, so W,
X and dY are each cast both ways from one read. Gradients pass straight through
the rounding: they are those of the product of the cast operands. Experts
(``FP4ExpertWeight``, ``experts_*``): tokens sorted by expert with int32
``offsets`` on the device; loads may be anything, zero included. Rows before the
first and after the last expert's, as in a batch padded to a fixed capacity, have
no influence on any result and are zero in Y and dX (unwritten in a given ``out``).

FP4_NV casts of a training step use the tensor's own scale
(``ops.fp4_tensor_scale``; with experts, that of the rows they have). A
forward-only call takes X's scale as given, 1 by default: group scales then span
2^-9 .. 448, the range of normalised activations, and X is read once. The modules
take X's own scale with and without gradients.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import ops


def _own(fmt: int):
    """The scale of a training step's casts."""
    return ops.FP4_OWN_SCALE if fmt == ops.FP4_NV else None


class FP4Weight:
    """A weight W [out, in] in 4 bits: ``w`` (forward) and, with ``dgrad``, ``wt``
    (the cast of W^T, for the data gradient)."""

    _dims = 2

    def __init__(self, w: torch.Tensor, fmt: int = ops.FP4_NV, dgrad: bool = True):
        self.fmt = fmt
        self.dgrad = dgrad
        self.update(w)

    def update(self, w: torch.Tensor) -> None:
        self.shape = tuple(w.shape)
        if len(self.shape) != self._dims:
            raise ValueError("weight must be 2-D [out_features, in_features]" if self._dims == 2 else
                             "weight must be 3-D [experts, out_features, in_features]")
        if not w.is_contiguous() and ((w.stride(-1) != 1 and self.shape[-1] > 1) or
                                      (self._dims == 3 and w.stride(0) != self.shape[1] * w.stride(1))):
            w = w.contiguous()
        scale = _own(self.fmt)
        if self.dgrad:
            self.w, self.wt = ops.fp4_cast_dual(w, self.fmt, scale)
        else:
            self.w, self.wt = ops.fp4_cast(w, self.fmt, scale), None


class FP4ExpertWeight(FP4Weight):
    """The weights W [experts, out, in] of a layer of experts in 4 bits."""

    _dims = 3


def _need_wt(w: FP4Weight) -> ops.FP4Tensor:
    if w.wt is None:
        raise ValueError("the weight was cast without dgrad=True")
    return w.wt


def forward(x: torch.Tensor, w: FP4Weight, x_scale: torch.Tensor | None = None,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """Y [T, out] = X [T, in] W^T (bf16)."""
    return ops.fp4_linear(x, w.w, x_scale, out=out)


def forward_saving(x: torch.Tensor, w: FP4Weight):
    """Y = X W^T plus X's cast along the tokens for the weight gradient: (Y, cast)."""
    return ops.fp4_linear_saving(x, w.w, _own(w.fmt))


def backward(dy: torch.Tensor, w: FP4Weight, x_cols: ops.FP4Tensor, need_dx: bool = True,
             dw_out: torch.Tensor | None = None, accumulate: bool = False):
    """dX = dY W (bf16, or None) and dW (+)= dY^T X (fp32) with dY cast both ways
    from one read and x_cols from ``forward_saving``."""
    return ops.fp4_linear_backward(dy, _need_wt(w) if need_dx else None, x_cols, _own(w.fmt), None, dw_out, accumulate)


def dgrad(dy: torch.Tensor, w: FP4Weight, out: torch.Tensor | None = None) -> torch.Tensor:
    """dX [T, in] = dY [T, out] W (bf16)."""
    return ops.fp4_linear(dy, _need_wt(w), _own(w.fmt), out=out)


def experts_forward(x: torch.Tensor, offsets: torch.Tensor, w: FP4ExpertWeight, x_scale: torch.Tensor | None = None,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """Y [T, out]: rows offsets[e] .. offsets[e+1] of X [T, in] times W[e]^T (bf16)."""
    return ops.fp4_linear(x, w.w, x_scale, offsets, out=out)


def experts_forward_saving(x: torch.Tensor, offsets: torch.Tensor, w: FP4ExpertWeight):
    """experts_forward plus X's cast along each expert's tokens: (Y, cast)."""
    return ops.fp4_linear_saving(x, w.w, _own(w.fmt), offsets)


def experts_backward(dy: torch.Tensor, offsets: torch.Tensor, w: FP4ExpertWeight, x_cols: ops.FP4Tensor,
                     need_dx: bool = True, dw_out: torch.Tensor | None = None, accumulate: bool = False):
    """dX [T, in] (bf16, or None) and dW [experts, out, in] (+)= dY_e^T X_e (fp32)."""
    return ops.fp4_linear_backward(dy, _need_wt(w) if need_dx else None, x_cols, _own(w.fmt), offsets, dw_out,
                                   accumulate)


def _forward(x, offsets, w4):
    """A module's forward without a backward: X under its own scale, as in training."""
    scale = _own(w4.fmt)
    return forward(x, w4, scale) if offsets is None else experts_forward(x, offsets, w4, scale)


class _FP4Fn(torch.autograd.Function):
    """Both layers' autograd: offsets is None for the plain one."""

    @staticmethod
    def forward(ctx, x, weight, w4, offsets, module):
        ctx.w4, ctx.module, ctx.x_dtype = w4, module, x.dtype
        if not ctx.needs_input_grad[1]:
            ctx.save_for_backward(offsets)
            ctx.x_cols = None
            return _forward(x, offsets, w4)
        y, cols = forward_saving(x, w4) if offsets is None else experts_forward_saving(x, offsets, w4)
        ctx.save_for_backward(offsets, cols.buf)
        ctx.x_cols = (cols.ld, cols._scale, cols.fmt, cols.batch, cols.rows, cols.cols)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        w4, module = ctx.w4, ctx.module
        offsets = ctx.saved_tensors[0]
        dy = dy.contiguous()
        if ctx.x_cols is None:
            if not ctx.needs_input_grad[0]:
                return None, None, None, None, None
            if offsets is None:
                dx = dgrad(dy, w4)
            else:
                dx = ops.fp4_linear(dy, _need_wt(w4), _own(w4.fmt), offsets)
            return dx.to(ctx.x_dtype), None, None, None, None
        x_cols = ops.FP4Tensor(ctx.saved_tensors[1], *ctx.x_cols, offsets, offsets is not None)
        main = module.main_grad
        kw = dict(need_dx=ctx.needs_input_grad[0], dw_out=main, accumulate=main is not None)
        dx, dw = backward(dy, w4, x_cols, **kw) if offsets is None else experts_backward(dy, offsets, w4, x_cols, **kw)
        return (None if dx is None else dx.to(ctx.x_dtype), None if main is not None else dw.to(module.weight.dtype),
                None, None, None)


class FP4Linear(torch.nn.Module):
    """nn.Linear (no bias) whose fwd / dgrad / wgrad run through the 4-bit casts
    and products. With ``accumulate_main_grad`` the weight gradient is added into
    the fp32 buffer ``main_grad`` instead of being returned to autograd.

    The weight's casts are kept until the weight changes: by an in-place operation
    or by being given other storage. A write through ``weight.data`` shows in
    neither; call ``forget_casts`` after one. In a CUDA graph a training step casts
    the weight anew with every replay, and since replays may change the weight
    unseen, calls outside the graph keep no casts from then on; a forward without
    gradients uses the casts kept when it was captured, which live as long as the
    graph (their memory is free for others with the first cast after its end)."""

    _weight_type = FP4Weight

    def __init__(self, in_features: int, out_features: int, fmt: int = ops.FP4_NV, device=None,
                 dtype=torch.bfloat16, accumulate_main_grad: bool = False):
        super().__init__()
        self._init((out_features, in_features), fmt, device, dtype, accumulate_main_grad)

    def _init(self, shape, fmt, device, dtype, accumulate_main_grad):
        self.weight = torch.nn.Parameter(torch.empty(shape, device=device, dtype=dtype))
        torch.nn.init.normal_(self.weight, std=0.02)
        self.fmt = fmt
        self.main_grad = torch.zeros(shape, device=device, dtype=torch.float32) if accumulate_main_grad else None
        self._trained_in_graph = False
        self.forget_casts()

    def forget_casts(self) -> None:
        """Has the next forward cast the weight anew."""
        self._kept = None
        ops._drop_held()

    def __getstate__(self):
        # a copy makes casts of its own
        return {**self.__dict__, "_kept": None, "_trained_in_graph": False}

    def fp4_weight(self, dgrad: bool = True) -> FP4Weight:
        """The weight's casts, made anew when the weight has changed."""
        w = self.weight
        capturing = w.is_cuda and torch.cuda.is_current_stream_capturing()
        # (casts, version and storage of what was cast, stream and event behind the
        # casts): one object, set and read at once, since other threads do too. It keeps
        # the storage, so that no other can have its address.
        kept = self._kept
        if kept is not None:
            w4, version, of = kept[:3]
            if (self._trained_in_graph or (dgrad and not w4.dgrad) or version != w._version or
                    of.data_ptr() != w.data_ptr() or of.device != w.device or of.dtype != w.dtype):
                kept = None
        training = capturing and torch.is_grad_enabled() and w.requires_grad
        if training:
            self._trained_in_graph = True
        if training or (capturing and kept is None):
            return self._cast(dgrad)     # part of the graph: not for calls outside it
        if kept is None:
            ops._drop_held()
            version, of = w._version, w.detach()
            w4 = self._cast(dgrad)
            stream = torch.cuda.current_stream(w.device)
            self._kept = (w4, version, of, stream, stream.record_event())
        elif capturing:
            ops._hold_in_graph(w4, kept[4])  # the graph reads them, however often the weight changes
        else:
            stream = torch.cuda.current_stream(w.device)
            if stream != kept[3]:
                stream.wait_event(kept[4])
                for c in (w4.w, w4.wt):
                    if c is not None:
                        c.buf.record_stream(stream)
        return w4

    def _cast(self, dgrad: bool) -> FP4Weight:
        with torch.no_grad():
            return self._weight_type(self.weight.detach(), self.fmt, dgrad=dgrad)

    def _apply_layer(self, x: torch.Tensor, offsets: torch.Tensor | None) -> torch.Tensor:
        # without gradients the calls below go past autograd, which would refuse (the
        # level by itself first: 0.6 us a call less)
        if forward_ad._current_level >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in (x, self.weight)):
            raise NotImplementedError("4-bit layers have no forward-mode derivatives")
        if torch.is_grad_enabled() and (x.requires_grad or self.weight.requires_grad):
            return _FP4Fn.apply(x, self.weight, self.fp4_weight(), offsets, self)
        return _forward(x, offsets, self.fp4_weight(dgrad=False))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """x [..., in_features] -> [..., out_features] (bf16)."""
        if x.shape[-1] != self.weight.shape[1]:
            raise ValueError(f"expected {self.weight.shape[1]} input features, got {x.shape[-1]}")
        x2 = x.reshape(-1, x.shape[-1])
        y = self._apply_layer(x2, None)
        return y.reshape(*x.shape[:-1], y.shape[-1])


class FP4Experts(FP4Linear):
    """A layer of experts: ``weight`` [experts, out, in], tokens sorted by expert."""

    _weight_type = FP4ExpertWeight

    def __init__(self, experts: int, in_features: int, out_features: int, fmt: int = ops.FP4_NV, device=None,
                 dtype=torch.bfloat16, accumulate_main_grad: bool = False):
        torch.nn.Module.__init__(self)
        self._init((experts, out_features, in_features), fmt, device, dtype, accumulate_main_grad)

    def forward(self, x: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
        """x [T, in_features], offsets int32 [experts + 1] -> [T, out_features] (bf16)."""
        if x.dim() != 2 or x.shape[1] != self.weight.shape[2]:
            raise ValueError(f"expected [tokens, {self.weight.shape[2]}], got {tuple(x.shape)}")
        if offsets.shape[0] != self.weight.shape[0] + 1:
            raise ValueError(f"offsets must have {self.weight.shape[0] + 1} entries")
        return self._apply_layer(x, offsets)
