"""A mixture of experts around the 4-bit experts' products: routing, the exchange of rows
with the experts and the whole layer.

  weights, experts = route(logits, k)          which experts, with which weights
  plan = ops.expert_plan(experts, n)           the slots' order by expert, offsets on the device
  xs = dispatch(x, plan)                       rows sorted by expert, for FP4Experts with plan.offsets
  y = combine(ys, plan, weights, add=x)        weighted sums back, and what they are added to

``route``, ``dispatch`` and ``combine`` are ``ops``' calls of those names with gradients;
nothing waits for the device. ``FP4MoE`` puts a layer norm, a router and two layers of 4-bit
experts around them.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import fp4, norm, ops


class _RouteFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, bias, score, groups, kept, group_best, renormalise, scale):
        weights, experts = ops.route(logits, k, bias, score, groups, kept, group_best, renormalise, scale)
        ctx.save_for_backward(logits, experts)
        ctx.how = (score, renormalise, scale)
        ctx.mark_non_differentiable(experts)
        return weights, experts

    @staticmethod
    @once_differentiable
    def backward(ctx, dweights, _):
        logits, experts = ctx.saved_tensors
        return (ops.route_backward(dweights.contiguous(), logits, experts, *ctx.how), *(None,) * 8)


def route(logits: torch.Tensor, k: int, bias: torch.Tensor | None = None, score: str = "softmax", groups: int = 1,
          kept: int = 1, group_best: int = 1, renormalise: bool = True, scale: float = 1.0):
    """``ops.route`` with the weights differentiable once in the logits."""
    ops._refuse_forward_mode("route", logits)
    if torch.is_grad_enabled() and logits.requires_grad:
        return _RouteFn.apply(logits, k, bias, score, groups, kept, group_best, renormalise, scale)
    return ops.route(logits, k, bias, score, groups, kept, group_best, renormalise, scale)


def _tables(plan: ops.ExpertPlan) -> tuple[torch.Tensor, ...]:
    """A plan's tables as autograd can save them (ExpertPlan(*tables) is the plan again)."""
    return tuple(t.clone() if t.is_inference() else t for t in (plan.offsets, plan.rows))


class _DispatchFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.save_for_backward(*_tables(plan))
        return ops.expert_dispatch(x, plan)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        return ops.expert_combine(dxs, ops.ExpertPlan(*ctx.saved_tensors)), None


def dispatch(x: torch.Tensor, plan: ops.ExpertPlan) -> torch.Tensor:
    """``ops.expert_dispatch``, differentiable once in x."""
    ops._refuse_forward_mode("dispatch", x)
    if torch.is_grad_enabled() and x.requires_grad:
        return _DispatchFn.apply(x, plan)
    return ops.expert_dispatch(x, plan)


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, plan, weights, add):
        ctx.save_for_backward(ys, weights, *_tables(plan))
        return ops.expert_combine(ys, plan, weights, add)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ys, weights, *tables = ctx.saved_tensors
        need_ys, _, need_w, need_add = ctx.needs_input_grad
        dys = dw = None
        if need_ys and weights is None:
            dys = ops.expert_dispatch(dy, ops.ExpertPlan(*tables))
        elif need_ys or need_w:
            dys, dw = ops.expert_combine_backward(dy, ys, ops.ExpertPlan(*tables), weights)
        return dys if need_ys else None, None, dw if need_w else None, dy if need_add else None


def combine(ys: torch.Tensor, plan: ops.ExpertPlan, weights: torch.Tensor | None = None, add: torch.Tensor | None = None) -> torch.Tensor:
    """``ops.expert_combine``, differentiable once in ys, weights and add."""
    ops._refuse_forward_mode("combine", ys, weights, add)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (ys, weights, add)):
        return _CombineFn.apply(ys, plan, weights, add)
    return ops.expert_combine(ys, plan, weights, add)


class Router(torch.nn.Module):
    """Scores of every token for every expert, and the k it goes to.

    The scores' products are torch's in fp32, under autocast too, and so are their weights unless
    the module is cast. (Where the process lets fp32 products be TF32, by
    torch.set_float32_matmul_precision, these are, and the choices follow them.) With
    ``balance`` the buffer ``bias`` ([experts], zero at first; keep it in fp32, whose steps
    are finer than ``balance_step``'s) is added to the scores that choose, not to the
    weights; ``balance_step`` moves it against the load of a batch. The other arguments
    are ``ops.route``'s."""

    def __init__(self, features: int, experts: int, k: int, balance: bool = False, device=None, score: str = "softmax",
                 groups: int = 1, kept: int = 1, group_best: int = 1, renormalise: bool = True, scale: float = 1.0):
        super().__init__()
        if not 1 <= k <= experts:
            raise ValueError("k must be between 1 and the number of experts")
        if score not in ops.SCORES:
            raise ValueError(f"score must be one of {', '.join(ops.SCORES)}")
        if groups < 1 or experts % groups or not 1 <= kept <= groups or group_best not in (1, 2):
            raise ValueError("groups must divide the experts, kept be between 1 and groups, group_best 1 or 2")
        self.features, self.experts, self.k = features, experts, k
        self.how = dict(score=score, groups=groups, kept=kept, group_best=group_best, renormalise=renormalise, scale=scale)
        self.weight = torch.nn.Parameter(torch.empty((experts, features), device=device))
        torch.nn.init.normal_(self.weight, std=features ** -0.5)
        self.register_buffer("bias", torch.zeros(experts, device=device) if balance else None)

    def forward(self, x: torch.Tensor):
        """x [tokens, features] -> (weights fp32 [tokens, k], experts int32 [tokens, k])."""
        if x.dim() != 2 or x.shape[1] != self.features:
            raise ValueError(f"expected [tokens, {self.features}], got {tuple(x.shape)}")
        bias = None if self.bias is None else self.bias.float()
        with torch.autocast(x.device.type, enabled=False):
            logits = torch.nn.functional.linear(x.float(), self.weight.float())
        return route(logits, self.k, bias, **self.how)

    @torch.no_grad()
    def balance_step(self, plan: ops.ExpertPlan, rate: float = 1e-3) -> None:
        """bias += rate for experts with fewer rows than the mean, -= rate for those with more."""
        if self.bias is None:
            raise ValueError("the router was made without balance=True")
        load = plan.offsets.diff().float()
        self.bias += (rate * torch.sign(load.mean() - load)).to(self.bias.dtype)


class FP4MoE(torch.nn.Module):
    """A layer of 4-bit experts with all that stands around them:

      h = LayerNorm(x);  weights, experts = Router(h)
      y = x + sum over a token's experts of weight * down(silu(gate(h)) * up(h))

    gate and up are one FP4Experts layer [experts, 2 hidden, features], down is another;
    ``accumulate_main_grad`` is theirs. Further arguments are the Router's. ``plan`` is the
    last batch's, for ``router.balance_step``."""

    def __init__(self, features: int, hidden: int, experts: int, k: int, fmt: int = ops.FP4_NV, device=None,
                 dtype=torch.bfloat16, accumulate_main_grad: bool = False, eps: float = 1e-5, **router):
        super().__init__()
        self.norm = norm.LayerNorm(features, eps, device=device, dtype=torch.bfloat16)
        self.router = Router(features, experts, k, device=device, **router)
        self.up = fp4.FP4Experts(experts, features, 2 * hidden, fmt, device, dtype, accumulate_main_grad)
        self.down = fp4.FP4Experts(experts, hidden, features, fmt, device, dtype, accumulate_main_grad)
        self.plan = None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """x [..., features] bf16 -> the same shape."""
        if x.dtype != torch.bfloat16:
            raise TypeError(f"x must be bfloat16, got {x.dtype}")
        x2 = x.reshape(-1, x.shape[-1])
        h = self.norm(x2)
        weights, experts = self.router(h)
        plan = self.plan = ops.expert_plan(experts, self.router.experts)
        gate, up = self.up(dispatch(h, plan), plan.offsets).chunk(2, dim=-1)
        ys = self.down(torch.nn.functional.silu(gate) * up, plan.offsets)
        return combine(ys, plan, weights, x2).reshape(x.shape)
