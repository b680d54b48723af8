"""A small mixture of experts trained and then decoded in 4 bits.

The 4-bit layers as a model uses them: tokens are routed to one expert each,
sorted by expert and run through two layers of experts (FP4Experts, ragged
loads, offsets that stay on the device) and a shared projection (FP4Linear),
forward and backward in 4 bits with the weight gradients accumulated into fp32
main grads; then single tokens go through the same weights, each call one launch
per layer. Run: python examples/fp4_experts.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from quantised_linear_layers_gb300 import fp4, ops  # noqa: E402


class Block(torch.nn.Module):
    def __init__(self, dim: int, hidden: int, experts: int, fmt: int):
        super().__init__()
        self.router = torch.nn.Parameter(torch.randn(experts, dim, device="cuda") * 0.02)
        self.up = fp4.FP4Experts(experts, dim, hidden, fmt, device="cuda", accumulate_main_grad=True)
        self.down = fp4.FP4Experts(experts, hidden, dim, fmt, device="cuda", accumulate_main_grad=True)
        self.out = fp4.FP4Linear(dim, dim, fmt, device="cuda", accumulate_main_grad=True)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        score = torch.softmax(x.float() @ self.router.t(), dim=-1)
        gate, expert = score.max(dim=-1)
        order = torch.argsort(expert, stable=True)
        count = torch.bincount(expert, minlength=self.router.shape[0])
        offsets = torch.nn.functional.pad(count.cumsum(0), (1, 0)).to(torch.int32)
        h = torch.nn.functional.silu(self.up(x[order], offsets))
        y = self.down(h, offsets) * gate[order, None].to(x.dtype)
        back = torch.empty_like(order)
        back[order] = torch.arange(order.numel(), device=x.device)
        return self.out(x + y[back])


def train(fmt: int, steps: int, tokens: int = 2048, dim: int = 512, hidden: int = 1024, experts: int = 8, lr: float = 0.5):
    """Fits the block to a fixed random map; returns it and the loss of every step."""
    torch.manual_seed(0)
    block = Block(dim, hidden, experts, fmt)
    layers = [block.up, block.down, block.out]
    target = torch.randn(dim, dim, device="cuda") * dim ** -0.5
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, dim, device="cuda").bfloat16()
        loss = (block(x).float() - x.float() @ target).square().mean()
        loss.backward()
        with torch.no_grad():
            for layer in layers:                  # plain gradient steps, scaled to each weight's size
                g = layer.main_grad
                rms = g.square().mean().sqrt().clamp(min=1e-12)
                layer.weight -= (lr * 1e-2 * g / rms * layer.weight.float().square().mean().sqrt()).to(layer.weight.dtype)
                layer.main_grad.zero_()
            block.router -= 0.1 * block.router.grad
            block.router.grad = None
        losses.append(float(loss.detach()))
    return block, losses


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 150
    for name, fmt in (("nv", ops.FP4_NV), ("mx", ops.FP4_MX)):
        block, losses = train(fmt, steps)
        tokens = torch.randn(4, 512, device="cuda").bfloat16()
        with torch.no_grad():
            batch = block(tokens)
            singles = torch.cat([block(t[None]) for t in tokens])
        rel = float((singles.float() - batch.float()).norm() / batch.float().norm())
        assert ops.device_status() == 0
        print(f"{name}: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {steps} steps; "
              f"single tokens against the batch: {rel:.1e}")


if __name__ == "__main__":
    main()
