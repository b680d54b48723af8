"""4-bit layers refuse forward-mode derivatives, which they do not have, before
they touch the GPU."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from quantised_linear_layers_gb300 import fp4


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("which", ["x", "weight"])
@pytest.mark.parametrize("experts", [False, True])
def test_forward_mode_derivatives_are_refused(experts, which, grad):
    layer = fp4.FP4Experts(2, 8, 4) if experts else fp4.FP4Linear(8, 4)
    layer.weight.requires_grad_(False)
    x = torch.ones((3, 8), dtype=torch.bfloat16)
    args = (torch.tensor([0, 1, 3], dtype=torch.int32),) if experts else ()
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        if which == "x":
            x = forward_ad.make_dual(x, torch.ones_like(x))
        else:
            w = layer.weight.detach().clone()
            del layer.weight
            layer.weight = forward_ad.make_dual(w, torch.ones_like(w))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            layer(x, *args)
