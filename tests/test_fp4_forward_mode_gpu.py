"""4-bit layers refuse forward-mode derivatives, which they do not have."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from fp4_checks import acts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp4():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantised_linear_layers_gb300 import build, fp4 as f, ops as o
    build.build()
    o.load_library()
    return f


def test_forward_mode_derivatives_are_refused(fp4):
    layer = fp4.FP4Linear(64, 32, device="cuda")
    layer.weight.requires_grad_(False)
    x = acts(4, 64, seed=1)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for grad in (False, True):
            with torch.set_grad_enabled(grad), pytest.raises(NotImplementedError):
                layer(dual)
        assert layer(x).shape == (4, 32)
    with pytest.raises((RuntimeError, NotImplementedError)):
        torch.func.jvp(layer, (x,), (torch.ones_like(x),))
