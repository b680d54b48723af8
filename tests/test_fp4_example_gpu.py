"""The example of the 4-bit layers trains: its loss falls in both formats."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
def test_example_trains_and_decodes(fmt):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantised_linear_layers_gb300 import build, ops
    build.build()
    spec = importlib.util.spec_from_file_location("fp4_experts", os.path.join(ROOT, "examples", "fp4_experts.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    block, losses = example.train(fmt, 60)
    assert ops.device_status() == 0
    assert sum(losses[-5:]) < 0.9 * sum(losses[:5])
    with torch.no_grad():
        y = block(torch.randn(1, 512, device="cuda").bfloat16())
    assert y.shape == (1, 512) and bool(torch.isfinite(y).all())
