"""A forward captured at once after casts that another stream is still to make."""
import pytest
import torch

from fp4_checks import acts

pytestmark = pytest.mark.gpu


def test_capture_behind_casts_of_another_stream():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantised_linear_layers_gb300 import build, fp4, ops
    build.build()
    ops.load_library()
    x, w = acts(20, 1024, seed=1), acts(2048, 1024, seed=2)
    layer = fp4.FP4Linear(1024, 2048, device="cuda")
    with torch.no_grad():
        layer.weight.copy_(w)
        want = fp4.forward(x, fp4.FP4Weight(w), "own")
        big = torch.randn((4096, 4096), device="cuda")
        made, used = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(used):
            layer(x)                                     # what the call needs once is there before the capture
        layer.forget_casts()
        big @ big
        torch.cuda.synchronize()
        with torch.cuda.stream(made):
            for _ in range(20):
                big = big @ big * 1e-3
            layer(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(used):
            graph.capture_begin()
            out = layer(x)
            graph.capture_end()
            graph.replay()
            got = out.clone()
        torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert ops.device_status() == 0
