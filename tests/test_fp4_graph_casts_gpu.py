"""How long captured graphs keep the casts of a 4-bit layer that they read."""
import gc
import time
import weakref

import pytest
import torch

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


def test_casts_live_as_long_as_the_graphs_that_read_them(fp4):
    x = acts(5, 96, seed=1)
    layer = fp4.FP4Linear(96, 48, device="cuda")
    graphs, outs, wants, casts = [], [], [], []
    with torch.no_grad():
        for seed in range(3):
            layer.weight.copy_(acts(48, 96, seed=seed))
            wants.append(layer(x).clone())
            casts.append(weakref.ref(layer.fp4_weight(dgrad=False)))
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                outs.append((layer(x), layer(x)))
        layer.forget_casts()
        layer.weight.copy_(acts(48, 96, seed=9))
        layer(x)
        gc.collect()
        assert all(c() is not None for c in casts)
        junk = [torch.full((4096,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
        for g, out, want in zip(graphs, outs, wants):
            g.replay()
            assert torch.equal(out[0], want) and torch.equal(out[1], want)
        del junk, g
        torch.cuda.synchronize()
        # the graphs go one by one, and each takes its own casts with it
        for i in (1, 0, 2):
            graphs[i].reset()
            end = time.monotonic() + 20
            while casts[i]() is not None and time.monotonic() < end:
                layer.forget_casts()
                layer(x)
                time.sleep(0.01)
            assert casts[i]() is None
            left = [j for j in {1: (0, 2), 0: (2,), 2: ()}[i]]
            assert all(casts[j]() is not None for j in left)
            for j in left:
                graphs[j].replay()
                assert torch.equal(outs[j][0], wants[j])
