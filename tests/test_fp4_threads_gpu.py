"""A 4-bit layer shared by threads, each on a stream of its own."""
import threading

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


def test_threads_on_streams_of_their_own(fp4):
    """Threads share a layer whose casts are dropped again and again, each behind work of its own stream."""
    x, w = acts(20, 512, seed=1), acts(1024, 512, seed=2)
    layer = fp4.FP4Linear(512, 1024, device="cuda")
    with torch.no_grad():
        layer.weight.copy_(w)
    want = fp4.forward(x, fp4.FP4Weight(w), "own")
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(i):
        try:
            big = torch.randn((1024, 1024), device="cuda")
            with torch.cuda.stream(torch.cuda.Stream()), torch.no_grad():
                for n in range(60):
                    if n % 4 == i:
                        layer.forget_casts()
                        big = big @ big * 1e-2
                    if not torch.equal(layer(x), want):
                        wrong.append((i, n))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and not wrong
