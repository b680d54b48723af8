"""Experts whose offsets leave rows out, as a batch padded to a fixed capacity
does: whatever such rows hold has no influence on any expert."""
import pytest
import torch

import fp4_reference as ref
from fp4_checks import acts, np64

pytestmark = pytest.mark.gpu

OFFSETS = [[3, 40, 40, 200], [0, 0, 5, 90], [2, 2, 5, 6], [0, 0, 0, 0], [7, 7, 7, 7], [1, 300, 301, 700]]
IDS = ["_".join(map(str, o)) for o in OFFSETS]
PADDING = [float("nan"), float("inf"), 1e30]


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantised_linear_layers_gb300 import build, ops as o
    build.build()
    o.load_library()
    return o


@pytest.fixture(autouse=True)
def clean(ops):
    yield
    ops.set_gemm_path(0)
    assert ops.device_status() == 0


def padded(x, offs, value):
    """x with `value` in the rows of no expert."""
    x = x.clone()
    x[:offs[0]], x[offs[-1]:] = value, value
    return x


@pytest.mark.parametrize("value", PADDING, ids=["nan", "inf", "large"])
@pytest.mark.parametrize("offs", OFFSETS, ids=IDS)
@pytest.mark.parametrize("form", ["even", "odd", "wide", "odd_wide"])
def test_own_scale_is_that_of_the_experts_rows(ops, offs, form, value):
    """Rows on 16-byte boundaries or anywhere, one after the other or apart."""
    m, k = offs[-1] + 9, 200 if form in ("even", "wide") else 203
    for dtype in (torch.bfloat16, torch.float32):
        big = padded(acts(m, k + 8 if "wide" in form else k, seed=1, dtype=dtype), offs, value)
        x = big[:, 8:] if form == "wide" else big[:, 3:k + 3] if form == "odd_wide" else big
        off = torch.tensor(offs, dtype=torch.int32, device="cuda")
        want = ref.tensor_scale(np64(x)[offs[0]:offs[-1]])
        a = ops.fp4_cast(x, 0, ops.FP4_OWN_SCALE, off)
        assert float(a.scale) == want
        for c in ops.fp4_cast_dual(x, 0, ops.FP4_OWN_SCALE, off):
            assert float(c.scale) == want


def test_own_scale_of_many_rows(ops):
    """Above the size that one cluster takes."""
    for dtype, k in ((torch.bfloat16, 1024), (torch.bfloat16, 1023), (torch.float32, 1023)):
        x = acts(3000, k, seed=2, dtype=dtype)
        off = torch.tensor([5, 700, 700, 2990], dtype=torch.int32, device="cuda")
        for value in PADDING:
            y = padded(x, [5, 2990], value)
            assert float(ops.fp4_cast(y, 0, ops.FP4_OWN_SCALE, off).scale) == ref.tensor_scale(np64(x)[5:2990])
        none = torch.full((4,), 8, dtype=torch.int32, device="cuda")
        assert float(ops.fp4_cast(x, 0, ops.FP4_OWN_SCALE, none).scale) == 2.0 ** -80
