"""Scale bytes of groups past the last are zero in every cast, as the layout says."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
from fp4_checks import acts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantised_linear_layers_gb300 import build, ops as o
    build.build()
    o.load_library()
    return o


def scale_bytes(a, kcols):
    """[rows, groups with those past the last of kcols] of one cast's scale blocks."""
    words = -(-kcols // (4 * ref.GROUP[a.fmt]))
    r, g = np.arange(a.rows)[:, None], np.arange(4 * words)[None, :]
    at = ((r // 128) * words + g // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + g % 4
    return a.sf.cpu().numpy()[at]


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k", [(1, 1), (7, 130), (17, 33), (65, 200), (129, 64), (250, 97)])
def test_groups_past_the_last(ops, m, k, dtype, fmt):
    x = acts(m, k, seed=m + k, dtype=dtype)
    g = ref.GROUP[fmt]
    rows, cols = ops.fp4_cast_dual(x, fmt)
    turned = ops.fp4_cast(x.t(), fmt)
    whole = ops.fp4_cast(x.t().contiguous(), fmt)
    for a, n in ((rows, k), (cols, m), (turned, m), (whole, m), (ops.fp4_cast(x, fmt), k)):
        assert (scale_bytes(a, n)[:, -(-n // g):] == 0).all()
    for a in (cols, turned):
        assert np.array_equal(scale_bytes(a, m), scale_bytes(whole, m))


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
def test_groups_past_an_experts_rows(ops, fmt):
    offs = [0, 5, 5, 300, 417]
    x = acts(420, 70, seed=1)
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    cols = ops.fp4_cast_dual(x, fmt, offsets=off)[1]
    b = scale_bytes(cols, int(ops.load_library().fp4_column_extent(420, 4)))
    at, g = 0, ref.GROUP[fmt]
    for lo, hi in zip(offs[:-1], offs[1:]):
        n = -(-(hi - lo) // 256) * 256
        assert (b[:, (at + hi - lo + g - 1) // g:(at + n) // g] == 0).all()
        at += n
