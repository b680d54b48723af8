"""Experts whose offsets leave rows out, as a batch padded to a fixed capacity
does: whatever such rows hold has no influence on any expert, and results that
the calls allocate are zero there."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
from fp4_checks import acts, check, np64

pytestmark = pytest.mark.gpu

FMTS = pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
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


@pytest.fixture(scope="module")
def fp4(ops):
    from quantised_linear_layers_gb300 import fp4 as f
    return f


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


def nan_memory(*shapes):
    """Leaves NaN in memory that the next allocations of these sizes are likely to get."""
    junk = [torch.full(s, float("nan"), dtype=d, device="cuda") for s, d in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del junk


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


@FMTS
@pytest.mark.parametrize("path", [0, 2, 3], ids=["auto", "single", "pair"])
@pytest.mark.parametrize("n,k", [(136, 96), (257, 203), (1, 33)])
@pytest.mark.parametrize("offs", OFFSETS, ids=IDS)
def test_step_of_a_padded_batch(ops, fp4, offs, n, k, path, fmt):
    """Forward and both gradients within the bounds of the experts' rows alone; zeros in the rows of no expert."""
    m, e = offs[-1] + 9, len(offs) - 1
    x0, dy0, w = acts(m, k, seed=1), acts(m, n, seed=2, mul=1e-3), acts(e, n, k, seed=3, mul=0.02)
    off, w4 = torch.tensor(offs, dtype=torch.int32, device="cuda"), fp4.FP4ExpertWeight(w, fmt)
    rows = slice(offs[0], offs[-1])
    s = (lambda v: float(ref.tensor_scale(np64(v)))) if fmt == 0 else (lambda v: 1.0)
    sx, sd, sw = s(x0[rows]), s(dy0[rows]), s(w)
    ops.set_gemm_path(path)
    x, dy = padded(x0, offs, PADDING[0]), padded(dy0, offs, PADDING[1])
    shapes = [((m, n), torch.bfloat16), ((m, k), torch.bfloat16)]
    nan_memory(*shapes)
    y, saved = fp4.experts_forward_saving(x, off, w4)
    nan_memory(*shapes)
    dx, dw = fp4.experts_backward(dy, off, w4, saved)
    nan_memory(*shapes)
    y2 = fp4.experts_forward(x, off, w4, "own")
    nan_memory(*shapes)
    y3 = ops.gemm_fp4_nt_ragged(ops.fp4_cast(x, fmt, "own", off), w4.w)
    nan_memory(*shapes)
    y4 = ops.gemm_fp4_nt_ragged(ops.fp4_cast(x, fmt, "own", off), w4.w, dtype=torch.float32)
    assert torch.equal(y2, y) and torch.equal(y3, y)
    for d in (y, dx, y4):
        assert bool((d[:offs[0]] == 0).all()) and bool((d[offs[-1]:] == 0).all())
    for i, (lo, hi) in enumerate(zip(offs[:-1], offs[1:])):
        if lo == hi:
            assert bool((dw[i] == 0).all())
            continue
        xi, di, wi = np64(x0)[lo:hi], np64(dy0)[lo:hi], np64(w[i])
        check(y[lo:hi], ref.values(xi, fmt, sx), ref.values(wi, fmt, sw))
        check(y4[lo:hi], ref.values(xi, fmt, sx), ref.values(wi, fmt, sw))
        check(dx[lo:hi], ref.values(di, fmt, sd), ref.values(wi.T, fmt, sw))
        check(dw[i], ref.values(di.T, fmt, sd), ref.values(xi.T, fmt, sx))


@FMTS
@pytest.mark.parametrize("m,offs", [(300, [3, 40, 40, 200]), (16, [1, 3, 3, 12]), (40, [0, 0, 0, 0])],
                         ids=["300", "16", "none"])
def test_two_layers_in_a_row(ops, fp4, m, offs, fmt):
    """Two layers of experts on a padded batch equal the same layers on the experts' rows alone, bit for bit; the
    padding's gradient is zero."""
    torch.manual_seed(0)
    up, down = (fp4.FP4Experts(3, a, b, fmt, device="cuda") for a, b in ((96, 136), (136, 96)))
    x0, dy0 = acts(m, 96, seed=5), acts(m, 96, seed=6, mul=1e-3)
    rows = slice(offs[0], offs[-1])

    def step(x, dy, o):
        off = torch.tensor(o, dtype=torch.int32, device="cuda")
        x = x.clone().requires_grad_()
        nan_memory(*[((x.shape[0], c), torch.bfloat16) for c in (96, 136)])
        y = down(torch.nn.functional.silu(up(x, off)), off)
        nan_memory(*[((x.shape[0], c), torch.bfloat16) for c in (96, 136)])
        grads = torch.autograd.grad(y, [x, up.weight, down.weight], dy)
        with torch.no_grad():
            assert torch.equal(down(torch.nn.functional.silu(up(x, off)), off), y)
        return [y.detach(), *grads]

    ops.set_gemm_path(2)
    got = step(padded(x0, offs, float("nan")), padded(dy0, offs, float("nan")), offs)
    want = step(x0[rows], dy0[rows], [o - offs[0] for o in offs])
    for g, w in zip(got[2:], want[2:]):
        assert torch.equal(g, w)
    for g, w in zip(got[:2], want[:2]):
        assert torch.equal(g[rows], w)
        assert bool((g[:offs[0]] == 0).all()) and bool((g[offs[-1]:] == 0).all())


@FMTS
def test_a_given_output_keeps_its_rows(ops, fp4, fmt):
    """Rows of no expert are not written where the caller gives the output."""
    for m, offs in ((300, [3, 40, 40, 200]), (16, [1, 3, 3, 12])):
        x, w4 = acts(m, 96, seed=5), fp4.FP4ExpertWeight(acts(3, 136, 96, seed=3), fmt)
        off = torch.tensor(offs, dtype=torch.int32, device="cuda")
        out = torch.full((m, 136), -7.0, dtype=torch.bfloat16, device="cuda")
        fp4.experts_forward(x, off, w4, out=out)
        assert torch.equal(out[offs[0]:offs[-1]], fp4.experts_forward(x, off, w4)[offs[0]:offs[-1]])
        assert bool((out[:offs[0]] == -7).all()) and bool((out[offs[-1]:] == -7).all())
