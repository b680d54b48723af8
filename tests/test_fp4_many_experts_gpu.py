"""Experts' calls with more experts than a warp has lanes, up to the limit of
512: casts, products and gradients against 64 bits."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
from fp4_checks import acts, check, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp4():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantised_linear_layers_gb300 import build, fp4 as f, ops as o
    build.build()
    o.load_library()
    return f


def loads(experts, seed, rows):
    """Row counts: many empty experts, one long one, the last never empty."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 4, experts) * (rng.random(experts) < 0.5)
    c[experts // 3] += rows
    c[-1] += 1
    return c


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
@pytest.mark.parametrize("path", [0, 2, 3], ids=["auto", "single", "pair"])
@pytest.mark.parametrize("experts,first,rows", [(32, 0, 200), (33, 3, 130), (64, 0, 0), (65, 2, 300), (256, 0, 140),
                                                (511, 1, 5), (512, 0, 257)])
def test_step(fp4, experts, first, rows, path, fmt):
    from quantised_linear_layers_gb300 import ops
    n, k = 72, 100
    offs = np.concatenate([[0], np.cumsum(loads(experts, experts, rows))]) + first
    m = int(offs[-1])
    x, dy, w = acts(m, k, seed=1), acts(m, n, seed=2, mul=1e-3), acts(experts, n, k, seed=3, mul=0.02)
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    t = ops.fp4_tensor_scale(w) if fmt == 0 else None
    wr, wc = ops.fp4_cast_dual(w, fmt, t)
    tw = 1.0 if t is None else float(t)
    ops.set_gemm_path(path)
    try:
        y, saved = ops.fp4_linear_saving(x, wr, None, off)
        dx, dw = ops.fp4_linear_backward(dy, wc, saved, None, off)
        again = ops.fp4_linear(x, wr, None, off)
    finally:
        ops.set_gemm_path(0)
    assert ops.device_status() == 0
    assert torch.equal(again[first:], y[first:])
    where = ref.expert_sf_rows(offs.tolist())
    rows_of = np.array(sorted(where))
    a = ops.fp4_cast(x, fmt, offsets=off)
    got = ref.unpack(a.q.cpu().numpy()[rows_of], a.sf.cpu().numpy(), fmt, len(rows_of), k, sf_rows=[where[r] for r in rows_of])
    assert np.array_equal(got, ref.values(np64(x)[rows_of], fmt))
    xn, dn, wn = np64(x), np64(dy), np64(w)
    for i in range(experts):
        lo, hi = offs[i], offs[i + 1]
        if lo == hi:
            assert bool((dw[i] == 0).all())
            continue
        check(y[lo:hi], ref.values(xn[lo:hi], fmt), ref.values(wn[i], fmt, tw))
        check(dx[lo:hi], ref.values(dn[lo:hi], fmt), ref.values(wn[i].T, fmt, tw))
        check(dw[i], ref.values(dn[lo:hi].T, fmt), ref.values(xn[lo:hi].T, fmt))
    assert ops.device_status() == 0


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
@pytest.mark.parametrize("experts", [33, 512])
def test_few_rows(fp4, experts, fmt):
    """Up to 16 rows, cast inside the product: in experts on both sides of every turn of 32."""
    from quantised_linear_layers_gb300 import ops
    n, k = 72, 100
    x, w = acts(16, k, seed=1), acts(experts, n, k, seed=3, mul=0.02)
    wr = ops.fp4_cast(w, fmt)
    rng = np.random.default_rng(experts)
    for first, last in ((0, experts - 1), (31, 32), (experts - 1, experts - 1)):
        picks = np.sort(np.concatenate([[first, last], rng.integers(first, last + 1, 14)]))
        offs = np.searchsorted(picks, np.arange(experts + 1))
        y = ops.fp4_linear(x, wr, None, torch.tensor(offs, dtype=torch.int32, device="cuda"))
        for i in np.unique(picks):
            lo, hi = offs[i], offs[i + 1]
            check(y[lo:hi], ref.values(np64(x)[lo:hi], fmt), ref.values(np64(w[i]), fmt))
    assert ops.device_status() == 0


def test_one_more_is_refused(fp4):
    from quantised_linear_layers_gb300 import ops
    x, w = acts(16, 64, seed=1), acts(513, 8, 64, seed=2)
    off = torch.zeros(514, dtype=torch.int32, device="cuda")
    wr = ops.fp4_cast(w)
    for call in (lambda: ops.fp4_cast(x, 0, None, off), lambda: ops.fp4_linear(x, wr, None, off),
                 lambda: ops.fp4_cast_dual(x, 0, None, off)):
        with pytest.raises(ops.QLError):
            call()
