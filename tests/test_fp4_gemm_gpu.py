"""4-bit products and layers on the GPU against the numpy definition in 64
bits. The casts are exact (test_fp4_cast_gpu.py), so the product's bound is that
of its fp32 accumulation alone (fp4_reference.bound)."""
import copy
import pickle

import numpy as np
import pytest
import torch

import fp4_reference as ref

pytestmark = pytest.mark.gpu

FMTS = pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
PATHS = pytest.mark.parametrize("path", [0, 2, 3], ids=["auto", "single", "pair"])


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


def acts(*shape, seed, dtype=torch.bfloat16, mul=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-3, 4, (*shape[:-1], 1), generator=g).float())
    return (x * mul).to(dtype).cuda()


def np64(x):
    return x.detach().float().cpu().numpy().astype(np.float64)


def check(got, xv, wv, d0=None):
    want, absum = ref.product(xv, wv)
    if d0 is not None:
        want, absum = want + d0, absum + np.abs(d0)
    got, is_bf16 = np64(got), got.dtype == torch.bfloat16
    e = ref.bound(absum, xv.shape[1])
    if is_bf16:
        # a bf16 result is the rounding of some value within the fp32 bound
        bad = (got < ref.bf16(want - e)) | (got > ref.bf16(want + e))
    else:
        bad = ~(np.abs(got - want) <= e)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off: {got[bad][:4]} for {want[bad][:4]}, bound {e[bad][:4]}"


SHAPES = [(1, 1, 1), (1, 128, 64), (7, 33, 65), (16, 130, 256), (17, 128, 320), (64, 300, 1000), (65, 1000, 96),
          (129, 257, 511), (300, 520, 2051), (1, 512, 7168), (513, 769, 129), (256, 256, 256), (40, 4096, 1024)]


@FMTS
@PATHS
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(ops, m, n, k, path, fmt):
    x, w = acts(m, k, seed=m + k), acts(n, k, seed=n, mul=0.02)
    ts = ops.fp4_tensor_scale(w) if fmt == 0 else None
    a, b = ops.fp4_cast(x, fmt), ops.fp4_cast(w, fmt, ts)
    xv, wv = ref.values(np64(x), fmt), ref.values(np64(w), fmt, 1.0 if ts is None else float(ts))
    ops.set_gemm_path(path)
    check(ops.gemm_fp4_nt(a, b), xv, wv)
    check(ops.gemm_fp4_nt(a, b, dtype=torch.float32), xv, wv)
    d = torch.randn((m, n), device="cuda")
    d0 = np64(d)
    ops.gemm_fp4_nt(a, b, out=d, accumulate=True)
    check(d, xv, wv, d0)


@FMTS
@PATHS
def test_strided_output_keeps_its_surroundings(ops, path, fmt):
    m, n, k = 140, 264, 192
    x, w = acts(m, k, seed=1), acts(n, k, seed=2)
    a, b = ops.fp4_cast(x, fmt), ops.fp4_cast(w, fmt)
    xv, wv = ref.values(np64(x), fmt), ref.values(np64(w), fmt)
    ops.set_gemm_path(path)
    for dtype in (torch.bfloat16, torch.float32):
        for lead, extra in ((0, 0), (8, 24), (1, 2)):
            big = torch.full((m + 2, n + lead + extra), -7.0, dtype=dtype, device="cuda")
            view = big[1:m + 1, lead:lead + n]
            ops.gemm_fp4_nt(a, b, out=view)
            check(view, xv, wv)
            big[1:m + 1, lead:lead + n] = -7.0
            assert bool((big == -7.0).all())


@FMTS
def test_the_same_every_time_and_on_every_path(ops, fmt):
    """Products of one cast are the same bits call after call; with sums that fp32 holds exactly, on every path."""
    x = torch.randint(-4, 5, (200, 900)).bfloat16().cuda()
    w = torch.randint(-4, 5, (300, 900)).bfloat16().cuda()
    a, b = ops.fp4_cast(x, fmt), ops.fp4_cast(w, fmt)
    outs = []
    for path in (0, 0, 2, 3):
        ops.set_gemm_path(path)
        outs.append(ops.gemm_fp4_nt(a, b, dtype=torch.float32))
    assert all(torch.equal(o, outs[0]) for o in outs)


@FMTS
def test_empty(ops, fmt):
    x, w = acts(5, 64, seed=1), acts(7, 64, seed=2)
    a, b = ops.fp4_cast(x, fmt), ops.fp4_cast(w, fmt)
    assert ops.gemm_fp4_nt(ops.fp4_cast(x[:0], fmt), b).shape == (0, 7)
    assert ops.gemm_fp4_nt(a, ops.fp4_cast(w[:0], fmt)).shape == (5, 0)
    a0, b0 = ops.fp4_cast(x[:, :0], fmt), ops.fp4_cast(w[:, :0], fmt)
    assert bool((ops.gemm_fp4_nt(a0, b0) == 0).all())
    d = torch.ones((5, 7), device="cuda")
    ops.gemm_fp4_nt(a0, b0, out=d, accumulate=True)
    assert bool((d == 1).all())


@FMTS
@PATHS
def test_non_finite_rows_stay_in_their_rows(ops, path, fmt):
    x, w = acts(140, 256, seed=1), acts(300, 256, seed=2)
    x[3, 100], x[130, 7], w[17, 255] = float("nan"), float("inf"), float("nan")
    ops.set_gemm_path(path)
    d = ops.gemm_fp4_nt(ops.fp4_cast(x, fmt), ops.fp4_cast(w, fmt))
    bad = torch.zeros((140, 300), dtype=torch.bool, device="cuda")
    bad[3], bad[130], bad[:, 17] = True, True, True
    assert torch.equal(torch.isnan(d), bad)


OFFSETS = [[0, 5], [0, 0, 130, 130, 131, 300], [0, 256, 512, 513], [3, 40, 40, 200], list(range(10)),
           [0, 700, 700, 1300]]


@FMTS
@PATHS
@pytest.mark.parametrize("offs", OFFSETS, ids=[f"{len(o) - 1}_{o[-1]}" for o in OFFSETS])
def test_experts_product(ops, offs, path, fmt):
    m, n, k, e = offs[-1] + 3, 330, 200, len(offs) - 1
    x, w = acts(m, k, seed=1), acts(e, n, k, seed=2, mul=0.02)
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    ts = ops.fp4_tensor_scale(w) if fmt == 0 else None
    a, b = ops.fp4_cast(x, fmt, offsets=off), ops.fp4_cast(w, fmt, ts)
    ops.set_gemm_path(path)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((m, n), -7.0, dtype=dtype, device="cuda")
        ops.gemm_fp4_nt_ragged(a, b, out=out)
        xv = ref.values(np64(x), fmt)
        for i, (lo, hi) in enumerate(zip(offs[:-1], offs[1:])):
            if hi > lo:
                check(out[lo:hi], xv[lo:hi], ref.values(np64(w[i]), fmt, 1.0 if ts is None else float(ts)))
        assert bool((out[:offs[0]] == -7).all()) and bool((out[offs[-1]:] == -7).all())


@FMTS
@PATHS
@pytest.mark.parametrize("offs", OFFSETS, ids=[f"{len(o) - 1}_{o[-1]}" for o in OFFSETS])
def test_experts_weight_gradient(ops, offs, path, fmt):
    t, n, k, e = offs[-1] + 3, 330, 200, len(offs) - 1
    x, dy = acts(t, k, seed=1), acts(t, n, seed=2, mul=1e-3)
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    ts = ops.fp4_tensor_scale(dy) if fmt == 0 else None
    tv = 1.0 if ts is None else float(ts)
    cx, cy = ops.fp4_cast_dual(x, fmt, None, off)[1], ops.fp4_cast_dual(dy, fmt, ts, off)[1]
    ops.set_gemm_path(path)
    d = ops.gemm_fp4_wgrad_ragged(cy, cx)
    acc = torch.randn((e, n, k), device="cuda")
    d0 = np64(acc)
    ops.gemm_fp4_wgrad_ragged(cy, cx, out=acc, accumulate=True)
    for i, (lo, hi) in enumerate(zip(offs[:-1], offs[1:])):
        if hi == lo:
            assert bool((d[i] == 0).all())
            assert np.array_equal(np64(acc[i]), d0[i])
            continue
        yv, xv = ref.values(np64(dy)[lo:hi].T, fmt, tv), ref.values(np64(x)[lo:hi].T, fmt)
        check(d[i], yv, xv)
        check(acc[i], yv, xv, d0[i])


# Tiles of 256 x 256 on up to 76 pairs of SMs: 38, 49, and 81 and 110 in two rounds; the last tile of columns ends in
# its first half.
@FMTS
@pytest.mark.parametrize("mt,nt", [(1, 38), (7, 7), (9, 9), (11, 10)])
def test_product_in_rounds_of_tiles(ops, mt, nt, fmt):
    m, n, k = mt * 256 - 19, nt * 256 - 136, 330
    x, w = acts(m, k, seed=m + k), acts(n, k, seed=n, mul=0.02)
    ops.set_gemm_path(3)
    a, b = ops.fp4_cast(x, fmt), ops.fp4_cast(w, fmt)
    xv, wv = ref.values(np64(x), fmt), ref.values(np64(w), fmt)
    check(ops.gemm_fp4_nt(a, b), xv, wv)
    d = torch.randn((m, n), device="cuda")
    d0 = np64(d)
    ops.gemm_fp4_nt(a, b, out=d, accumulate=True)
    check(d, xv, wv, d0)
    # rows of D that no 16-byte store can address
    wide = torch.full((m, n + 5), -7.0, dtype=torch.bfloat16, device="cuda")
    ops.gemm_fp4_nt(a, b, out=wide[:, 2:2 + n])
    check(wide[:, 2:2 + n], xv, wv)
    assert bool((wide[:, :2] == -7).all()) and bool((wide[:, 2 + n:] == -7).all())


@FMTS
@pytest.mark.parametrize("offs", [[0, 700, 700, 2000, 2600], [0, 1, 257, 300, 300, 301, 1999]], ids=["96", "112"])
def test_experts_product_in_rounds_of_tiles(ops, offs, fmt):
    m, n, k, e = offs[-1] + 3, 8 * 256 - 136, 200, len(offs) - 1
    x, w = acts(m, k, seed=1), acts(e, n, k, seed=2, mul=0.02)
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    ops.set_gemm_path(3)
    out = torch.full((m, n), -7.0, dtype=torch.bfloat16, device="cuda")
    ops.gemm_fp4_nt_ragged(ops.fp4_cast(x, fmt, offsets=off), ops.fp4_cast(w, fmt), out=out)
    xv = ref.values(np64(x), fmt)
    for i, (lo, hi) in enumerate(zip(offs[:-1], offs[1:])):
        if hi > lo:
            check(out[lo:hi], xv[lo:hi], ref.values(np64(w[i]), fmt))
    assert bool((out[offs[-1]:] == -7).all())


@FMTS
@pytest.mark.parametrize("offs", [[0, 300, 300], [0, 5, 333], [0, 90, 91, 400]], ids=["empty", "80", "120"])
def test_experts_weight_gradient_in_rounds_of_tiles(ops, offs, fmt):
    t, n, k, e = offs[-1], 8 * 256 - 136, 1100, len(offs) - 1
    x, dy = acts(t, k, seed=1), acts(t, n, seed=2, mul=1e-3)
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    cx, cy = ops.fp4_cast_dual(x, fmt, None, off)[1], ops.fp4_cast_dual(dy, fmt, None, off)[1]
    ops.set_gemm_path(3)
    d = ops.gemm_fp4_wgrad_ragged(cy, cx)
    acc = torch.randn((e, n, k), device="cuda")
    d0 = np64(acc)
    ops.gemm_fp4_wgrad_ragged(cy, cx, out=acc, accumulate=True)
    for i, (lo, hi) in enumerate(zip(offs[:-1], offs[1:])):
        if hi == lo:
            assert bool((d[i] == 0).all())
            assert np.array_equal(np64(acc[i]), d0[i])
            continue
        yv, xv = ref.values(np64(dy)[lo:hi].T, fmt), ref.values(np64(x)[lo:hi].T, fmt)
        check(d[i], yv, xv)
        check(acc[i], yv, xv, d0[i])


def test_offsets_out_of_order_are_reported_and_stay_inside(ops):
    x, w = acts(100, 64, seed=1), acts(3, 40, 64, seed=2)
    off = torch.tensor([0, 90, 30, 500], dtype=torch.int32, device="cuda")
    guard = torch.full((104, 40), -7.0, dtype=torch.bfloat16, device="cuda")
    ops.gemm_fp4_nt_ragged(ops.fp4_cast(x, 0, offsets=off), ops.fp4_cast(w, 0), out=guard[:100])
    assert ops.device_status() == 1
    assert bool((guard[100:] == -7).all())
    cols = ops.fp4_cast_dual(x, 0, offsets=off)[1]
    ops.gemm_fp4_wgrad_ragged(cols, cols)
    assert ops.device_status() == 1


def test_experts_without_tokens(ops, fp4):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    w = fp4.FP4ExpertWeight(acts(3, 40, 64, seed=2))
    x = acts(5, 64, seed=3)[:0]
    y, cols = fp4.experts_forward_saving(x, off, w)
    dx, dw = fp4.experts_backward(acts(5, 40, seed=4)[:0], off, w, cols)
    assert y.shape == (0, 40) and dx.shape == (0, 64) and bool((dw == 0).all())


# ---------------------------------------------------------------- layers
@FMTS
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("t,n,k", [(1, 64, 96), (77, 130, 200), (300, 257, 515)])
def test_layer_step(ops, fp4, t, n, k, dtype, fmt):
    """Forward and both gradients against the formulas over the cast operands."""
    x, w, dy = acts(t, k, seed=1, dtype=dtype), acts(n, k, seed=2, mul=0.02), acts(t, n, seed=3, mul=1e-3)
    s = (lambda v: float(ref.tensor_scale(np64(v)))) if fmt == 0 else (lambda v: 1.0)
    w4 = fp4.FP4Weight(w, fmt)
    y, saved = fp4.forward_saving(x, w4)
    dx, dw = fp4.backward(dy, w4, saved)
    check(y, ref.values(np64(x), fmt, s(x)), ref.values(np64(w), fmt, s(w)))
    check(dx, ref.values(np64(dy), fmt, s(dy)), ref.values(np64(w).T, fmt, s(w)))
    check(dw, ref.values(np64(dy).T, fmt, s(dy)), ref.values(np64(x).T, fmt, s(x)))
    assert torch.equal(fp4.dgrad(dy, w4), dx)
    assert torch.equal(fp4.forward(x, w4, ops.fp4_tensor_scale(x) if fmt == 0 else None), y)


@FMTS
def test_linear_module(ops, fp4, fmt):
    """autograd through FP4Linear equals the functions; the fp32 main grad accumulates; a changed weight is cast anew."""
    torch.manual_seed(0)
    layer = fp4.FP4Linear(200, 130, fmt, device="cuda")
    x = acts(6, 11, 200, seed=5).requires_grad_()
    dy = acts(6, 11, 130, seed=6, mul=1e-3)
    y = layer(x)
    y.backward(dy)
    w4 = fp4.FP4Weight(layer.weight.detach(), fmt)
    y2, saved = fp4.forward_saving(x.detach().reshape(-1, 200), w4)
    dx2, dw2 = fp4.backward(dy.reshape(-1, 130), w4, saved)
    assert torch.equal(y.reshape(-1, 130), y2) and torch.equal(x.grad.reshape(-1, 200), dx2)
    assert torch.equal(layer.weight.grad, dw2.bfloat16())
    with torch.no_grad():
        assert torch.equal(layer(x), y)
        layer.weight.mul_(2)
        # doubling every weight doubles the scales and nothing else
        assert torch.equal(layer(x).float(), 2 * y.float())
    main = fp4.FP4Linear(200, 130, fmt, device="cuda", accumulate_main_grad=True)
    with torch.no_grad():
        main.weight.copy_(w4_source(layer) / 2)
    for _ in range(2):
        main(x.detach()).backward(dy)
    assert main.weight.grad is None
    assert torch.allclose(main.main_grad, 2 * dw2, rtol=2.0 ** -22, atol=0)
    frozen = fp4.FP4Linear(200, 130, fmt, device="cuda")
    frozen.weight.requires_grad_(False)
    xf = x.detach().clone().requires_grad_()
    with torch.no_grad():
        frozen.weight.copy_(main.weight)
    frozen(xf).backward(dy)
    assert torch.equal(xf.grad.reshape(-1, 200), dx2)


def w4_source(layer):
    return layer.weight.detach()


@FMTS
def test_experts_module(ops, fp4, fmt):
    torch.manual_seed(0)
    offs = [0, 70, 70, 81, 150]
    layer = fp4.FP4Experts(4, 96, 130, fmt, device="cuda")
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    x, dy = acts(150, 96, seed=5).requires_grad_(), acts(150, 130, seed=6, mul=1e-3)
    y = layer(x, off)
    y.backward(dy)
    s = (lambda v: float(ref.tensor_scale(np64(v)))) if fmt == 0 else (lambda v: 1.0)
    w = layer.weight.detach()
    for i, (lo, hi) in enumerate(zip(offs[:-1], offs[1:])):
        if lo == hi:
            assert bool((layer.weight.grad[i] == 0).all())
            continue
        xs, ds = x.detach()[lo:hi], dy[lo:hi]
        wi = np64(w[i])
        check(y[lo:hi], ref.values(np64(xs), fmt, s(x)), ref.values(wi, fmt, s(w)))
        check(x.grad[lo:hi], ref.values(np64(ds), fmt, s(dy)), ref.values(wi.T, fmt, s(w)))
    with torch.no_grad():
        assert torch.equal(layer(x, off), y)


@FMTS
def test_gradients_against_differences(ops, fp4, fmt):
    """On operands that the format holds exactly the layer is the plain product, so differences of the loss
    sum(dy * Y) along a direction of the operand equal the gradient's (the loss is linear in each operand)."""
    torch.manual_seed(3)
    pick = torch.tensor([-6.0, -4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4, 6])

    def exactly(*shape):
        v = pick[torch.randint(0, 15, shape)]
        v[..., ::8, :] = 6.0                                   # every group, in either direction, has its scale at 1
        v[..., ::8] = 6.0
        return v.cuda()

    t, n, k = 64, 96, 64
    x, w, dy = exactly(t, k), exactly(n, k), exactly(t, n)
    w4 = fp4.FP4Weight(w.bfloat16(), fmt)
    _, saved = fp4.forward_saving(x.bfloat16(), w4)
    dx, dw = fp4.backward(dy.bfloat16(), w4, saved)
    loss = lambda xx, ww: float((dy.double() * ops.gemm_fp4_nt(  # noqa: E731
        ops.fp4_cast(xx, fmt), ops.fp4_cast(ww, fmt), dtype=torch.float32).double()).sum())
    for seed in range(4):
        torch.manual_seed(seed)
        x2, w2 = exactly(t, k), exactly(n, k)
        want = float((dw.double() * (w2 - w).double()).sum())
        assert loss(x, w2) - loss(x, w) == want                # whole multiples of 1/16 below 2^24: exact
        want = float(((dy.double() @ w.double()) * (x2 - x).double()).sum())
        assert loss(x2, w) - loss(x, w) == want
    exact_dx = dy.double() @ w.double()
    assert torch.equal(dx.double(), exact_dx.float().bfloat16().double())


@FMTS
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 4096, 7168), (3, 300, 515), (16, 257, 2048), (16, 128, 96), (9, 640, 4099),
                                   (17, 300, 515), (31, 4096, 2048), (33, 300, 700), (64, 130, 7168), (65, 300, 515),
                                   (200, 300, 1000)])
def test_forward_call_equals_cast_and_product(ops, m, n, k, dtype, fmt):
    """Bit for bit, also where the product casts X itself (up to 8 rows), for rows that start anywhere."""
    big, w = acts(m, k + 3, seed=m + k, dtype=dtype), acts(n, k, seed=n, mul=0.02)
    b = ops.fp4_cast(w, fmt, ops.fp4_tensor_scale(w) if fmt == 0 else None)
    t = torch.tensor([0.25], device="cuda") if fmt == 0 else None
    for x in (big[:, :k].contiguous(), big[:, 1:k + 1], big[:, 3:].t().contiguous().t()):
        for scale in (None, t):
            want = ops.gemm_fp4_nt(ops.fp4_cast(x, fmt, scale), b)
            assert torch.equal(ops.fp4_linear(x, b, scale), want)
            if m <= 64 and k < 3000:
                check(want, ref.values(np64(x), fmt, 1.0 if scale is None else 0.25),
                      ref.values(np64(w), fmt, 1.0 if b.scale is None else float(b.scale)))
        if fmt == 0:
            want = ops.gemm_fp4_nt(ops.fp4_cast(x, fmt, ops.fp4_tensor_scale(x)), b)
            assert torch.equal(ops.fp4_linear(x, b, ops.FP4_OWN_SCALE), want)
    out = torch.full((m, n + 5), -7.0, dtype=torch.bfloat16, device="cuda")
    ops.fp4_linear(x, b, out=out[:, 2:n + 2])
    assert torch.equal(out[:, 2:n + 2], ops.fp4_linear(x, b)) and bool((out[:, :2] == -7).all()) and bool((out[:, n + 2:] == -7).all())


@FMTS
@pytest.mark.parametrize("offs", [[0, 1], [0, 3, 3, 7, 16], [2, 2, 5, 6], [0, 9, 25], [0, 1, 40, 64], [0, 100, 100, 331]],
                         ids=["1", "16", "6", "25", "64", "331"])
def test_forward_call_by_expert(ops, offs, fmt):
    m, n, k, e = offs[-1], 300, 515, len(offs) - 1
    x, w = acts(m, k, seed=1), acts(e, n, k, seed=2, mul=0.02)
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    b = ops.fp4_cast(w, fmt)
    want = torch.full((m, n), -7.0, dtype=torch.bfloat16, device="cuda")
    ops.gemm_fp4_nt_ragged(ops.fp4_cast(x, fmt, offsets=off), b, out=want)
    got = torch.full_like(want, -7.0)
    ops.fp4_linear(x, b, offsets=off, out=got)
    assert torch.equal(got, want)
    xv = ref.values(np64(x), fmt)
    for i, (lo, hi) in enumerate(zip(offs[:-1], offs[1:])):
        if hi > lo:
            check(got[lo:hi], xv[lo:hi], ref.values(np64(w[i]), fmt))


@FMTS
def test_forward_call_non_finite(ops, fmt):
    x, w = acts(7, 640, seed=1), acts(300, 640, seed=2)
    x[2, 100], x[5, 639] = float("nan"), float("-inf")
    d = ops.fp4_linear(x, ops.fp4_cast(w, fmt))
    bad = torch.zeros((7, 300), dtype=torch.bool, device="cuda")
    bad[2], bad[5] = True, True
    assert torch.equal(torch.isnan(d), bad)


def test_side_stream_and_graph(ops, fp4):
    x, w = acts(48, 512, seed=1), acts(384, 512, seed=2)
    w4 = fp4.FP4Weight(w, 0, dgrad=False)
    want = fp4.forward(x, w4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = fp4.forward(x, w4)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    buf = x.clone()
    with torch.cuda.graph(graph):
        out = fp4.forward(buf, w4)
    buf.copy_(2 * x)
    graph.replay()
    assert torch.equal(out.float(), 2 * want.float())


def test_time_out_is_reported(ops):
    """A producer that issues nothing: the waits run out, the call ends and the status says so."""
    a, b = ops.fp4_cast(acts(40, 512, seed=1), 0), ops.fp4_cast(acts(300, 512, seed=2), 0)
    off = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    ra, rb = ops.fp4_cast(acts(40, 512, seed=1), 0, offsets=off), ops.fp4_cast(acts(1, 300, 512, seed=2), 0)
    ops.set_wait_limit_ms(50)
    ops.test_stall_gemm_producer(True)
    try:
        for path in (0, 2, 3):
            ops.set_gemm_path(path)
            ops.gemm_fp4_nt(a, b)
            assert ops.device_status() == 5
            ops.gemm_fp4_nt_ragged(ra, rb)
            assert ops.device_status() == 5
            ops.fp4_linear(acts(9, 512, seed=1), b)
            assert ops.device_status() == 5
    finally:
        ops.test_stall_gemm_producer(False)
        ops.set_wait_limit_ms(2000)
    ops.set_gemm_path(0)
    check(ops.gemm_fp4_nt(a, b), ref.values(np64(acts(40, 512, seed=1)), 0), ref.values(np64(acts(300, 512, seed=2)), 0))


def test_mx_takes_no_notice_of_a_tensor_scale(ops):
    x, w = acts(70, 200, seed=1), acts(130, 200, seed=2)
    b, half = ops.fp4_cast(w, 1), torch.tensor([0.5], device="cuda")
    want = ops.fp4_cast(x, 1)
    for scale in (half, ops.FP4_OWN_SCALE):
        a = ops.fp4_cast(x, 1, scale)
        r, c = ops.fp4_cast_dual(x, 1, scale)
        assert a.scale is None and r.scale is None and c.scale is None
        for v in (a, r):
            assert torch.equal(ops.fp4_dequant(v), ops.fp4_dequant(want))
        assert torch.equal(ops.fp4_linear(x, b, scale), ops.gemm_fp4_nt(want, b))
        assert torch.equal(ops.fp4_linear(x[:3], b, scale), ops.gemm_fp4_nt(want, b)[:3])


def test_refusals(ops, fp4):
    x, w = acts(8, 64, seed=1), acts(16, 64, seed=2)
    a, b, bm = ops.fp4_cast(x), ops.fp4_cast(w), ops.fp4_cast(w, 1)
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    r = ops.fp4_cast(x, offsets=off)
    one = torch.ones(1, device="cuda")
    for bad in (lambda: ops.fp4_cast(x, 2), lambda: ops.fp4_cast(x[0]), lambda: ops.fp4_cast(x.cpu()),
                lambda: ops.fp4_cast(x, 0, one.double()),
                lambda: ops.fp4_cast(x, 0, one.cpu()), lambda: ops.fp4_cast(x, 0, None, off.long()),
                lambda: ops.fp4_cast(x[None], 0, None, off), lambda: ops.fp4_cast_dual(x.t()),
                lambda: ops.gemm_fp4_nt(a, bm), lambda: ops.gemm_fp4_nt(a, ops.fp4_cast(w[:, :32])),
                lambda: ops.gemm_fp4_nt(r, b), lambda: ops.gemm_fp4_nt_ragged(a, ops.fp4_cast(w[None])),
                lambda: ops.gemm_fp4_nt_ragged(r, r),
                lambda: ops.gemm_fp4_nt_ragged(r, ops.fp4_cast(torch.stack([w, w]))),
                lambda: ops.gemm_fp4_nt(a, b, accumulate=True),
                lambda: ops.gemm_fp4_nt(a, b, out=torch.empty((8, 16), dtype=torch.bfloat16, device="cuda"), accumulate=True),
                lambda: ops.gemm_fp4_nt(a, b, out=torch.empty((8, 15), device="cuda")),
                lambda: ops.gemm_fp4_nt(a, b, out=torch.empty((16, 8), device="cuda").t()),
                lambda: ops.fp4_linear(x[0], b), lambda: ops.fp4_linear(x[:, :32], b), lambda: ops.fp4_linear(x, b, offsets=off[:1]),
                lambda: ops.fp4_linear(x, ops.fp4_cast(torch.stack([w, w]))),
                lambda: ops.fp4_cast(x, 0, 0.5),
                lambda: ops.fp4_cast(torch.stack([x, x, x])[::2], 0, ops.FP4_OWN_SCALE),
                lambda: ops.fp4_linear(x, b, out=torch.empty((8, 16), device="cuda")),
                lambda: ops.gemm_fp4_wgrad_ragged(a, b), lambda: ops.fp4_dequant(r), lambda: fp4.FP4Weight(w[None]),
                lambda: fp4.dgrad(acts(8, 16, seed=3), fp4.FP4Weight(w, dgrad=False)),
                lambda: fp4.FP4Linear(64, 16, device="cuda")(acts(8, 63, seed=1))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        ops.fp4_cast(x.half())


def test_rows_of_out_that_overlap_are_refused(ops):
    a, b = ops.fp4_cast(acts(8, 64, seed=1)), ops.fp4_cast(acts(16, 64, seed=2))
    for dtype in (torch.bfloat16, torch.float32):
        for out in (torch.zeros((1, 16), dtype=dtype, device="cuda").expand(8, 16),
                    torch.zeros(100, dtype=dtype, device="cuda").as_strided((8, 16), (8, 1))):
            with pytest.raises(ValueError):
                ops.gemm_fp4_nt(a, b, out=out)
            with pytest.raises(ValueError):
                ops.fp4_dequant(ops.fp4_cast(acts(8, 16, seed=1)), dtype, out=out)
    with pytest.raises(ValueError):
        ops.fp4_linear(acts(8, 64, seed=1), b, out=torch.zeros((1, 16), dtype=torch.bfloat16, device="cuda").expand(8, 16))
    one = torch.zeros((8, 1), device="cuda")                     # rows of one column: any stride from 1 on
    ops.gemm_fp4_nt(a, ops.fp4_cast(acts(1, 64, seed=2)), out=one)
    assert bool((one != 0).any())


def test_backward_refuses_a_cast_by_experts_without_them(ops):
    x, off = acts(64, 64, seed=1), torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ops.fp4_linear_backward(acts(64, 32, seed=2), None, ops.fp4_cast(x, offsets=off))
    with pytest.raises(ValueError):
        ops.fp4_linear_backward(acts(64, 32, seed=2), None, ops.fp4_cast(x), None, off)


def test_own_scale_of_nothing_and_of_transposed_batches(ops):
    least = float(ops.fp4_tensor_scale(torch.empty((0, 5), device="cuda")))
    for x in (torch.empty((0, 64), device="cuda"), torch.empty((7, 0), dtype=torch.bfloat16, device="cuda")):
        assert float(ops.fp4_cast(x, 0, ops.FP4_OWN_SCALE).scale) == least
        assert [float(c.scale) for c in ops.fp4_cast_dual(x, 0, ops.FP4_OWN_SCALE)] == [least, least]
    x = acts(3, 40, 70, seed=1)
    got, want = ops.fp4_cast(x.transpose(1, 2), 0, ops.FP4_OWN_SCALE), ops.fp4_cast_dual(x, 0, ops.FP4_OWN_SCALE)[1]
    assert float(got.scale) == float(want.scale)
    assert torch.equal(got.q, want.q) and torch.equal(got.sf[:-16], want.sf[:-16])


def test_layer_sees_every_change_of_its_weight(fp4):
    x, w1, w2 = acts(20, 96, seed=1), acts(48, 96, seed=2), acts(48, 96, seed=3)
    layer = fp4.FP4Linear(96, 48, device="cuda")

    def want(w):
        return fp4.forward(x, fp4.FP4Weight(w), "own")

    with torch.no_grad():
        layer.weight.copy_(w1)
        assert torch.equal(layer(x), want(w1))
        layer.weight.copy_(w2)
        assert torch.equal(layer(x), want(w2))
        layer.weight.data = w1.clone()
        assert torch.equal(layer(x), want(w1))
        for w in (w2, w1, w2):                       # storage that comes and goes
            layer.weight.data = w.clone()
            assert torch.equal(layer(x), want(w))
        layer.weight.data.copy_(w1)
        layer.forget_casts()
        assert torch.equal(layer(x), want(w1))
        layer.float()
        assert torch.equal(layer(x), want(w1))
        other = copy.deepcopy(layer)
        other.weight.copy_(w2)
        assert torch.equal(other(x), want(w2)) and torch.equal(layer(x), want(w1))


def test_copies_of_a_cast_stand_by_themselves(ops):
    x, w = acts(20, 96, seed=1), acts(48, 96, seed=2)
    rows, cols = ops.fp4_cast_dual(w, 0, ops.FP4_OWN_SCALE)
    want, a = ops.gemm_fp4_nt(ops.fp4_cast(x), rows), ops.fp4_cast(x)
    for c in (copy.deepcopy(rows), pickle.loads(pickle.dumps(rows))):
        assert c.q_ptr == c.buf.data_ptr() != rows.q_ptr and c.scale_ptr != rows.scale_ptr
        assert float(c.scale) == float(rows.scale)
        assert torch.equal(ops.gemm_fp4_nt(a, c), want)


def test_layer_on_two_streams(fp4):
    """The casts are made behind other work of a stream and used at once on another one."""
    x, w = acts(20, 1024, seed=1), acts(2048, 1024, seed=2)
    layer = fp4.FP4Linear(1024, 2048, device="cuda")
    with torch.no_grad():
        layer.weight.copy_(w)
        want = fp4.forward(x, fp4.FP4Weight(w), "own")
        big = torch.randn((4096, 4096), device="cuda")
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(20):
                big = big @ big * 1e-3
            first = layer(x)
        second = layer(x)
        torch.cuda.synchronize()
    assert torch.equal(first, want) and torch.equal(second, want)


def test_training_step_in_a_graph_follows_its_weight(fp4):
    x, w, dy = acts(40, 96, seed=1), acts(48, 96, seed=2), acts(40, 48, seed=3, mul=1e-3)
    layers = []
    for _ in range(2):
        layer = fp4.FP4Linear(96, 48, device="cuda")
        with torch.no_grad():
            layer.weight.copy_(w)
        layers.append(layer)

    def step(layer):
        y = layer(x)
        grad, = torch.autograd.grad(y, layer.weight, dy)
        with torch.no_grad():
            layer.weight.sub_(grad, alpha=1e3)
        return y.detach()

    eager = [step(layers[0]).clone() for _ in range(3)]
    assert not torch.equal(eager[0], eager[2])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [step(layers[1]).clone()]
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(layers[1])
    for _ in range(2):
        graph.replay()
        got.append(y.clone())
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    for _ in range(2):                               # and a call outside the graph sees what the graph left
        with torch.no_grad():
            assert torch.equal(layers[1](x), layers[0](x))
        graph.replay()
        step(layers[0])


def test_forward_in_a_graph_keeps_its_casts(fp4):
    x, w1, w2 = acts(5, 96, seed=1), acts(48, 96, seed=2), acts(48, 96, seed=3)
    layer = fp4.FP4Linear(96, 48, device="cuda")
    with torch.no_grad():
        layer.weight.copy_(w1)
        want = layer(x).clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = layer(x)
        layer.weight.copy_(w2)
        layer(x)
        junk = [torch.full((4096,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
        graph.replay()
        assert torch.equal(y, want)
        del junk


def test_no_second_derivative(fp4):
    layer = fp4.FP4Linear(96, 48, device="cuda")
    x = acts(5, 96, seed=1).requires_grad_()
    dx, = torch.autograd.grad(layer(x).float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.float().sum().backward()


@FMTS
def test_linear_of_nothing(ops, fmt):
    x, w = acts(40, 64, seed=1), acts(16, 64, seed=2)
    own = ops.FP4_OWN_SCALE if fmt == 0 else None
    for m in (0, 3, 40):
        for scale in (None, own):
            assert ops.fp4_linear(x[:m], ops.fp4_cast(w[:0], fmt), scale).shape == (m, 0)
            d = ops.fp4_linear(x[:m, :0], ops.fp4_cast(w[:, :0], fmt), scale)
            assert d.shape == (m, 16) and bool((d == 0).all())
    off = torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda")
    assert ops.fp4_linear(x[:3], ops.fp4_cast(torch.stack([w, w])[:, :0], fmt), None, off).shape == (3, 0)
    d, cols = ops.fp4_linear_saving(x[:0], ops.fp4_cast(w, fmt), own)
    dx, dw = ops.fp4_linear_backward(acts(0, 16, seed=3), ops.fp4_cast_dual(w, fmt, own)[1], cols, own)
    assert d.shape == (0, 16) and dx.shape == (0, 64) and bool((dw == 0).all()) and dw.shape == (16, 64)
