"""Layer norm and its gradients against 64 bits."""
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantised_linear_layers_gb300 import ops
    return ops


def acts(m, n, dtype, seed=0, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, n), generator=g) * (1 + 15 * (torch.rand((1, n), generator=g) < 0.01))
    return ((x + offset * torch.randn((m, 1), generator=g)) * torch.exp2(torch.randint(-2, 3, (m, 1), generator=g))).to(dtype).cuda()


def params(n, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.2 * torch.randn(n, generator=g)).to(dtype).cuda(), (0.1 * torch.randn(n, generator=g)).to(dtype).cuda()


def check(ops, x, w, b, out, eps=1e-5, dy=None):
    y, tol, _, mean, rstd, _ = ref.norm(x, w, b, eps, out)
    got = ops.layer_norm(x, w, b, eps, dtype=out)
    assert got.dtype == out
    ref.close(got, y, tol, "y")
    again, stats = ops.layer_norm_saving(x, w, b, eps, dtype=out)
    assert torch.equal(again, got)
    c = ref.adds(x.shape[1])
    std = torch.sqrt(1 / rstd ** 2)
    ref.close(stats[0][:, None], mean, ref.U * (2 * mean.abs() + c * std), "mean")
    ref.close(stats[1][:, None], rstd, ref.U * (c + 6) * rstd, "rstd")
    if dy is None:
        g = torch.Generator().manual_seed(7)
        dy = (1e-3 * torch.randn(x.shape, generator=g)).to(out).cuda()
    want = ref.norm_backward(dy, x, w, eps, x.dtype)
    dx, dw, db = ops.layer_norm_backward(dy, x, stats, w, sums=True)
    assert dx.dtype == x.dtype and dw.dtype == db.dtype == F
    ref.close(dx, *want["dx"], "dx")
    ref.close(dw, *want["dw"], "dw")
    ref.close(db, *want["db"], "db")
    assert torch.equal(ops.layer_norm_backward(dy, x, stats, w, sums=False)[0], dx)
    for a, c in zip(ops.layer_norm_backward(dy, x, stats, w, sums=True), (dx, dw, db)):
        assert torch.equal(a, c)                       # the same sums in the same order
    assert ops.device_status() == 0


SIZES = [(1, 1), (1, 2), (3, 7), (5, 31), (2, 32), (7, 33), (300, 64), (130, 257), (9, 1000), (33, 1003), (40, 2048), (3, 2056),
         (17, 4099), (5, 7168), (700, 776), (2, 8192), (3, 8200), (2, 16384), (2, 16391), (1, 40000), (1300, 96), (2000, 1032),
         (1501, 1027)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("x_dtype,out", [(BF, BF), (F, F), (F, BF), (BF, F)])
def test_sizes(ops, m, n, x_dtype, out):
    w, b = params(n, F)
    check(ops, acts(m, n, x_dtype, m + n), w, b, out, eps=1e-5 if n > 1 else 1.0)


@pytest.mark.parametrize("n", [776, 1003])
@pytest.mark.parametrize("w_dtype", [BF, F])
def test_weights_are_optional(ops, n, w_dtype):
    x = acts(37, n, BF)
    w, b = params(n, w_dtype)
    for ww, bb in ((None, None), (w, None), (None, b), (w, b)):
        check(ops, x, ww, bb, BF)


@pytest.mark.parametrize("n", [64, 1003, 4096])
@pytest.mark.parametrize("dtype", [BF, F])
def test_strides(ops, n, dtype):
    wide = acts(12, 2 * n + 24, dtype)
    w, b = params(n, F)
    for x in (wide[:, :n], wide[:, 1:n + 1], wide[:, 8:n + 8], wide[::2, 3:n + 3], wide[:, ::2][:, :n], wide[:1].expand(5, -1)[:, :n],
              wide.t()[:n].t()):
        check(ops, x, w, b, dtype)
    # a gradient of a sum: every row the same memory
    x = wide[:, :n]
    one = torch.full((1, 1), 1e-3, dtype=dtype, device="cuda").expand(12, n)
    check(ops, x, w, b, dtype, dy=one)
    # weights that start off a 16-byte boundary
    ww, bb = params(n + 3, F)
    check(ops, x.contiguous(), ww[1:n + 1], bb[3:n + 3], dtype)


def test_out_is_written_and_nothing_else(ops):
    x = acts(6, 776, BF)
    w, b = params(776, F)
    for dtype in (BF, F):
        for first in (8, 5):                           # on a 16-byte boundary, where sums run in the order of the new tensor's, and off it
            room = torch.full((8, 800), 7.0, dtype=dtype, device="cuda")
            view = room[1:7, first:first + 776]
            got = ops.layer_norm(x, w, b, out=view)
            assert got.data_ptr() == view.data_ptr() and got.dtype == dtype
            ref.close(view, *ref.norm(x, w, b, 1e-5, dtype)[:2], "y")
            assert first != 8 or torch.equal(view, ops.layer_norm(x, w, b, dtype=dtype))
            view.fill_(7.0)
            assert torch.equal(room, torch.full_like(room, 7.0))


@pytest.mark.parametrize("n", [8, 1003, 7168])
def test_rows_far_from_zero(ops, n):
    """A mean of 4096 deviations: what the first sum rounds off is put right by the second."""
    g = torch.Generator().manual_seed(3)
    x = (4096 + torch.randn((4, n), generator=g)).cuda()
    w, b = params(n, F)
    check(ops, x, w, b, F)


def test_constant_rows_and_eps(ops):
    x = torch.full((3, 64), 2.5, device="cuda")
    assert torch.equal(ops.layer_norm(x), torch.zeros_like(x))
    assert torch.isnan(ops.layer_norm(x, eps=0.0)).all()          # 0 / 0
    check(ops, acts(4, 64, F), None, None, F, eps=0.0)
    check(ops, acts(4, 64, F), None, None, F, eps=3.0)


@pytest.mark.parametrize("n", [40, 1003, 7168])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_is_not_finite_stays_in_its_row(ops, n, bad):
    x = acts(5, n, BF)
    clean = ops.layer_norm(x)
    x[2, n // 2] = bad
    y, stats = ops.layer_norm_saving(x)
    assert torch.isnan(y[2]).all()
    keep = [0, 1, 3, 4]
    assert torch.equal(y[keep], clean[keep])
    dx, _, _ = ops.layer_norm_backward(torch.ones_like(x), x, stats)
    assert torch.isnan(dx[2]).all() and torch.isfinite(dx[keep]).all()


def test_nothing_to_do(ops):
    w, b = params(64, F)
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    y, stats = ops.layer_norm_saving(x, w, b)
    assert y.shape == (0, 64) and stats.shape == (2, 0)
    dx, dw, db = ops.layer_norm_backward(x, x, stats, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    x = torch.empty((5, 0), dtype=BF, device="cuda")
    y, stats = ops.layer_norm_saving(x)
    assert y.shape == (5, 0)
    assert ops.layer_norm_backward(x, x, stats, sums=True)[1].shape == (0,)


@pytest.mark.parametrize("n", [24, 100])
def test_gradients_against_differences(ops, n):
    """d/dx and d/dw of <y, v> by central differences of the 64-bit formula."""
    x, v = acts(3, n, F, 5), acts(3, n, F, 6)
    w, b = params(n, F)
    _, stats = ops.layer_norm_saving(x, w, b)
    dx, dw, db = ops.layer_norm_backward(v, x, stats, w)

    def f(x, w, b):
        return (ref.norm(x, w, b, 1e-5, F)[0] * v.cpu().double()).sum(1)
    step = 1e-5
    xd, wd, bd = x.cpu().double(), w.cpu().double(), b.cpu().double()
    for i in range(0, n, 7):
        e = torch.zeros(n, dtype=torch.float64)
        e[i] = step
        for got, d in ((dx[:, i].cpu().double(), (f(xd + e, wd, bd) - f(xd - e, wd, bd)) / (2 * step)),
                       (dw[i].cpu().double(), (f(xd, wd + e, bd) - f(xd, wd - e, bd)).sum() / (2 * step)),
                       (db[i].cpu().double(), (f(xd, wd, bd + e) - f(xd, wd, bd - e)).sum() / (2 * step))):
            # differences of values of size ~1e3 in 64 bits over 2e-5, and fp32's own 1e-5
            assert torch.allclose(got, d, rtol=2e-5, atol=1e-4 * float(v.abs().max()))


@pytest.mark.parametrize("m,n,dtype", [(5, 40, BF), (3, 7168, BF), (2000, 1032, BF), (2000, 1027, F), (2000, 1027, BF), (2, 16391, F)])
def test_in_place(ops, m, n, dtype):
    w, b = params(n, F)
    x = acts(m, n, dtype)
    y = ops.layer_norm(x, w, b)
    assert ops.layer_norm(x, w, b, out=x).data_ptr() == x.data_ptr()
    assert torch.equal(x, y)


def test_statistics_of_what_has_none(ops):
    x = acts(4, 1003, F)
    x[1, 5] = float("nan")
    _, stats = ops.layer_norm_saving(x)
    assert torch.isnan(stats[:, 1]).all() and torch.isfinite(stats[:, [0, 2, 3]]).all()
    _, stats = ops.layer_norm_saving(torch.empty((5, 0), device="cuda"))
    assert torch.isnan(stats).all()


@pytest.mark.parametrize("n", [7168, 264])
def test_rows_past_32_bits(ops, n):
    """Rows 2^20 elements apart equal the same rows side by side."""
    m = 2049
    room = [torch.empty((m - 1 << 20) + n, dtype=BF, device="cuda").as_strided((m, n), (1 << 20, 1)) for _ in range(3)]
    x, dy, y = room
    x.copy_(acts(m, n, BF))
    dy.copy_(acts(m, n, BF, 1))
    w, b = params(n, F)
    want, stats = ops.layer_norm_saving(x.contiguous(), w, b)
    got, far = ops.layer_norm_saving(x, w, b, out=y)
    assert torch.equal(got, want) and torch.equal(far, stats)
    for a, c in zip(ops.layer_norm_backward(dy, x, stats, w), ops.layer_norm_backward(dy.contiguous(), x.contiguous(), stats, w)):
        assert torch.equal(a, c)


@pytest.mark.parametrize("m,n", [(700, 1003), (1300, 520), (2000, 261), (400, 8201)])
@pytest.mark.parametrize("x_dtype,out", [(BF, BF), (F, F), (F, BF), (BF, F)])
def test_many_rows_that_start_anywhere(ops, m, n, x_dtype, out):
    """x and dy with starts of their own, alike in all rows or in none, and the first and the last
    element of their memory among them."""
    w, b = params(n, F)
    for i, (x_first, x_wide, dy_first, dy_wide) in enumerate(((1, n + 1, 0, n), (0, n, 1, n + 1), (3, n + 8 - n % 8, 5, n + 9), (7, n + 7, 7, n + 7))):
        x, dy = (torch.empty(f + (m - 1) * s + n, dtype=d, device="cuda")[f:].as_strided((m, n), (s, 1), f)
                 for f, s, d in ((x_first, x_wide, x_dtype), (dy_first, dy_wide, out)))
        x.copy_(acts(m, n, x_dtype, i))
        dy.copy_(1e-3 * acts(m, n, out, i + 9))
        check(ops, x, w, b, out, dy=dy)


@pytest.mark.parametrize("n", [(1 << 20) + 3, 1 << 22])
@pytest.mark.parametrize("x_dtype,out", [(BF, BF), (F, F), (F, BF), (BF, F)])
def test_sums_of_long_rows_stay_exact(ops, n, x_dtype, out):
    """Rows whose terms all err the same way: errors that do not grow with the row's length. A term
    passes a run of 64 and two trees of 32."""
    c = 80
    g = torch.Generator().manual_seed(1)
    x = (torch.where(torch.rand((2, n), generator=g) < 0.5, -1.1, 1.1) + torch.tensor([[0.3], [300.0]])).to(x_dtype).cuda()
    dy = (1.1e-3 + 1e-5 * torch.randn((2, n), generator=g)).to(out).cuda()
    y, stats = ops.layer_norm_saving(x, dtype=out)
    want, tol, _, mean, rstd, _ = ref.norm(x, None, None, 1e-5, out, c)
    ref.close(y, want, tol, "y")
    ref.close(stats[0][:, None], mean, ref.U * (2 * mean.abs() + c / rstd), "mean")
    ref.close(stats[1][:, None], rstd, ref.U * (c + 6) * rstd, "rstd")
    dx, _, _ = ops.layer_norm_backward(dy, x, stats)
    ref.close(dx, *ref.norm_backward(dy, x, None, 1e-5, x_dtype, c)["dx"], "dx")


def test_sums_of_many_long_rows_stay_exact(ops):
    """The gradients of weight and bias over 65536 rows alike: a term passes a run of 64 and the joins of
    at most 10 parts."""
    m, n, c = 65536, 16391, 80
    x = acts(1, n, F)
    dy = torch.full((1, n), 1.1e-3, device="cuda")
    _, stats = ops.layer_norm_saving(x)
    _, dw, db = ops.layer_norm_backward(dy.to(BF).expand(m, n), x.to(BF).expand(m, n), stats.expand(2, m).contiguous(), sums=True)
    v = dy.to(BF).cpu().double()
    h = (x.to(BF).cpu().double() - stats[0].cpu().double()) * stats[1].cpu().double()
    # two roundings of h, one of the product
    ref.close(db[None], m * v, c * ref.U * m * v, "db")
    ref.close(dw[None], m * v * h, (c + 3) * ref.U * m * v * h.abs(), "dw")


def test_an_infinity_in_long_rows_stays_one(ops):
    m, n = 300, 16400
    x, dy = acts(m, n, F), torch.ones((m, n), device="cuda")
    dy[7, 3], dy[9, 5] = float("inf"), float("nan")
    _, stats = ops.layer_norm_saving(x)
    dx, _, db = ops.layer_norm_backward(dy, x, stats, sums=True)
    assert db[3] == float("inf") and torch.isnan(db[5]) and torch.equal(db[10:], torch.full_like(db[10:], m))
    bad = torch.zeros(m, dtype=torch.bool, device="cuda")
    bad[[7, 9]] = True
    assert not torch.isfinite(dx[bad]).any() and torch.isfinite(dx[~bad]).all()       # g - mean(g) - h mean(g h): NaN or an infinity
