"""The exchange of rows with the experts: plans equal to a sort, rows moved as they are,
weighted sums and gradients against 64 bits."""
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


def experts_of(m, k, n, seed=0, none=0.1, some=None):
    g = torch.Generator().manual_seed(seed)
    e = torch.randint(0, n, (m, k), generator=g)
    if some is not None:
        e = torch.tensor(some)[torch.randint(0, len(some), (m, k), generator=g)]
    e[torch.rand((m, k), generator=g) < none] = -1
    return e.to(torch.int32).cuda()


def rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def sorted_plan(e, n):
    flat = torch.where(e < 0, n, e).flatten().long()
    order = torch.sort(flat, stable=True)[1]
    rows = torch.empty_like(order)
    rows[order] = torch.arange(len(order), device=e.device)
    rows[flat == n] = -1
    ends = torch.bincount(flat, minlength=n + 1)[:n].cumsum(0)
    return torch.nn.functional.pad(ends, (1, 0)).int(), rows.view(e.shape).int()


@pytest.mark.parametrize("m,k,n", [(1, 1, 1), (1, 8, 256), (3, 2, 5), (31, 1, 8), (33, 3, 31), (128, 8, 512), (129, 8, 33), (1000, 1, 64),
                                   (1024, 1, 7), (1025, 1, 7), (500, 9, 511), (4096, 8, 256), (16384, 8, 160), (16391, 8, 512), (70000, 2, 8)])
@pytest.mark.parametrize("none", [0.0, 0.1, 1.0])
def test_plans(ops, m, k, n, none):
    e = experts_of(m, k, n, m + k + n, none)
    p = ops.expert_plan(e, n)
    offsets, rows = sorted_plan(e, n)
    assert torch.equal(p.offsets, offsets) and torch.equal(p.rows, rows)
    if m * k <= 300:
        assert ref.plan(e, n) == (p.offsets.tolist(), p.rows.flatten().tolist())
    assert ops.device_status() == 0


def test_plans_of_uneven_loads(ops):
    for some in ([3], [0, 63], [5, 5, 5, 5, 5, 9], [63]):
        for m in (40, 3000, 40000):
            e = experts_of(m, 2, 64, m, 0.0, some)
            p = ops.expert_plan(e, 64)
            offsets, rows = sorted_plan(e, 64)
            assert torch.equal(p.offsets, offsets) and torch.equal(p.rows, rows)


def test_indices_that_name_no_expert_are_left_out_and_reported(ops):
    e = torch.tensor([[0, 5], [9, 2], [-2, 1]], dtype=torch.int32, device="cuda")
    p = ops.expert_plan(e, 5)
    assert ops.device_status() == 1 and ops.device_status() == 0
    assert p.offsets.tolist() == [0, 1, 2, 3, 3, 3] and p.rows.tolist() == [[0, -1], [-1, 2], [-1, 1]]


def check(ops, x, e, n, weights, ys, dy, dxs, add=None):
    p = ops.expert_plan(e, n)
    m, k = e.shape
    rows, used = p.rows.cpu().long(), int(p.offsets[-1])
    xs = ops.expert_dispatch(x, p)
    want = torch.zeros((m * k, x.shape[1]), dtype=x.dtype)
    tok = torch.arange(m)[:, None].expand(m, k)
    on = rows >= 0
    want[rows[on]] = x.cpu()[tok[on]]
    assert torch.equal(xs.cpu(), want)
    assert used == int(on.sum())

    def gather(a):
        a = a.detach().cpu().double()
        return torch.where(on[:, :, None], a[rows.clamp(min=0)], torch.zeros((), dtype=torch.float64))
    w = weights.cpu().double()
    y = ops.expert_combine(ys, p, weights, add)
    terms = gather(ys) * torch.where(on, w, torch.zeros((), dtype=torch.float64))[:, :, None]
    base = torch.zeros((m, ys.shape[1]), dtype=torch.float64) if add is None else add.detach().cpu().double()
    total = base + terms.sum(1)
    mag = base.abs() + terms.abs().sum(1)
    assert y.dtype == ys.dtype
    ref.close(y, total, (k + 1) * ref.U * mag + ref.HALF[ys.dtype] * total.abs() * (1 + 2 ** -7), "y")
    one = gather(dxs)
    dx = ops.expert_combine(dxs, p)
    ref.close(dx, one.sum(1), (k + 1) * ref.U * one.abs().sum(1) + ref.HALF[dxs.dtype] * one.sum(1).abs() * (1 + 2 ** -7), "dx")
    dys, dw = ops.expert_combine_backward(dy, ys, p, weights)
    g = dy.detach().cpu().double()
    want = torch.zeros((m * k, ys.shape[1]), dtype=torch.float64)
    want[rows[on]] = (g[:, None] * w[:, :, None])[on]
    ref.close(dys, want, (ref.HALF[ys.dtype] + 2 * ref.U) * want.abs(), "dys")
    prod = gather(ys) * g[:, None]
    ref.close(dw, prod.sum(2), (ys.shape[1] // 128 + 20) * ref.U * prod.abs().sum(2), "dw")
    assert (dys[used:] == 0).all() and (dw.cpu()[~on] == 0).all()
    assert ops.device_status() == 0


@pytest.mark.parametrize("m,k,n,cols", [(1, 1, 1, 1), (1, 8, 256, 7168), (3, 2, 5, 33), (17, 8, 512, 1003), (64, 9, 31, 520), (5, 17, 8, 4096),
                                        (200, 2, 8, 776), (33, 6, 160, 2050), (2, 33, 40, 96)])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("none", [0.0, 0.3, 1.0])
def test_rows(ops, m, k, n, cols, dtype, none):
    e = experts_of(m, k, n, m + cols, none)
    check(ops, rand((m, cols), dtype, 1), e, n, rand((m, k), F, 2), rand((m * k, cols), dtype, 3), rand((m, cols), dtype, 4),
          rand((m * k, cols), dtype, 5), rand((m, cols), dtype, 6) if none else None)


@pytest.mark.parametrize("dtype", [BF, F])
def test_strides(ops, dtype):
    m, k, n = 12, 3, 7
    e = experts_of(m, k, n, 3)
    for cols, cut in ((64, slice(0, 64)), (64, slice(1, 65)), (63, slice(8, 71)), (64, slice(4, 68)), (32, slice(0, 64, 2))):
        wide = [rand((r, 80), dtype, s)[:, cut] for r, s in ((m, 1), (m * k, 2), (m, 3), (m * k, 4), (m, 5))]
        check(ops, wide[0], e, n, rand((m, k), F, 2), wide[1], wide[2], wide[3], wide[4])
    one = torch.full((1, 1), 0.5, dtype=dtype, device="cuda").expand(m, 64)        # the gradient of a sum
    check(ops, rand((1, 64), dtype, 1).expand(m, 64), e, n, rand((m, k), F, 2), rand((m * k, 64), dtype, 3), one, rand((m * k, 64), dtype, 4))


def test_outs_are_written_and_nothing_else(ops):
    m, k, n = 10, 3, 6
    p = ops.expert_plan(experts_of(m, k, n, 3), n)
    for cols in (64, 63):
        x, ys = rand((m, cols), BF, 1), rand((m * k, cols), BF, 2)
        room = torch.full((m * k + 2, 80), 7.0, dtype=BF, device="cuda")
        view = room[1:m * k + 1, 8:8 + cols]
        assert ops.expert_dispatch(x, p, out=view).data_ptr() == view.data_ptr()
        assert torch.equal(view, ops.expert_dispatch(x, p))
        view.fill_(7.0)
        assert torch.equal(room, torch.full_like(room, 7.0))
        view = room[1:m + 1, 8:8 + cols]
        ops.expert_combine(ys, p, out=view)
        assert torch.equal(view, ops.expert_combine(ys, p))
        view.fill_(7.0)
        assert torch.equal(room, torch.full_like(room, 7.0))


def test_rows_of_no_expert_have_no_influence(ops):
    """Whatever stands past the last expert's rows, and the weights of slots without one."""
    m, k, n, cols = 20, 4, 6, 136
    e = experts_of(m, k, n, 5, 0.4)
    p = ops.expert_plan(e, n)
    used = int(p.offsets[-1])
    ys, w, dy = rand((m * k, cols), BF, 1), rand((m, k), F, 2), rand((m, cols), BF, 3)
    clean = ops.expert_combine(ys, p, w), *ops.expert_combine_backward(dy, ys, p, w)
    ys[used:] = float("nan")
    w[e < 0] = float("inf")
    for a, b in zip(clean, (ops.expert_combine(ys, p, w), *ops.expert_combine_backward(dy, ys, p, w))):
        assert torch.equal(a, b)


def test_nothing_to_do(ops):
    p = ops.expert_plan(torch.empty((0, 3), dtype=torch.int32, device="cuda"), 5)
    assert p.offsets.tolist() == [0] * 6 and p.rows.shape == (0, 3)
    x = torch.empty((0, 16), dtype=BF, device="cuda")
    assert ops.expert_dispatch(x, p).shape == (0, 16) and ops.expert_combine(x, p).shape == (0, 16)
    assert ops.expert_combine_backward(x, x, p, torch.empty((0, 3), device="cuda"))[1].shape == (0, 3)
    p = ops.expert_plan(torch.zeros((4, 2), dtype=torch.int32, device="cuda"), 3)
    x = torch.empty((8, 0), dtype=BF, device="cuda")
    assert ops.expert_combine(x, p).shape == (4, 0)
    assert not ops.expert_combine_backward(x[:4], x, p, torch.ones((4, 2), device="cuda"))[1].any()


@pytest.mark.parametrize("m,k,n,apart", [(2500, 2, 520, 1 << 19), (2500, 2, 521, (1 << 19) + 1), (600, 8, 2048, 1 << 19)])
def test_rows_past_32_bits(ops, m, k, n, apart):
    """Rows far apart equal the same rows side by side."""
    def far(rows):
        return torch.empty((rows - 1) * apart + n, dtype=BF, device="cuda").as_strided((rows, n), (apart, 1))
    p = ops.expert_plan(experts_of(m, k, 16), 16)
    x, ys, dy, w = rand((m, n), BF, 1), rand((m * k, n), BF, 2), rand((m, n), BF, 3), rand((m, k), F, 4)
    there = far(m * k)
    assert torch.equal(ops.expert_dispatch(x, p, out=there), ops.expert_dispatch(x, p))
    there.copy_(ys)
    assert torch.equal(ops.expert_combine(there, p, w, x), ops.expert_combine(ys, p, w, x))
    for a, b in zip(ops.expert_combine_backward(dy, there, p, w), ops.expert_combine_backward(dy, ys, p, w)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("m,k,n", [(5, 2, 40), (5, 2, 41), (2500, 2, 520), (600, 8, 2048)])
def test_sums_onto_what_they_are_added_to(ops, m, k, n):
    p = ops.expert_plan(experts_of(m, k, 16), 16)
    ys, add, w = rand((m * k, n), BF, 2), rand((m, n), BF, 3), rand((m, k), F, 4)
    want = ops.expert_combine(ys, p, w, add)
    assert torch.equal(ops.expert_combine(ys, p, w, add, out=add), want) and torch.equal(add, want)


@pytest.mark.parametrize("m,k,n,dtype", [(2500, 8, 2048, BF), (2500, 7, 2040, BF), (2600, 4, 1000, BF), (2433, 3, 1024, F), (400, 8, 7168, BF), (305, 5, 8200, F),
                                         (2500, 2, 2048, BF), (2500, 1, 264, BF)])
def test_many_tokens_take_the_same_sums(ops, m, k, n, dtype):
    """Whole vectors of many tokens against rows off their boundaries, whose elements go one by
    one: the same terms in the same order."""
    p = ops.expert_plan(experts_of(m, k, 16, none=0.2), 16)
    ys, add, w = rand((m * k, n), dtype, 2), rand((m, n), dtype, 3), rand((m, k), F, 4)
    room = torch.empty((m * k, n + 1), dtype=dtype, device="cuda")
    room[:, 1:].copy_(ys)
    for ww in (w, None):
        assert torch.equal(ops.expert_combine(ys, p, ww, add), ops.expert_combine(room[:, 1:], p, ww, add))
    assert torch.equal(ops.expert_combine_backward(add, ys, p, w)[0], ops.expert_combine_backward(add, room[:, 1:], p, w)[0])
