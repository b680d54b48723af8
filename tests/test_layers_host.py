"""Layer norm, routing and the exchange with the experts without a GPU: sizes, and the
refusals of the C entry points and of the calls over tensors; the reference against closed
forms."""
import ctypes
import math

import pytest
import torch

import layer_reference as ref

INV, UNS, ALI = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from quantised_linear_layers_gb300 import build, ops
    build.build()
    return ops.load_library()


P = ctypes.c_void_p(64)
Q = ctypes.c_void_p(72)


def test_workspaces(L):
    assert L.expert_plan_workspace_size(0, 8) == L.expert_plan_workspace_size(1024, 512) == 0
    assert L.expert_plan_workspace_size(1025, 8) == 2 * 8 * 4
    assert L.expert_plan_workspace_size(131072, 256) == 128 * 256 * 4
    assert L.layer_norm_backward_workspace_size(0, 64) == L.layer_norm_backward_workspace_size(64, 0) == 0
    assert L.layer_norm_backward_workspace_size(1, 64) >= 2 * 64 * 4
    # parts stop growing with the rows
    assert L.layer_norm_backward_workspace_size(1 << 20, 64) == L.layer_norm_backward_workspace_size(1 << 24, 64)


def test_layer_norm_refuses(L):
    def f(x=P, xt=0, m=4, n=64, sx=64, w=P, b=P, wt=1, eps=1e-5, y=P, yt=0, sy=64, mean=None, rstd=None):
        return L.layer_norm(x, xt, m, n, sx, w, b, wt, eps, y, yt, sy, mean, rstd, None)
    assert f(xt=2) == f(yt=3) == f(wt=7) == f(m=-1) == f(n=-1) == f(eps=-1.0) == f(eps=math.nan) == INV
    assert f(x=None) == f(y=None) == f(sy=63) == f(mean=P) == f(rstd=P) == INV
    assert f(m=1 << 31) == f(n=1 << 31) == UNS
    assert f(m=0, x=None, y=None) == f(n=0, x=None, y=None) == 0


def test_layer_norm_backward_refuses(L):
    def f(dy=P, dt=0, sdy=64, x=P, xt=0, sx=64, mean=P, rstd=P, w=P, wt=1, m=4, n=64, dx=P, sdx=64, dw=P, db=P, ws=P, size=1 << 20):
        return L.layer_norm_backward(dy, dt, sdy, x, xt, sx, mean, rstd, w, wt, m, n, dx, sdx, dw, db, ws, size, None)
    assert f(dt=2) == f(xt=2) == f(wt=2) == f(m=-1) == f(n=-1) == INV
    assert f(dy=None) == f(x=None) == f(mean=None) == f(rstd=None) == f(dx=None) == f(sdx=63) == INV
    assert f(dw=None) == f(db=None) == f(ws=None) == f(size=8) == INV
    assert f(ws=Q) == ALI
    assert f(m=1 << 31) == f(n=1 << 31) == UNS
    assert f(n=0, dy=None) == f(m=0, dw=None, db=None, dy=None) == 0


def test_route_refuses(L):
    def f(l=P, t=1, m=4, n=16, s=16, bias=None, k=2, score=0, groups=1, kept=1, best=1, re=1, scale=1.0, w=P, e=P):
        return L.expert_route(l, t, m, n, s, bias, k, score, groups, kept, best, re, scale, w, e, None)
    assert f(t=2) == f(m=-1) == f(n=0) == f(k=0) == f(k=17) == f(score=2) == f(score=-1) == INV
    assert f(groups=0) == f(groups=3) == f(groups=4, kept=5) == f(kept=0) == f(best=0) == f(best=3) == INV
    assert f(l=None) == f(w=None) == f(e=None) == INV
    assert f(n=513) == f(n=512, k=33) == f(n=512, groups=64) == f(m=1 << 31) == UNS
    assert f(m=0, l=None, w=None, e=None) == 0

    def b(dw=P, l=P, t=1, m=4, n=16, s=16, e=P, k=2, score=0, re=1, scale=1.0, d=P, sd=16):
        return L.expert_route_backward(dw, l, t, m, n, s, e, k, score, re, scale, d, sd, None)
    assert b(t=2) == b(m=-1) == b(n=0) == b(k=0) == b(k=17) == b(score=2) == INV
    assert b(dw=None) == b(l=None) == b(e=None) == b(d=None) == b(sd=15) == INV
    assert b(n=513) == b(n=512, k=33) == UNS
    assert b(m=0, dw=None) == 0


def test_exchange_refuses(L):
    def plan(e=P, slots=8, n=4, o=P, r=P, ws=None, size=0):
        return L.expert_plan(e, slots, n, o, r, ws, size, None)
    assert plan(slots=-1) == plan(n=0) == plan(e=None) == plan(o=None) == plan(r=None) == plan(slots=2000) == INV
    assert plan(slots=2000, ws=P, size=31) == INV and plan(slots=2000, ws=Q, size=32) == ALI
    assert plan(n=513) == plan(slots=(1 << 26) + 1) == UNS

    def there(x=P, t=0, m=4, n=64, sx=64, r=P, o=P, e=8, k=2, xs=P, s=64):
        return L.expert_dispatch(x, t, m, n, sx, r, o, e, k, xs, s, None)
    assert there(t=2) == there(m=-1) == there(n=-1) == there(k=0) == there(e=0) == INV
    assert there(x=None) == there(r=None) == there(o=None) == there(xs=None) == there(s=63) == INV
    assert there(m=1 << 31) == there(n=(1 << 22) + 1) == there(m=1 << 20, k=65) == there(e=513) == UNS
    assert there(m=0, x=None) == there(n=0, x=None) == 0

    def back(ys=P, t=0, s=64, r=P, w=P, a=None, sa=0, m=4, n=64, k=2, y=P, sy=64):
        return L.expert_combine(ys, t, s, r, w, a, sa, m, n, k, y, sy, None)
    assert back(t=2) == back(m=-1) == back(k=0) == back(ys=None) == back(r=None) == back(y=None) == back(sy=63) == INV
    assert back(m=1 << 20, k=65) == UNS
    assert back(m=0, ys=None) == 0

    def grad(dy=P, t=0, sdy=64, ys=P, sys=64, r=P, o=P, e=8, w=P, m=4, n=64, k=2, dys=P, s=64, dw=P):
        return L.expert_combine_backward(dy, t, sdy, ys, sys, r, o, e, w, m, n, k, dys, s, dw, None)
    assert grad(t=2) == grad(m=-1) == grad(k=0) == grad(e=0) == grad(dw=None) == INV
    assert grad(dy=None) == grad(ys=None) == grad(r=None) == grad(o=None) == grad(w=None) == grad(dys=None) == grad(s=63) == INV
    assert grad(e=513) == UNS
    assert grad(m=0, dw=None) == 0


def test_elements_off_their_boundaries_are_refused(L):
    odd, two = ctypes.c_void_p(65), ctypes.c_void_p(66)

    def norm(x=P, w=P, b=P, y=P, mean=P, rstd=P):
        return L.layer_norm(x, 0, 4, 64, 64, w, b, 1, 1e-5, y, 1, 64, mean, rstd, None)
    assert norm(x=odd) == norm(w=two) == norm(b=two) == norm(y=two) == norm(mean=two) == norm(rstd=two) == ALI

    def back(dy=P, x=P, mean=P, rstd=P, w=P, dx=P, dw=P, db=P):
        return L.layer_norm_backward(dy, 1, 64, x, 0, 64, mean, rstd, w, 0, 4, 64, dx, 64, dw, db, P, 1 << 20, None)
    assert back(dy=two) == back(x=odd) == back(mean=two) == back(rstd=two) == back(w=odd) == back(dx=odd) == back(dw=two) == back(db=two) == ALI

    def route(l=P, bias=None, w=P, e=P):
        return L.expert_route(l, 0, 4, 16, 16, bias, 2, 0, 1, 1, 1, 1, 1.0, w, e, None)
    assert route(l=odd) == route(bias=two) == route(w=two) == route(e=two) == ALI

    def route_back(dw=P, l=P, e=P, d=P):
        return L.expert_route_backward(dw, l, 0, 4, 16, 16, e, 2, 0, 1, 1.0, d, 16, None)
    assert route_back(dw=two) == route_back(l=odd) == route_back(e=two) == route_back(d=odd) == ALI
    for e, o, r in ((two, P, P), (P, two, P), (P, P, two)):
        assert L.expert_plan(e, 8, 4, o, r, None, 0, None) == ALI
    for x, r, o, xs in ((two, P, P, P), (P, two, P, P), (P, P, two, P), (P, P, P, two)):
        assert L.expert_dispatch(x, 1, 4, 64, 64, r, o, 8, 2, xs, 64, None) == ALI
    for ys, r, w, add, y in ((odd, P, P, P, P), (P, two, P, P, P), (P, P, two, P, P), (P, P, P, odd, P), (P, P, P, P, odd)):
        assert L.expert_combine(ys, 0, 64, r, w, add, 64, 4, 64, 2, y, 64, None) == ALI
    for i in range(7):
        p = [P] * 7
        p[i] = two
        dy, ys, r, o, w, dys, dw = p
        assert L.expert_combine_backward(dy, 1, 64, ys, 64, r, o, 8, w, 4, 64, 2, dys, 64, dw, None) == ALI


def test_calls_refuse_host_tensors(L):
    from quantised_linear_layers_gb300 import ops
    x, e = torch.zeros(4, 8), torch.zeros((4, 2), dtype=torch.int32)
    plan = ops.ExpertPlan(torch.zeros(5, dtype=torch.int32), e)
    for call in (lambda: ops.layer_norm(x), lambda: ops.layer_norm_saving(x), lambda: ops.layer_norm_backward(x, x, x),
                 lambda: ops.route(x, 2), lambda: ops.route_backward(x, x, e), lambda: ops.expert_plan(e, 4),
                 lambda: ops.expert_dispatch(x, plan), lambda: ops.expert_combine(x, plan),
                 lambda: ops.expert_combine_backward(x, x, plan, x), lambda: ops.layer_norm(x, dtype=torch.float16),
                 lambda: ops.route(x, 2, score="relu")):
        with pytest.raises(ValueError):
            call()


def test_modules_refuse():
    from quantised_linear_layers_gb300 import moe, norm
    for how in (dict(k=0), dict(k=9), dict(k=2, score="relu"), dict(k=2, groups=3), dict(k=2, groups=4, kept=5), dict(k=2, group_best=3)):
        with pytest.raises(ValueError):
            moe.Router(16, 8, **how)
    r = moe.Router(16, 8, 2)
    with pytest.raises(ValueError):
        r(torch.zeros(3, 15))
    with pytest.raises(ValueError):
        r.balance_step(None)
    with pytest.raises(ValueError):
        norm.LayerNorm(16)(torch.zeros(3, 15))
    with pytest.raises(TypeError):
        moe.FP4MoE(32, 32, 4, 2)(torch.zeros(3, 32))
    assert norm.LayerNorm(16, affine=False).weight is None and norm.LayerNorm(16, bias=False).bias is None


def test_forward_mode_is_refused():
    from torch.autograd import forward_ad
    from quantised_linear_layers_gb300 import moe, norm
    x = torch.ones(2, 4)
    with forward_ad.dual_level():
        d = forward_ad.make_dual(x, torch.ones_like(x))
        for call in (lambda: norm.layer_norm(d), lambda: norm.layer_norm(x, d[0]), lambda: moe.route(d, 1), lambda: moe.dispatch(d, None),
                     lambda: moe.combine(d, None, x), lambda: moe.combine(x, None, d), lambda: moe.combine(x, None, x, d)):
            with pytest.raises(NotImplementedError):
                call()


def test_reference_closed_forms():
    y = ref.norm(torch.tensor([[1.0, 3.0]]), None, None, 0.0, torch.float32)[0]
    assert torch.equal(y, torch.tensor([[-1.0, 1.0]], dtype=torch.float64))
    inf = math.inf
    l = torch.tensor([[1.0, 3.0, 3.0, -inf], [-inf] * 4, [0.0, 0.0, 0.0, 0.0]])
    assert ref.choose(l, 2).tolist() == [[1, 2], [-1, -1], [0, 1]]
    assert ref.choose(l, 4).tolist()[0] == [1, 2, 0, -1]
    assert ref.choose(l, 2, torch.tensor([9.0, 0.0, 0.0, 9.0]), "sigmoid").tolist() == [[0, 1], [-1, -1], [0, 3]]
    assert ref.choose(l, 2, groups=2, kept=1).tolist() == [[1, 0], [-1, -1], [0, 1]]
    w, _ = ref.route_weights(l, ref.choose(l, 2), "softmax", True, 3.0)
    assert torch.allclose(w, torch.tensor([[1.5, 1.5], [0.0, 0.0], [1.5, 1.5]], dtype=torch.float64))
    assert ref.plan(torch.tensor([[1, 0], [-1, 1]], dtype=torch.int32), 3) == ([0, 1, 3, 3], [1, 0, -1, 2])


def test_exchanges_of_more_blocks_than_a_grid_are_unsupported(L):
    """Rows for which no device has memory: refused as too large before any launch."""
    m, n = 1 << 26, 1 << 22
    assert L.expert_dispatch(P, 0, m, n, n, P, P, 8, 1, P, n, None) == UNS
    assert L.expert_combine(P, 0, n, P, None, None, 0, m, n, 1, P, n, None) == UNS
    assert L.expert_combine_backward(P, 0, n, P, n, P, P, 8, P, m, n, 1, P, n, P, None) == UNS
