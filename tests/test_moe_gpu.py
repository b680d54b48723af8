"""The operators around the experts together, as a layer uses them: with gradients, in the
layer of 4-bit experts, on other streams, in threads and in captured graphs."""
import copy
import threading

import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import types
    from quantised_linear_layers_gb300 import fp4, moe, norm, ops
    return types.SimpleNamespace(fp4=fp4, moe=moe, norm=norm, ops=ops)


def rand(shape, dtype, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def dense(x, gamma, beta, router, mix, experts, add, score, renormalise):
    """Norm, routing, experts that scale their rows and the sums back, in 64 bits for chosen experts."""
    n = x.shape[1]
    mean = x.mean(1, keepdim=True)
    h = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + 1e-5) * gamma + beta
    l = h @ router.t()
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    w = torch.gather(s, 1, experts)
    if renormalise:
        w = w / w.sum(1, keepdim=True)
    return add + (w[:, :, None] * (h[:, None] * mix[experts])).sum(1)


@pytest.mark.parametrize("m,n,e,k", [(1, 32, 4, 1), (33, 96, 8, 2), (40, 130, 20, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gradients_through_all_of_it(pkg, m, n, e, k, score, renormalise):
    """fp32 all along: every gradient within 2^-14 of its largest, where 64 bits differ from it
    by the bounds of the parts: routing's gradient 2^-17 of terms whose sums may cancel to an
    eighth, and less from sums of up to n terms (130 * 2^-24)."""
    leaves = dict(x=rand((m, n), F, 1), gamma=1 + rand((n,), F, 2, 0.2), beta=rand((n,), F, 3, 0.1), router=rand((e, n), F, 4, n ** -0.5),
                  mix=rand((e, n), F, 5), add=rand((m, n), F, 6))
    for t in leaves.values():
        t.requires_grad_()
    v = rand((m, n), F, 7)
    h = pkg.norm.layer_norm(leaves["x"], leaves["gamma"], leaves["beta"])
    weights, experts = pkg.moe.route(torch.nn.functional.linear(h, leaves["router"]), k, score=score, renormalise=renormalise)
    plan = pkg.ops.expert_plan(experts, e)
    xs = pkg.moe.dispatch(h, plan)
    order = torch.argsort(experts.flatten(), stable=True)
    ys = xs * leaves["mix"][experts.flatten()[order].long()]
    y = pkg.moe.combine(ys, plan, weights, leaves["add"])
    (y * v).sum().backward()
    wide = {name: t.detach().double().requires_grad_() for name, t in leaves.items()}
    want = dense(*(wide[c] for c in ("x", "gamma", "beta", "router", "mix")), experts.long(), wide["add"], score, renormalise)
    (want * v.double()).sum().backward()
    assert (y.detach() - want.detach()).abs().max() <= 2.0 ** -16 * want.detach().abs().max()
    for name, t in leaves.items():
        g, w = t.grad.double(), wide[name].grad
        if w.abs().max() < 1e-9:                        # one weight, renormalised: constant
            assert g.abs().max() < 1e-6
        else:
            assert (g - w).abs().max() <= 2.0 ** -14 * w.abs().max(), name


def test_what_needs_no_gradient_gets_none(pkg):
    x, w, b = rand((4, 32), F, 1), rand((32,), F, 2), rand((32,), F, 3)
    assert not pkg.norm.layer_norm(x, w, b).requires_grad
    for need in ((0,), (1,), (2,), (0, 1, 2)):
        ts = [t.clone().requires_grad_(i in need) for i, t in enumerate((x, w, b))]
        pkg.norm.layer_norm(*ts).sum().backward()
        assert [t.grad is not None for t in ts] == [i in need for i in range(3)]
    plan = pkg.ops.expert_plan(torch.zeros((4, 1), dtype=torch.int32, device="cuda"), 2)
    ys, g, add = rand((4, 32), F, 4), rand((4, 1), F, 5), rand((4, 32), F, 6)
    for need in ((0,), (1,), (2,), (0, 1, 2)):
        ts = [t.clone().requires_grad_(i in need) for i, t in enumerate((ys, g, add))]
        pkg.moe.combine(ts[0], plan, ts[1], ts[2]).sum().backward()
        assert [t.grad is not None for t in ts] == [i in need for i in range(3)]
    with torch.no_grad():
        assert not pkg.moe.dispatch(x.requires_grad_(), plan).requires_grad


def test_second_derivatives_are_refused(pkg):
    x = rand((4, 32), F, 1).requires_grad_()
    g, = torch.autograd.grad(pkg.norm.layer_norm(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def by_hand(pkg, layer, x):
    """FP4MoE's forward with torch's own sort between the same products."""
    h = pkg.ops.layer_norm(x, layer.norm.weight, layer.norm.bias, layer.norm.eps, dtype=BF)
    w, e = pkg.ops.route(torch.nn.functional.linear(h.float(), layer.router.weight), layer.router.k, layer.router.bias, **layer.router.how)
    n, k = layer.router.experts, layer.router.k
    flat = e.flatten().long()
    order = torch.argsort(flat, stable=True)
    offsets = torch.nn.functional.pad(torch.bincount(flat, minlength=n).cumsum(0), (1, 0)).to(torch.int32)
    gate, up = layer.up(h[order // k], offsets).chunk(2, -1)
    ys = layer.down(torch.nn.functional.silu(gate) * up, offsets)
    back = torch.empty_like(order)
    back[order] = torch.arange(len(order), device=x.device)
    mine = ys[back].view(*e.shape, -1).double() * w.double()[:, :, None]
    y = x.double() + mine.sum(1)
    return y, (k + 2) * ref.U * (x.double().abs() + mine.abs().sum(1)) + ref.HALF[BF] * (1 + 2 ** -7) * y.abs()


@pytest.mark.parametrize("tokens", [1, 7, 130])
@pytest.mark.parametrize("fmt", [0, 1])
def test_layer(pkg, tokens, fmt):
    torch.manual_seed(0)
    layer = pkg.moe.FP4MoE(64, 96, 8, 2, fmt, device="cuda", accumulate_main_grad=True, balance=True, score="sigmoid", groups=4, kept=2, group_best=2)
    x = rand((tokens, 64), BF, 1)
    with torch.no_grad():
        y = layer(x)
        ref.close(y, *by_hand(pkg, layer, x), "y")
    x.requires_grad_()
    y2 = layer(x[None])
    assert y2.shape == (1, tokens, 64)
    y2.square().mean().backward()
    for t in (x, layer.norm.weight, layer.norm.bias, layer.router.weight):
        assert t.grad is not None and torch.isfinite(t.grad).all() and t.grad.abs().max() > 0
    for part in (layer.up, layer.down):
        assert part.weight.grad is None and part.main_grad.abs().max() > 0
    load = layer.plan.offsets.diff()
    layer.router.balance_step(layer.plan, 0.5)
    assert torch.equal(layer.router.bias, 0.5 * torch.sign(load.float().mean() - load))
    twin = copy.deepcopy(layer)
    with torch.no_grad():
        assert torch.equal(twin(x), layer(x))
    layer.zero_grad()
    layer.to(BF)                                    # a model cast as a whole: every parameter in bf16
    y3 = layer(x)
    y3.float().square().mean().backward()
    assert torch.isfinite(y3).all() and layer.router.weight.grad.dtype == BF
    assert pkg.ops.device_status() == 0


def test_layer_without_tokens(pkg):
    layer = pkg.moe.FP4MoE(64, 32, 4, 2, device="cuda")
    with torch.no_grad():
        assert layer(torch.empty((0, 64), dtype=BF, device="cuda")).shape == (0, 64)


def test_layer_of_no_tokens_has_gradients(pkg):
    layer = pkg.moe.FP4MoE(64, 32, 4, 2, device="cuda")
    x = torch.empty((0, 64), dtype=BF, device="cuda", requires_grad=True)
    layer(x).sum().backward()
    assert x.grad.shape == (0, 64)
    for p in layer.parameters():
        assert p.grad is None or not p.grad.any()


@pytest.mark.parametrize("tokens", [1, 40])
def test_tokens_that_reach_no_expert_stay_as_they_are(pkg, tokens):
    layer = pkg.moe.FP4MoE(64, 32, 4, 2, device="cuda", balance=True)
    layer.router.bias.fill_(float("-inf"))
    x = rand((tokens, 64), BF, 1).requires_grad_()
    y = layer(x)
    assert torch.equal(y, x) and layer.plan.offsets.tolist() == [0] * 5
    y.sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x))
    for p in layer.parameters():
        assert p.grad is None or not p.grad.any()
    assert pkg.ops.device_status() == 0


def test_router_keeps_fp32_under_autocast(pkg):
    router = pkg.moe.Router(64, 16, 4, device="cuda")
    x = rand((50, 64), BF, 1)
    want = router(x)
    with torch.autocast("cuda", dtype=BF):
        got = router(x)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def calls(pkg, x, w, b, logits, bias, ys, dy, dw):
    ops = pkg.ops
    y, stats = ops.layer_norm_saving(x, w, b)
    dx, gw, gb = ops.layer_norm_backward(dy, x, stats, w)
    weights, experts = ops.route(logits, 4, bias, "sigmoid", 4, 2, 2)
    dl = ops.route_backward(dw, logits, experts, "sigmoid")
    p = ops.expert_plan(experts, logits.shape[1])
    xs = ops.expert_dispatch(x, p)
    out = ops.expert_combine(ys, p, weights, x)
    dys, dg = ops.expert_combine_backward(dy, ys, p, weights)
    return [y, stats, dx, gw, gb, weights, experts, dl, p.offsets, p.rows, xs, out, dys, dg, ops.expert_combine(xs, p)]


def inputs(m, n, seed):
    return [rand((m, n), BF, seed), rand((n,), F, seed + 1), rand((n,), F, seed + 2), rand((m, 64), F, seed + 3), rand((64,), F, seed + 4, 0.1),
            rand((m * 4, n), BF, seed + 5), rand((m, n), BF, seed + 6), rand((m, 4), F, seed + 7)]


@pytest.mark.parametrize("m,n", [(3, 64), (1000, 1032), (2500, 264)])
def test_captured_graphs_follow_their_inputs(pkg, m, n):
    """Two graphs of one pool, replayed in turn on other inputs than they were captured on."""
    at = inputs(m, n, 0)
    calls(pkg, *at)
    torch.cuda.synchronize()
    graphs, outs, pool = [], [], None
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(calls(pkg, *at))
        pool = g.pool()
        graphs.append(g)
    for seed in (10, 20):
        new = inputs(m, n, seed)
        for a, b in zip(at, new):
            a.copy_(b)
        want = [t.clone() for t in calls(pkg, *new)]
        for g, o in zip(graphs, outs):
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(o, want):
                assert torch.equal(a, b)


def captured_step(step):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    return g, out


@pytest.mark.parametrize("m,n", [(5, 96), (700, 1032)])
def test_a_captured_training_step(pkg, m, n):
    """Forward and gradients of norm, routing and the exchange in one graph, on new inputs."""
    def values(seed):
        return [rand((m, n), F, seed), 1 + rand((n,), F, seed + 1, 0.2), rand((n,), F, seed + 2, 0.1), rand((16, n), F, seed + 3, n ** -0.5), rand((n,), F, seed + 4)]
    leaves = [t.requires_grad_() for t in values(0)]

    def step():
        x, gamma, beta, router, mix = leaves
        h = pkg.norm.layer_norm(x, gamma, beta)
        weights, experts = pkg.moe.route(torch.nn.functional.linear(h, router), 4, score="sigmoid")
        plan = pkg.ops.expert_plan(experts, 16)
        y = pkg.moe.combine(pkg.moe.dispatch(h, plan) * mix, plan, weights, x)
        return [y.detach(), *torch.autograd.grad(y.square().mean(), leaves)]
    g, out = captured_step(step)
    for seed in (10, 20):
        with torch.no_grad():
            for t, v in zip(leaves, values(seed)):
                t.copy_(v)
        want = step()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_the_layer_in_a_captured_training_step(pkg):
    torch.manual_seed(0)
    layer = pkg.moe.FP4MoE(64, 96, 8, 2, device="cuda")
    x = rand((70, 64), BF, 1).requires_grad_()
    leaves = [x, layer.norm.weight, layer.norm.bias, layer.router.weight, layer.up.weight, layer.down.weight]

    def step():
        y = layer(x)
        return [y.detach(), *torch.autograd.grad(y.float().square().mean(), leaves)]
    g, out = captured_step(step)
    for seed in (2, 3):
        with torch.no_grad():
            x.copy_(rand((70, 64), BF, seed))
            layer.up.weight.mul_(1.25)
        want = step()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
    assert pkg.ops.device_status() == 0


def test_streams_and_threads(pkg):
    """Calls at once from threads with streams of their own equal the same calls alone."""
    sets = [inputs(m, n, s) for s, (m, n) in enumerate(((1000, 1032), (300, 520), (2500, 264), (40, 4096)))]
    want = [[t.clone() for t in calls(pkg, *s)] for s in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                got = calls(pkg, *sets[i])
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert pkg.ops.device_status() == 0


def test_calls_refuse_what_does_not_fit(pkg):
    ops = pkg.ops
    x, w = rand((4, 32), BF, 1), rand((32,), F, 2)
    _, stats = ops.layer_norm_saving(x, w)
    e = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    p = ops.expert_plan(e, 3)
    ys, g = rand((8, 32), BF, 3), rand((4, 2), F, 4)
    for call in (lambda: ops.layer_norm(x[0]), lambda: ops.layer_norm(x, w[:31]), lambda: ops.layer_norm(x, w.cpu()), lambda: ops.layer_norm(x, w, w.to(BF)),
                 lambda: ops.layer_norm(x, w.repeat(2)[::2]), lambda: ops.layer_norm(x, out=x.t()), lambda: ops.layer_norm(x, out=x[:1].expand(4, -1)),
                 lambda: ops.layer_norm(x, out=torch.empty_like(x, dtype=torch.int32)), lambda: ops.layer_norm(x, out=x, dtype=F),
                 lambda: ops.layer_norm_backward(x[:3], x, stats, w), lambda: ops.layer_norm_backward(x, x, stats[:, :3], w),
                 lambda: ops.layer_norm_backward(x, x, stats.t().contiguous().t(), w), lambda: ops.layer_norm_backward(x.cpu(), x, stats, w),
                 lambda: ops.route(x, 0), lambda: ops.route(x, 33), lambda: ops.route(x, 2, w[:31]), lambda: ops.route(x, 2, w.to(BF)),
                 lambda: ops.route(x, 2, groups=3), lambda: ops.route(x, 2, groups=4, kept=5), lambda: ops.route(x, 2, group_best=3),
                 lambda: ops.route_backward(g, x, e.long()), lambda: ops.route_backward(g[:, :1], x, e), lambda: ops.route_backward(g.to(BF), x, e),
                 lambda: ops.expert_plan(e.long(), 3), lambda: ops.expert_plan(e[0], 3), lambda: ops.expert_plan(e.t(), 3), lambda: ops.expert_plan(e, 0),
                 lambda: ops.expert_dispatch(x[:3], p), lambda: ops.expert_dispatch(x, (p.offsets, p.rows)), lambda: ops.expert_dispatch(x, p, out=x),
                 lambda: ops.expert_combine(ys[:7], p, g), lambda: ops.expert_combine(ys, p, g.t()), lambda: ops.expert_combine(ys, p, g[:3]),
                 lambda: ops.expert_combine(ys, p, g.to(BF)), lambda: ops.expert_combine(ys, p, g, x.float()), lambda: ops.expert_combine(ys, p, g, x[:3]),
                 lambda: ops.expert_combine_backward(x[:3], ys, p, g), lambda: ops.expert_combine_backward(x.float(), ys, p, g),
                 lambda: ops.expert_combine_backward(x, ys, p, None), lambda: ops.expert_dispatch(x, ops.ExpertPlan(p.offsets.cpu(), p.rows))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ops.layer_norm(x.to(torch.float16)), lambda: ops.route(x.to(torch.float16), 2), lambda: ops.expert_dispatch(x.double(), p)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: ops.route(rand((2, 600), F, 1), 2), lambda: ops.route(rand((2, 100), F, 1), 40), lambda: ops.expert_plan(e, 513)):
        with pytest.raises(ops.QLError) as error:
            call()
        assert error.value.status == 2
    with pytest.raises(ops.QLError):
        ops.layer_norm(x, eps=-1.0)
    assert ops.device_status() == 0


def test_a_given_out_counts_as_written(pkg):
    """Autograd sees that a tensor it saved has been written over; tensors without a version are taken as they are."""
    ops = pkg.ops
    p = ops.expert_plan(torch.zeros((4, 1), dtype=torch.int32, device="cuda"), 2)
    ys = rand((4, 32), F, 2)
    for write in (lambda t: ops.layer_norm(t, out=t), lambda t: ops.layer_norm_saving(t, out=t), lambda t: ops.expert_dispatch(ys, p, out=t),
                  lambda t: ops.expert_combine(ys, p, out=t), lambda t: ops.expert_combine(ys, p, None, t, out=t)):
        a = rand((4, 32), F, 1).requires_grad_() * 2
        y = a.square().sum()
        before = a._version
        write(a.detach())
        assert a._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    with torch.inference_mode():
        t = rand((4, 32), F, 1)
    want = ops.layer_norm(t)
    assert torch.equal(ops.layer_norm(t, out=t), want)


def test_autograd_keeps_the_plan(pkg):
    """A plan's tables are saved tensors: hooks see them, and tables written again are noticed."""
    m, k, n = 6, 2, 4
    e = torch.randint(-1, n, (m, k), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    x, ys, w = rand((m, 32), F, 1), rand((m * k, 32), F, 2), rand((m, k), F, 3)
    for call, leaf in ((lambda t, p: pkg.moe.dispatch(t, p), x), (lambda t, p: pkg.moe.combine(t, p, w), ys)):
        leaf = leaf.clone().requires_grad_()
        plan = pkg.ops.expert_plan(e, n)
        seen = []

        def pack(t):
            seen.append(t)
            return t.cpu()
        with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t.cuda()):
            y = call(leaf, plan)
        assert any(t is plan.rows or t.data_ptr() == plan.rows.data_ptr() for t in seen)
        v = rand(tuple(y.shape), F, 4)
        got, = torch.autograd.grad(y, leaf, v)
        want, = torch.autograd.grad(call(leaf, plan), leaf, v)
        assert torch.equal(got, want)
        y = call(leaf, plan)
        plan.rows.fill_(-1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
        with torch.inference_mode():
            frozen = pkg.ops.expert_plan(e, n)
        assert torch.equal(torch.autograd.grad(call(leaf, frozen), leaf, v)[0], want)


def test_sums_without_weights_have_gradients(pkg):
    m, k, n = 9, 3, 5
    e = torch.randint(-1, n, (m, k), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    plan = pkg.ops.expert_plan(e, n)
    ys, add = rand((m * k, 40), F, 2).requires_grad_(), rand((m, 40), F, 3).requires_grad_()
    v = rand((m, 40), F, 4)
    y = pkg.moe.combine(ys, plan, None, add)
    one = pkg.moe.combine(ys, plan, torch.ones((m, k), device="cuda"), add)
    assert torch.equal(y, one)
    for a, b in zip(torch.autograd.grad(y, (ys, add), v), torch.autograd.grad(one, (ys, add), v)):
        assert torch.equal(a, b)


def test_norm_of_no_columns(pkg):
    for shape in ((5, 0), (2, 3, 0), (0, 0), (0, 7), (2, 0, 7)):
        x = torch.empty(shape, device="cuda", requires_grad=True)
        w = torch.ones(shape[-1], device="cuda", requires_grad=True)
        y = pkg.norm.layer_norm(x, w)
        assert y.shape == shape
        y.sum().backward()
        assert x.grad.shape == shape and not w.grad.any()
        with torch.no_grad():
            assert pkg.norm.LayerNorm(shape[-1], device="cuda")(x).shape == shape


def test_outs_over_inputs_are_refused(pkg):
    """Rows that others are still read from are not written: but a norm's may be x's own, sums' add's."""
    ops = pkg.ops
    room = rand((12, 64), F, 1)
    p = ops.expert_plan(torch.zeros((4, 1), dtype=torch.int32, device="cuda"), 2)
    x, ys = room[:4], room[4:8]
    half, tall = room.view(24, 32)[:4], room.to(BF)
    for call in (lambda: ops.expert_dispatch(x, p, out=x), lambda: ops.expert_dispatch(x, p, out=room[1:5]), lambda: ops.expert_combine(ys, p, out=ys),
                 lambda: ops.expert_combine(ys, p, out=room[6:10]), lambda: ops.expert_combine(ys, p, None, x, out=room[1:5]),
                 lambda: ops.layer_norm(x, out=room[2:6]), lambda: ops.layer_norm(room[:, :32][:4], out=room[:, 16:48][:4]),
                 lambda: ops.layer_norm(room[:, :32][:4], out=half), lambda: ops.layer_norm(room[:1], out=room[:1].view(BF)[:, :64]),
                 lambda: ops.layer_norm_saving(tall[:4].view(F), out=tall[:4, :32])):
        with pytest.raises(ValueError):
            call()
    # side by side and row by row in one buffer
    want = ops.layer_norm(room[:, :32].contiguous())
    keep = room.clone()
    assert torch.equal(ops.layer_norm(room[:, :32], out=room[:, 32:]), want) and torch.equal(room[:, :32], keep[:, :32])
    room.copy_(keep)
    want = ops.expert_dispatch(room[0:8:2].contiguous(), p)
    assert torch.equal(ops.expert_dispatch(room[0:8:2], p, out=room[1:8:2]), want) and torch.equal(room[0:8:2], keep[0:8:2])
    room.copy_(keep)
    assert torch.equal(ops.expert_combine(x[:, ::2], p, out=room[:4, :32]), ops.expert_combine(keep[:4, ::2], p))      # of a copy
