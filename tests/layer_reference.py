"""Layer norm, routing and the exchange with the experts in 64 bits, from their
definitions, with the errors that fp32 arithmetic may have beside them.

U is half a step of fp32 (2^-24 of a value). A sum in which every term passes at most
c additions is within c U of the sum of its terms' magnitudes."""
import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def adds(n):
    """Additions that a term passes in a row's sum: a thread's run, then two trees of 32."""
    return max(64, -(-n // 256)) + 16


def close(got, want, tol, what=""):
    """got within tol of want everywhere, NaN where it is NaN, infinities equal."""
    got, want, tol = got.detach().cpu().double(), want.cpu(), tol.cpu()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, not {tuple(want.shape)}"
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    fine = ~(nan | inf)
    off = (got - want).abs()[fine]
    bad = ~(off <= tol.expand_as(want)[fine])
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, by {float(off[bad].max()):.3e} at most"


def norm(x, w, b, eps, out_dtype, c=None):
    """(y, its tolerance, h, mean, rstd, h's tolerance); c: additions that a term passes."""
    x = x.detach().cpu().double()
    n = x.shape[1]
    w = torch.ones(n, dtype=torch.float64) if w is None else w.detach().cpu().double()
    b = torch.zeros(n, dtype=torch.float64) if b is None else b.detach().cpu().double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    h = (x - mean) * rstd
    y = h * w + b
    c = adds(n) if c is None else c
    # the mean within c U of the mean |x - mean| (one standard deviation at most), the
    # variance within 2 c U, six roundings on the way
    dh = U * (c + (c + 6) * h.abs())
    tol = w.abs() * dh + 2 * U * ((h * w).abs() + y.abs()) + HALF[out_dtype] * y.abs() * (out_dtype != torch.float32)
    return y, tol * (1 + 2 ** -7), h, mean, rstd, dh


def norm_backward(dy, x, w, eps, dx_dtype, c=None):
    """{name: (value, tolerance)} of dx, dw, db."""
    _, _, h, mean, rstd, dh = norm(x, None, None, eps, torch.float32, c)
    dy = dy.detach().cpu().double()
    n = h.shape[1]
    g = dy if w is None else dy * w.detach().cpu().double()
    c1, c2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = rstd * (g - c1 - h * c2)
    c = adds(n) if c is None else c
    # h from the kept mean, which is rounded once more
    dh = dh + 2 * U * mean.abs() * rstd
    ga, gh = g.abs().mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
    e1 = (c + 4) * U * ga
    e2 = (c + 4) * U * gh + (g.abs() * dh).mean(1, keepdim=True)
    tol = rstd * (e1 + h.abs() * e2 + dh * c2.abs() + (c + 8) * U * (g.abs() + c1.abs() + (h * c2).abs()))
    tol = tol + HALF[dx_dtype] * dx.abs() * (dx_dtype != torch.float32)
    m = dy.shape[0]
    run = m + 16
    dw = (dy * h).sum(0)
    tw = run * U * (dy * h).abs().sum(0) + (dy.abs() * dh).sum(0)
    return {"dx": (dx, tol * (1 + 2 ** -7)), "dw": (dw, tw), "db": (dy.sum(0), run * U * dy.abs().sum(0))}


def scores(logits, score):
    l = logits.detach().cpu().double()
    if score == "sigmoid":
        return torch.sigmoid(l)
    top = l.amax(1, keepdim=True)
    top = torch.where(torch.isinf(top) & (top < 0), torch.zeros_like(top), top)
    e = torch.exp(l - top)
    total = e.sum(1, keepdim=True)
    return torch.where(total == 0, torch.zeros_like(e), e / total)


def choose(logits, k, bias=None, score="softmax", groups=1, kept=1, group_best=1):
    """The chosen experts [tokens, k], one token and one choice after the other."""
    l = logits.detach().cpu().double()
    s = scores(logits, score)
    m, n = l.shape
    b = torch.zeros(n, dtype=torch.float64) if bias is None else bias.detach().cpu().double()
    size = n // groups
    out = torch.full((m, k), -1, dtype=torch.int32)
    for t in range(m):
        reach = [not (math.isinf(l[t, e]) and l[t, e] < 0) and not (math.isinf(b[e]) and b[e] < 0) for e in range(n)]
        lowest = -1e300

        def value(e, of):
            return lowest if math.isnan(of) else of
        c = [value(e, float(s[t, e] + b[e])) if reach[e] else -math.inf for e in range(n)]
        allowed = set(range(n))
        if kept < groups:
            by = []
            for g in range(groups):
                best = sorted((c[e] for e in range(g * size, (g + 1) * size) if reach[e]), reverse=True)[:group_best]
                by.append(sum(best) if best else -math.inf)
            order = sorted(range(groups), key=lambda g: (-by[g], g))[:kept]
            allowed = {e for g in order if by[g] > -math.inf for e in range(g * size, (g + 1) * size)}
        order = c if bias is not None else [value(e, float(l[t, e])) if reach[e] else -math.inf for e in range(n)]
        best = sorted((e for e in allowed if reach[e]), key=lambda e: (-order[e], e))[:k]
        out[t, :len(best)] = torch.tensor(best, dtype=torch.int32)
    return out


def route_weights(logits, experts, score, renormalise, scale):
    """(weights, tolerance) of the chosen."""
    l = logits.detach().cpu().double()
    on = experts >= 0
    at = experts.clamp(min=0).long()
    lg = torch.where(on, torch.gather(l, 1, at), torch.full((), -math.inf, dtype=torch.float64))
    if renormalise:
        # log s relative to the largest, so that nothing underflows
        ls = torch.nn.functional.logsigmoid(lg) if score == "sigmoid" else lg
        ls = torch.where(on, ls, torch.full_like(ls, -math.inf))
        w = scale * torch.softmax(ls, 1)
        w = torch.where(on, w, torch.zeros_like(w))
        far = (lg - lg.amax(1, keepdim=True)).abs()
    else:
        w = torch.where(on, scale * torch.gather(scores(logits, score), 1, at), torch.zeros((), dtype=torch.float64))
        far = lg.abs() if score == "sigmoid" else (lg - l.amax(1, keepdim=True)).abs()
    # exp within 2^-22 and the rounding of its argument, up to 21 additions, divisions and
    # products; and what fp32 cannot hold
    tol = w.abs() * (2.0 ** -18 + torch.nan_to_num(far, 0, 0, 0) * 2 * U) + 1e-37
    return w, tol


def route_backward(dw, logits, experts, score, renormalise, scale, dtype):
    """(dlogits, tolerance): slot by slot."""
    l = logits.detach().cpu().double()
    m, n = l.shape
    s = scores(logits, score)
    d = torch.zeros_like(l)
    size = torch.zeros_like(l)                  # sums of the magnitudes that cancel
    dw = dw.detach().cpu().double() * scale
    for t in range(m):
        slots = [(j, int(e)) for j, e in enumerate(experts[t]) if 0 <= e < n]
        if not slots:
            continue
        if renormalise:
            lg = torch.stack([l[t, e] for _, e in slots])
            ls = torch.nn.functional.logsigmoid(lg) if score == "sigmoid" else lg
            q = torch.softmax(ls, 0)
            rest = torch.sigmoid(-lg) if score == "sigmoid" else torch.ones_like(lg)
            g = torch.stack([dw[t, j] for j, _ in slots])
            mean, mag = (q * g).sum(), (q * g).abs().sum()
            for i, (j, e) in enumerate(slots):
                d[t, e] += q[i] * rest[i] * (g[i] - mean)
                size[t, e] += q[i] * rest[i] * (g[i].abs() + mag)
        elif score == "sigmoid":
            for j, e in slots:
                v = dw[t, j] * s[t, e] * torch.sigmoid(-l[t, e])
                d[t, e] += v
                size[t, e] += v.abs()
        else:
            dp = torch.zeros(n, dtype=torch.float64)
            ap = torch.zeros(n, dtype=torch.float64)
            for j, e in slots:
                dp[e] += dw[t, j]
                ap[e] += dw[t, j].abs()
            d[t] = s[t] * (dp - (dp * s[t]).sum())
            size[t] = s[t] * (ap + (ap * s[t]).sum())
    finite = torch.where(torch.isinf(l), torch.zeros_like(l), l)
    far = finite.abs().amax(1, keepdim=True) * 4
    return d, size * (2.0 ** -17 + far * 2 * U) + HALF[dtype] * d.abs() + 1e-37


def plan(experts, num_experts):
    """(offsets, rows) as lists: the slots of expert 0, of expert 1, and so on."""
    flat = experts.cpu().flatten().tolist()
    rows, at, offsets = [-1] * len(flat), 0, [0]
    for e in range(num_experts):
        for i, f in enumerate(flat):
            if f == e:
                rows[i] = at
                at += 1
        offsets.append(at)
    return offsets, rows
