"""Cases of the operators around the experts' products: layer norm and its
training step, routing with its gradient, and the exchange of rows with the
experts (sorted by expert and back as weighted sums) with its gradients.

  layer norm  y = (x - mean) / sqrt(var + eps) * w + b over each row
  routing     scores s = softmax(logits) or sigmoid(logits), choice c = s + bias; of
              `groups` equal groups of experts the `kept` best stay (a group's score: the sum of
              its `group_best` largest c), of their experts the k best, ties to the lowest index;
              weights s, renormalised over the chosen or not, times `scale`. An expert with
              logit -inf is out of reach; a token that reaches none has experts -1, weights 0.
  exchange    slots (token, j) sorted by expert, stable; offsets of the experts' rows; rows
              xs = x of each slot's token, zeros past the last expert's; y = sum_j w_j ys(slot j)
"""
import math

import torch

own = False

EPS = 1e-5


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a single token's activations before a projection
        {"name": "norm_1x7168", "op": "norm", "m": 1, "n": 7168, "dtype": "bf16", "out": "bf16", "affine": True},
        # a long prompt's
        {"name": "norm_16384x7168", "op": "norm", "m": 16384, "n": 7168, "dtype": "bf16", "out": "bf16", "affine": True},
        # an fp32 stream of odd sizes, normalised into bf16 without weights
        {"name": "norm_2051x1003_f32_bf16", "op": "norm", "m": 2051, "n": 1003, "dtype": "f32", "out": "bf16",
         "affine": False},
        # a training step of the norm before a layer
        {"name": "norm_train_4096x7168", "op": "norm_train", "m": 4096, "n": 7168, "dtype": "bf16", "out": "bf16",
         "affine": True},
        # the same in fp32 at odd sizes
        {"name": "norm_train_1003x4099_f32", "op": "norm_train", "m": 1003, "n": 4099, "dtype": "f32", "out": "f32",
         "affine": True},
        # decoding one token over many experts: bias for balance, groups
        {"name": "route_1_8of256_groups", "op": "route", "m": 1, "experts": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "kept": 4, "group_best": 2, "renormalise": True, "scale": 2.5, "dtype": "f32", "padded": 0.0},
        # a long prompt through the same router
        {"name": "route_16384_8of256_groups", "op": "route", "m": 16384, "experts": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "kept": 4, "group_best": 2, "renormalise": True, "scale": 2.5, "dtype": "f32",
         "padded": 0.0},
        # a training step of a small softmax router, bf16 logits, some of the batch padding
        {"name": "route_train_4096_2of8", "op": "route_train", "m": 4096, "experts": 8, "k": 2, "score": "softmax",
         "bias": False, "groups": 1, "kept": 1, "group_best": 1, "renormalise": True, "scale": 1.0, "dtype": "bf16",
         "padded": 0.1},
        # odd numbers of tokens and experts, weights not renormalised: a dense gradient
        {"name": "route_train_5003_6of162", "op": "route_train", "m": 5003, "experts": 162, "k": 6, "score": "softmax",
         "bias": False, "groups": 9, "kept": 3, "group_best": 1, "renormalise": False, "scale": 16.0, "dtype": "f32",
         "padded": 0.0},
        # a decode batch to the experts and back
        {"name": "exchange_16x8of256x7168", "op": "exchange", "m": 16, "n": 7168, "experts": 256, "k": 8, "dtype": "bf16",
         "skew": 0.5, "padded": 0.0},
        # a prompt
        {"name": "exchange_4096x8of256x7168", "op": "exchange", "m": 4096, "n": 7168, "experts": 256, "k": 8,
         "dtype": "bf16", "skew": 0.5, "padded": 0.0},
        # a training step: both directions, part of the batch padding
        {"name": "exchange_train_4096x2of8x4096", "op": "exchange_train", "m": 4096, "n": 4096, "experts": 8, "k": 2,
         "dtype": "bf16", "skew": 0.5, "padded": 0.05},
    ]


def _log(rng, lo, hi, odd=0.5):
    """A size between lo and hi, spread over its logarithm; often one that is no multiple of anything."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() >= odd and v >= 64:
        v = v // 32 * 32
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "route", "route_train", "exchange", "exchange_train"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op.startswith("norm"):
        c["n"] = _log(rng, 33, 16384)
        c["m"] = _log(rng, 1, min(16384, (1 << 25) // c["n"]))
        c |= {"out": rng.choice([c["dtype"], c["dtype"], "bf16"]), "affine": rng.random() < 0.75}
    elif op.startswith("route"):
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _log(rng, max(2, 8 // groups), 512 // groups, odd=1.0)
        kept = rng.randint(1, groups)
        c |= {"m": _log(rng, 1, 16384), "experts": groups * size, "groups": groups, "kept": kept,
              "k": rng.randint(1, min(8, kept * size)), "group_best": rng.choice([1, 2]),
              "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "renormalise": rng.random() < 0.6,
              "scale": rng.choice([1.0, 1.0, 2.5]), "padded": rng.choice([0.0, 0.0, 0.1])}
        if op == "route_train" and c["k"] == 1:
            c["renormalise"] = False                   # one weight renormalised is constant: no gradient
    else:
        c |= {"n": _log(rng, 33, 7168), "experts": _log(rng, 2, 512, odd=1.0), "k": rng.randint(1, 8)}
        token = c["n"] * (2 * c["k"] + 2) * _size(c["dtype"]) * (2 if op == "exchange_train" else 1)
        c["m"] = _log(rng, 1, min(16384, 1_000_000_000 // token))
        c |= {"skew": round(rng.uniform(0.0, 1.5), 2), "padded": rng.choice([0.0, 0.0, 0.1])}
    return c


def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    op, m, es = case["op"], case["m"], _size(case["dtype"])
    if op.startswith("norm"):
        n, eo = case["n"], _size(case["out"])
        w = 2 * n * 4 if case["affine"] else 0
        if op == "norm":
            return {"bytes": m * n * (es + eo) + w, "flops": 8 * m * n}
        return {"bytes": m * n * (2 * es + 2 * eo) + 2 * w, "flops": 24 * m * n}      # x, dy read, y, dx written
    k, g = case["k"], case["experts"]
    if op.startswith("route"):
        fwd = m * g * es + m * k * 8 + (g * 4 if case["bias"] else 0)
        if op == "route":
            return {"bytes": fwd, "flops": 8 * m * g}
        return {"bytes": fwd + m * k * 4 + m * g * es, "flops": 16 * m * g}             # dw read, dlogits written
    n = case["n"]
    one = m * n * es
    fwd = one + k * one + k * one + one + m * k * 8 + g * 4
    if op == "exchange":
        return {"bytes": fwd, "flops": 2 * m * k * n}
    return {"bytes": fwd + one + k * one + k * one + one + m * k * 4, "flops": 7 * m * k * n}


# ---------------------------------------------------------------- inputs
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _acts(shape, gen, dtype):
    """Activations: rows of different loudness and offset, and a few loud channels."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= 1 + 15 * (torch.rand((1, shape[1]), generator=gen, device="cuda") < 0.01)
    x += 0.5 * torch.randn((shape[0], 1), generator=gen, device="cuda")
    x *= torch.exp2(torch.randint(-2, 3, (shape[0], 1), generator=gen, device="cuda").float())
    return x.to(dtype)


def _padding(case, gen):
    """Tokens that stand for nothing: the last ones of a batch of fixed size."""
    m = case["m"]
    return torch.arange(m, device="cuda") >= m - int(m * case["padded"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, m, dt = case["op"], case["m"], _dtype(case["dtype"])
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    s = {"case": case}
    if op.startswith("norm"):
        n = case["n"]
        s["x"] = _acts((m, n), gen, dt)
        s["w"] = 1 + 0.2 * rand(n) if case["affine"] else None
        s["b"] = 0.1 * rand(n) if case["affine"] else None
        if op == "norm_train":
            s["dy"] = (1e-3 * rand(m, n)).to(_dtype(case["out"]))
        return s
    g, k = case["experts"], case["k"]
    if op.startswith("route"):
        favour = 0.7 * rand(1, g)                      # some experts are liked more than others
        s["logits"] = (1.3 * rand(m, g) + favour).masked_fill_(_padding(case, gen)[:, None], -math.inf).to(dt)
        s["bias"] = None
        if case["bias"]:                               # it goes against the favour
            s["bias"] = (-0.1 if case["score"] == "sigmoid" else -0.5 / g) * favour[0] + 1e-3 / g * rand(g)
        if op == "route_train":
            s["dw"] = rand(m, k)
        return s
    n = case["n"]
    likes = -case["skew"] * torch.log1p(torch.randperm(g, generator=gen, device="cuda").float())
    noise = -torch.log(-torch.log(torch.rand((m, g), generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))
    best = torch.argsort(likes + noise, dim=1, descending=True)[:, :k]
    if g < k:                                          # more slots than experts: the rest goes nowhere
        best = torch.nn.functional.pad(best, (0, k - g), value=-1)
    s["experts"] = best.masked_fill(_padding(case, gen)[:, None], -1).to(torch.int32)
    s["w"] = torch.softmax(rand(m, k), dim=1)
    s["x"] = _acts((m, n), gen, dt)
    s["ys"] = rand(m * k, n).to(dt)                    # what the experts make of the sorted rows
    if op == "exchange_train":
        s["dy"] = (1e-3 * rand(m, n)).to(dt)
        s["dxs"] = (1e-3 * rand(m * k, n)).to(dt)      # and what comes back for them
    return s


# ---------------------------------------------------------------- plain form
def _norm(s):
    case, x, w = s["case"], s["x"].float(), s["w"]
    d = x - x.mean(1, keepdim=True)
    r = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    h = d * r
    y = (h if w is None else h * w + s["b"]).to(_dtype(case["out"]))
    if case["op"] == "norm":
        return y
    dy = s["dy"].float()
    g = dy if w is None else dy * w
    dx = r * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    out = {"y": y, "dx": dx.to(s["x"].dtype)}
    if w is not None:
        out |= {"dw": (dy * h).sum(0), "db": dy.sum(0)}
    return out


def _scores(case, logits):
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True).clamp(min=-1e30))
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _route(s):
    case, logits = s["case"], s["logits"]
    m, g, groups, k = case["m"], case["experts"], case["groups"], case["k"]
    wide = logits.double()                             # choices next to a border
    reach = wide > -math.inf
    c = _scores(case, wide)
    if s["bias"] is not None:
        c = c + s["bias"].double()
    c = c.masked_fill(~reach, -math.inf)
    if groups > 1:
        best = torch.sort(c.view(m, groups, -1), dim=2, descending=True)[0][:, :, :case["group_best"]].sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True)[1]
        place = torch.empty_like(order)
        place.scatter_(1, order, torch.arange(groups, device=c.device).expand(m, groups))
        c = c.masked_fill((place >= case["kept"]).repeat_interleave(g // groups, 1), -math.inf)
    top, experts = torch.sort(c, dim=1, descending=True, stable=True)
    top, experts = top[:, :k], experts[:, :k]
    there = top > -math.inf
    p = _scores(case, logits.float())
    q = torch.where(there, torch.gather(p, 1, experts), 0)
    total = q.sum(1, keepdim=True).clamp(min=1e-30)
    weights = case["scale"] * (q / total if case["renormalise"] else q)
    out = {"weights": weights, "experts": torch.where(there, experts, -1).to(torch.int32)}
    if case["op"] == "route":
        return out
    dq = case["scale"] * s["dw"] * there
    if case["renormalise"]:
        dq = (dq - (dq * q).sum(1, keepdim=True) / total) / total * there
    dp = torch.zeros_like(p).scatter_add_(1, experts, dq)
    dl = dp * p * (1 - p) if case["score"] == "sigmoid" else p * (dp - (dp * p).sum(1, keepdim=True))
    return out | {"dlogits": dl.to(logits.dtype)}


def _exchange(s):
    case, x, ys, w = s["case"], s["x"], s["ys"], s["w"]
    m, n, k, g = case["m"], case["n"], case["k"], case["experts"]
    key = torch.where(s["experts"] < 0, g, s["experts"]).flatten().long()
    order = torch.sort(key, stable=True)[1]
    counts = torch.zeros(g + 1, dtype=torch.int64, device=x.device).index_add_(0, key, torch.ones_like(key))
    ends = counts[:g].cumsum(0)
    offsets = torch.nn.functional.pad(ends, (1, 0)).to(torch.int32)
    used = (torch.arange(m * k, device=x.device) < ends[-1])[:, None]
    there = (key < g).view(m, k, 1)
    rows = torch.empty_like(order)
    rows[order] = torch.arange(m * k, device=x.device)
    token = order // k
    xs = torch.where(used, x[token], 0)
    mine = torch.where(there, ys[rows].view(m, k, n), 0).float()
    y = (mine * w[:, :, None]).sum(1).to(x.dtype)
    out = {"offsets": offsets, "xs": xs, "y": y}
    if case["op"] == "exchange":
        return out
    dy = s["dy"].float()
    dys = torch.where(used, dy[token] * w.flatten()[order][:, None], 0).to(ys.dtype)
    dw = (mine * dy[:, None]).sum(2)
    dx = torch.where(there, s["dxs"][rows].view(m, k, n), 0).float().sum(1).to(x.dtype)
    return out | {"dys": dys, "dw": dw, "dx": dx}


# ---------------------------------------------------------------- a user's calls
def _calls(s):
    from quantised_linear_layers_gb300 import ops
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return ops.layer_norm(s["x"], s["w"], s["b"], EPS, dtype=_dtype(case["out"]))
    if op == "norm_train":
        y, stats = ops.layer_norm_saving(s["x"], s["w"], s["b"], EPS, dtype=_dtype(case["out"]))
        dx, dw, db = ops.layer_norm_backward(s["dy"], s["x"], stats, s["w"])
        return {"y": y, "dx": dx, "dw": dw, "db": db} if case["affine"] else {"y": y, "dx": dx}
    if op.startswith("route"):
        how = {"score": case["score"], "renormalise": case["renormalise"], "scale": case["scale"]}
        weights, experts = ops.route(s["logits"], case["k"], s["bias"], groups=case["groups"], kept=case["kept"],
                                     group_best=case["group_best"], **how)
        out = {"weights": weights, "experts": experts}
        if op == "route_train":
            out["dlogits"] = ops.route_backward(s["dw"], s["logits"], experts, **how)
        return out
    plan = ops.expert_plan(s["experts"], case["experts"])
    xs = ops.expert_dispatch(s["x"], plan)
    y = ops.expert_combine(s["ys"], plan, s["w"])
    out = {"offsets": plan.offsets, "xs": xs, "y": y}
    if op == "exchange_train":
        out["dys"], out["dw"] = ops.expert_combine_backward(s["dy"], s["ys"], plan, s["w"])
        out["dx"] = ops.expert_combine(s["dxs"], plan)
    return out


def run(state):
    if own:
        return _calls(state)
    op = state["case"]["op"]
    return _norm(state) if op.startswith("norm") else _route(state) if op.startswith("route") else _exchange(state)


# ---------------------------------------------------------------- 64 bits
def _exact_norm(case, s):
    x = s["x"].double()
    n = case["n"]
    mean = x.sum(1, keepdim=True) / n
    h = (x - mean) / torch.sqrt(((x - mean) ** 2).sum(1, keepdim=True) / n + EPS)
    r = h.new_ones(1) / torch.sqrt(((x - mean) ** 2).sum(1, keepdim=True) / n + EPS)
    one, zero = x.new_ones(n), x.new_zeros(n)
    w = one if s["w"] is None else s["w"].double()
    y = h * w + (zero if s["b"] is None else s["b"].double())
    if case["op"] == "norm":
        return y
    dy = s["dy"].double()
    g = dy * w
    # dx_i = r (g_i - <g, 1> / n - h_i <g, h> / n)
    dx = r * (g - (g @ one)[:, None] / n - h * torch.einsum("ij,ij->i", g, h)[:, None] / n)
    out = {"y": y, "dx": dx}
    if s["w"] is not None:
        out |= {"dw": torch.einsum("ij,ij->j", dy, h), "db": dy.t() @ dy.new_ones(case["m"])}
    return out


def _exact_route(case, s):
    l, k, m, g = s["logits"].double(), case["k"], case["m"], case["experts"]
    sigmoid = case["score"] == "sigmoid"
    dead = torch.isneginf(l).all(1)
    l = torch.where(dead[:, None], torch.zeros_like(l), l)
    p = torch.sigmoid(l) if sigmoid else torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    c = p if s["bias"] is None else p + s["bias"].double()
    size = g // case["groups"]
    parts = c.reshape(m, case["groups"], size)
    left = parts.clone()
    score = torch.zeros(m, case["groups"], dtype=torch.float64, device=l.device)
    for _ in range(min(case["group_best"], size)):
        v, i = left.max(2)
        score += v
        left.scatter_(2, i[:, :, None], -math.inf)
    alive = torch.zeros_like(score, dtype=torch.bool)
    for _ in range(case["kept"]):
        best = score.max(1, keepdim=True).values
        first = (score == best).to(torch.int8).argmax(1, keepdim=True)
        alive.scatter_(1, first, True)
        score = score.scatter(1, first, -math.inf)
    c = torch.where(alive[:, :, None], parts, -math.inf).reshape(m, g).clone()
    chosen = []
    for _ in range(k):
        best = c.max(1, keepdim=True).values
        first = (c == best).to(torch.int8).argmax(1, keepdim=True)
        chosen.append(first)
        c = c.scatter(1, first, -math.inf)
    e = torch.cat(chosen, 1)
    on = (~dead)[:, None].double()
    lg, q = torch.gather(l, 1, e), torch.gather(p, 1, e)
    part = q / q.sum(1, keepdim=True)
    weights = case["scale"] * (part if case["renormalise"] else q) * on
    experts = torch.where(dead[:, None], -1, e).to(torch.int32)
    out = {"weights": weights, "experts": experts}
    if case["op"] == "route":
        return out
    dw = case["scale"] * s["dw"].double() * on
    if case["renormalise"]:
        slope = torch.sigmoid(-lg) if sigmoid else torch.ones_like(lg)
        d = torch.zeros_like(l).scatter_add_(1, e, part * slope * (dw - (part * dw).sum(1, keepdim=True)))
    elif sigmoid:
        d = torch.zeros_like(l).scatter_add_(1, e, dw * q * torch.sigmoid(-lg))
    else:
        d = torch.zeros_like(l).scatter_add_(1, e, dw * q) - p * (dw * q).sum(1, keepdim=True)
    return out | {"dlogits": d}


def _exact_exchange(case, s):
    m, n, k, g = case["m"], case["n"], case["k"], case["experts"]
    e, train = s["experts"].cpu().tolist(), case["op"] == "exchange_train"
    of = [[] for _ in range(g)]
    for t in range(m):
        for j in range(k):
            if e[t][j] >= 0:
                of[e[t][j]].append(t * k + j)
    ends = [0]
    for mine in of:
        ends.append(ends[-1] + len(mine))
    slots = torch.tensor([v for mine in of for v in mine], dtype=torch.int64, device="cuda")
    used = ends[-1]
    token, weight = slots // k, s["w"].double().flatten()[slots][:, None]
    xs = torch.zeros((m * k, n), dtype=torch.float64, device="cuda")
    xs[:used] = s["x"][token].double()
    y = torch.zeros((m, n), dtype=torch.float64, device="cuda")
    y.index_add_(0, token, s["ys"][:used].double() * weight)
    out = {"offsets": torch.tensor(ends, dtype=torch.int32, device="cuda"), "xs": xs, "y": y}
    if train:
        dy = s["dy"].double()[token]
        out["dys"] = torch.zeros_like(xs)
        out["dys"][:used] = dy * weight
        out["dw"] = torch.zeros(m * k, dtype=torch.float64, device="cuda")
        out["dw"][slots] = torch.einsum("ij,ij->i", dy, s["ys"][:used].double())
        out["dw"] = out["dw"].view(m, k)
        out["dx"] = torch.zeros_like(y).index_add_(0, token, s["dxs"][:used].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return (_exact_norm if op.startswith("norm") else _exact_route if op.startswith("route") else _exact_exchange)(case, s)
