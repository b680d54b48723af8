"""Cases of the microscaled 4-bit (E2M1) operators: the cast and its inverse,
the linear layer's product, its training step, and the products of ragged
experts.

Formats. "nv": groups of 16 along the reduction axis, each with an E4M3 scale,
under one power of two t per tensor; "mx": groups of 32 with a power of two.

  nv  s = E4M3(amax / (6 t)) in [2^-9, 448], value = E2M1(x / (s t)) s t
  mx  s = 2^ceil(log2(amax / 6)),            value = E2M1(x / s) s

amax is the group's largest magnitude; E2M1 and E4M3 round to nearest, ties to
even. t is 1 for the activations of a forward-only call and elsewhere the least
power of two with max|x| <= 2688 t (2688 = 6 * 448), at least 2^-80.
"""
import math

import torch

own = False

GROUP = {"nv": 16, "mx": 32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a single token's activations quantised before a product, and read back
        {"name": "cast_1x7168_nv", "op": "cast", "m": 1, "k": 7168, "fmt": "nv", "dtype": "bf16", "dynamic": False},
        # a prompt's activations kept in 4 bits
        {"name": "cast_16384x7168_mx", "op": "cast", "m": 16384, "k": 7168, "fmt": "mx", "dtype": "bf16",
         "dynamic": False},
        # an fp32 tensor of odd sizes with its own tensor scale (a gradient, a weight)
        {"name": "cast_1003x4099_f32_nv", "op": "cast", "m": 1003, "k": 4099, "fmt": "nv", "dtype": "f32",
         "dynamic": True},
        # decoding one sequence: one row against a whole weight
        {"name": "linear_1x4096x7168_nv", "op": "linear", "m": 1, "n": 4096, "k": 7168, "fmt": "nv", "dtype": "bf16"},
        # a decode batch
        {"name": "linear_64x4096x7168_mx", "op": "linear", "m": 64, "n": 4096, "k": 7168, "fmt": "mx",
         "dtype": "bf16"},
        # odd sizes in every direction, fp32 activations
        {"name": "linear_333x1001x2051_f32_mx", "op": "linear", "m": 333, "n": 1001, "k": 2051, "fmt": "mx",
         "dtype": "f32"},
        # a long prompt through the widest projection
        {"name": "linear_16384x18432x7168_nv", "op": "linear", "m": 16384, "n": 18432, "k": 7168, "fmt": "nv",
         "dtype": "bf16"},
        # a training step of the layer (weight cast, forward, both gradients)
        {"name": "train_4096x4096x7168_nv", "op": "train", "m": 4096, "n": 4096, "k": 7168, "fmt": "nv",
         "dtype": "bf16"},
        # the same at odd sizes, fp32 activations
        {"name": "train_509x776x1033_f32_mx", "op": "train", "m": 509, "n": 776, "k": 1033, "fmt": "mx",
         "dtype": "f32"},
        # decoding through experts: a few rows, some experts idle
        {"name": "experts_16_of_8x4096x7168_nv", "op": "experts", "m": 16, "experts": 8, "n": 4096, "k": 7168,
         "fmt": "nv", "dtype": "bf16", "skew": 1.0},
        # a prompt through experts of uneven load
        {"name": "experts_16384_of_8x4096x7168_nv", "op": "experts", "m": 16384, "experts": 8, "n": 4096, "k": 7168,
         "fmt": "nv", "dtype": "bf16", "skew": 0.5},
        # a training step of the experts
        {"name": "experts_train_4096_of_8x4096x4096_mx", "op": "experts_train", "m": 4096, "experts": 8, "n": 4096,
         "k": 4096, "fmt": "mx", "dtype": "bf16", "skew": 0.7},
    ]


def _log(rng, lo, hi, odd=0.5):
    """A size between lo and hi, spread over its logarithm; often one that is no multiple of anything."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() >= odd and v >= 64:
        v = v // 32 * 32
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["cast", "linear", "linear", "train", "experts", "experts_train"])
    c = {"op": op, "fmt": rng.choice(["nv", "mx"]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "cast":
        c |= {"m": _log(rng, 1, 16384), "k": _log(rng, 33, 7168), "dynamic": rng.random() < 0.5}
    elif op == "linear":
        c |= {"m": _log(rng, 1, 16384), "n": _log(rng, 64, 18432), "k": _log(rng, 64, 7168)}
    elif op == "train":
        c |= {"m": _log(rng, 1, 8192), "n": _log(rng, 64, 7168), "k": _log(rng, 64, 7168)}
    else:
        c |= {"m": _log(rng, 1, 8192), "experts": _log(rng, 1, 32, odd=1.0), "n": _log(rng, 64, 4096),
              "k": _log(rng, 64, 4096), "skew": round(rng.uniform(0.0, 1.5), 2)}
    return c


def work(case):
    m, k = case["m"], case["k"]
    es = 2 if case["dtype"] == "bf16" else 4
    q = 0.5 + 1.0 / GROUP[case["fmt"]]
    if case["op"] == "cast":
        return {"bytes": m * k * (es + q + 2), "flops": 4 * m * k}
    n = case["n"]
    if case["op"] == "linear":
        return {"bytes": m * k * es + n * k * q + m * n * 2, "flops": 2 * m * n * k}
    if case["op"] == "experts":
        used = sum(1 for s in _sizes(case) if s)
        return {"bytes": m * k * es + used * n * k * q + m * n * 2, "flops": 2 * m * n * k}
    g = case.get("experts", 1)       # a training step: x, w, dy read, y, dx, dw written
    return {"bytes": m * k * es + g * n * k * 2 + m * n * 2 + m * n * 2 + m * k * 2 + g * n * k * 4,
            "flops": 6 * m * n * k}


# ---------------------------------------------------------------- inputs
def _sizes(case):
    """Rows of each expert: a load that falls off over the experts, in an order of its own."""
    g, m = case["experts"], case["m"]
    share = [(1.0 + (i * 7919) % g) ** -case["skew"] for i in range(g)]
    total, sizes, given, acc = sum(share), [], 0, 0.0
    for s in share:
        acc += s
        upto = int(m * acc / total + 1e-9)
        sizes.append(upto - given)
        given = upto
    sizes[-1] += m - given
    return sizes


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _acts(shape, gen, dtype):
    """Activations: rows of different loudness and a few loud channels."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.exp2(torch.randint(-2, 3, (shape[0], 1), generator=gen, device="cuda").float())
    x *= 1 + 15 * (torch.rand((1, shape[1]), generator=gen, device="cuda") < 0.01)
    return x.to(dtype)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    m, k = case["m"], case["k"]
    s = {"x": _acts((m, k), gen, _dtype(case))}
    if case["op"] == "cast":
        return s
    n, g = case["n"], case.get("experts")
    w = torch.randn((n, k) if g is None else (g, n, k), generator=gen, device="cuda")
    s["w"] = (w.mul_(0.02)).bfloat16()
    if "train" in case["op"]:
        s["dy"] = (torch.randn((m, n), generator=gen, device="cuda") * 1e-3).bfloat16()
    if g is not None:
        sizes = _sizes(case)
        ends = torch.tensor([0] + sizes, dtype=torch.int64).cumsum(0)
        s["offsets"] = ends.to(torch.int32).cuda()
        s["most"] = max(max(sizes), 1)
        s["expert"] = torch.repeat_interleave(torch.arange(g), torch.tensor(sizes)).cuda()
        s["place"] = torch.arange(m, device="cuda") - ends.cuda()[s["expert"]]
    return s


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    if case["op"] in ("linear", "experts"):
        # the weight as a serving program keeps it: quantised once
        if own:
            from quantised_linear_layers_gb300 import fp4, ops
            fmt = {"nv": ops.FP4_NV, "mx": ops.FP4_MX}[case["fmt"]]
            s["w4"] = (fp4.FP4Weight if case["op"] == "linear" else fp4.FP4ExpertWeight)(s["w"], fmt, dgrad=False)
        else:
            s["wv"] = _values(s["w"], case["fmt"], _tensor_scale(s["w"]))
        del s["w"]
    return s


# ---------------------------------------------------------------- plain form
def _tensor_scale(x):
    f, e = torch.frexp(x.abs().amax().float())
    return torch.ldexp(torch.ones_like(f), (e - 12 + (f > 0.65625)).clamp(min=-80))


def _values(x, fmt, tensor_scale=None):
    """x along its last axis through the 4-bit format, as the fp32 values it then stands for."""
    g = GROUP[fmt]
    k = x.shape[-1]
    x = torch.nn.functional.pad(x.float(), (0, -k % g)).unflatten(-1, (-1, g))
    amax = x.abs().amax(-1, keepdim=True)
    if fmt == "nv":
        t = torch.ones((), device=x.device) if tensor_scale is None else tensor_scale
        s = (amax / (6.0 * t)).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn).float() * t
    else:
        f, e = torch.frexp(amax)
        s = torch.ldexp(torch.ones_like(amax), (e - 3 + (f > 0.75)).clamp(-127, 127))
    y = x / s
    a = y.abs()
    q = 0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75) + (a > 2.5) + (a >= 3.5) \
        + 2.0 * (a > 5.0)
    return (torch.copysign(q, y) * s).flatten(-2)[..., :k]


def _spread(s, rows):
    """Rows sorted by expert as [experts, most rows of one, columns], zeros in the rest."""
    g = s["case"]["experts"]
    out = torch.zeros((g, s["most"], rows.shape[1]), device=rows.device)
    out[s["expert"], s["place"]] = rows.float()
    return out


def _plain(s):
    case = s["case"]
    op, fmt, x = case["op"], case["fmt"], s["x"]
    if op == "cast":
        return _values(x, fmt, _tensor_scale(x) if case["dynamic"] else None).bfloat16()
    if op == "linear":
        return (_values(x, fmt) @ s["wv"].t()).bfloat16()
    if op == "experts":
        y = torch.bmm(_spread(s, _values(x, fmt)), s["wv"].transpose(1, 2))
        return y[s["expert"], s["place"]].bfloat16()
    dy, w = s["dy"], s["w"]
    sx, sw, sd = _tensor_scale(x), _tensor_scale(w), _tensor_scale(dy)
    w_fwd, w_bwd = _values(w, fmt, sw), _values(w.transpose(-1, -2), fmt, sw)
    xv, dv = _values(x, fmt, sx), _values(dy, fmt, sd)
    if op == "train":
        y, dx = xv @ w_fwd.t(), dv @ w_bwd.t()
        dw = _values(dy.t(), fmt, sd) @ _values(x.t(), fmt, sx).t()
        return {"y": y.bfloat16(), "dx": dx.bfloat16(), "dw": dw}
    at = (s["expert"], s["place"])
    y = torch.bmm(_spread(s, xv), w_fwd.transpose(1, 2))[at]
    dx = torch.bmm(_spread(s, dv), w_bwd.transpose(1, 2))[at]
    dw = torch.bmm(_values(_spread(s, dy).transpose(1, 2), fmt, sd),
                   _values(_spread(s, x).transpose(1, 2), fmt, sx).transpose(1, 2))
    return {"y": y.bfloat16(), "dx": dx.bfloat16(), "dw": dw}


# ---------------------------------------------------------------- a user's calls
def _calls(s):
    from quantised_linear_layers_gb300 import fp4, ops
    case = s["case"]
    op, x = case["op"], s["x"]
    fmt = ops.FP4_NV if case["fmt"] == "nv" else ops.FP4_MX
    if op == "cast":
        a = ops.fp4_cast(x, fmt, ops.fp4_tensor_scale(x) if case["dynamic"] else None)
        return ops.fp4_dequant(a)
    if op == "linear":
        return fp4.forward(x, s["w4"])
    if op == "experts":
        return fp4.experts_forward(x, s["offsets"], s["w4"])
    if op == "train":
        w4 = fp4.FP4Weight(s["w"], fmt)
        y, saved = fp4.forward_saving(x, w4)
        dx, dw = fp4.backward(s["dy"], w4, saved)
    else:
        w4 = fp4.FP4ExpertWeight(s["w"], fmt)
        y, saved = fp4.experts_forward_saving(x, s["offsets"], w4)
        dx, dw = fp4.experts_backward(s["dy"], s["offsets"], w4, saved)
    return {"y": y, "dx": dx, "dw": dw}


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits
def _nearest(y, man_bits, least_exp):
    """y on a binary grid of man_bits fraction bits and smallest exponent least_exp, ties to even."""
    _, e = torch.frexp(y)
    step = torch.exp2((e.double() - 1).clamp(min=least_exp) - man_bits)
    return torch.round(y / step) * step


def _exact_values(x, fmt, tensor_scale=1.0):
    g = GROUP[fmt]
    rows, k = x.reshape(-1, x.shape[-1]).double(), x.shape[-1]
    out = torch.empty_like(rows)
    full = k // g * g
    for part in (rows[:, :full].reshape(-1, g) if full else None, rows[:, full:] if k > full else None):
        if part is None:
            continue
        amax = part.abs().max(dim=1, keepdim=True).values
        if fmt == "nv":
            s = _nearest(torch.clamp(amax / (6 * tensor_scale), 2.0 ** -9, 448.0), 3, -6) * tensor_scale
        else:
            f, e = torch.frexp(torch.clamp(amax, min=2.0 ** -120) / 6)
            s = torch.exp2((e - (f == 0.5).int()).double())
        v = torch.clamp(_nearest(part / s, 1, 0), -6, 6) * s
        if part.shape[1] == g:
            out[:, :full] = v.reshape(rows.shape[0], full)
        else:
            out[:, full:] = v
    return out.reshape(x.shape)


def exact(case, seed):
    s = _inputs(case, seed)
    op, fmt, x = case["op"], case["fmt"], s["x"]
    scale = lambda v: 2.0 ** max(-80, math.ceil(math.log2(v.double().abs().max().item() / 2688)))  # noqa: E731
    if op == "cast":
        return _exact_values(x, fmt, scale(x) if case["dynamic"] else 1.0)
    w = s["w"]
    if op == "linear":
        return _exact_values(x, fmt) @ _exact_values(w, fmt, scale(w)).t()
    spans = [(0, case["m"])]
    if "experts" in case:
        ends = s["offsets"].tolist()
        spans = list(zip(ends[:-1], ends[1:]))
    ws = w if w.dim() == 3 else w[None]
    if op == "experts":
        wv = _exact_values(ws, fmt, scale(w))
        xv = _exact_values(x, fmt)
        return torch.cat([xv[a:b] @ wv[i].t() for i, (a, b) in enumerate(spans)])
    dy, sx, sw, sd = s["dy"], scale(x), scale(w), scale(s["dy"])
    xv, dv = _exact_values(x, fmt, sx), _exact_values(dy, fmt, sd)
    y, dx, dw = [], [], []
    for i, (a, b) in enumerate(spans):
        y.append(xv[a:b] @ _exact_values(ws[i], fmt, sw).t())
        dx.append(dv[a:b] @ _exact_values(ws[i].t().contiguous(), fmt, sw).t())
        if a == b:
            dw.append(torch.zeros(ws[i].shape, dtype=torch.float64, device=x.device))
        else:
            dw.append(_exact_values(dy[a:b].t().contiguous(), fmt, sd)
                      @ _exact_values(x[a:b].t().contiguous(), fmt, sx).t())
    dw = torch.stack(dw) if w.dim() == 3 else dw[0]
    return {"y": torch.cat(y), "dx": torch.cat(dx), "dw": dw}
