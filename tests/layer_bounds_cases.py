"""Small cases of layer norm, routing and the exchange over every kernel and form, for the
bounds-checked build: each call's outputs (as numpy arrays) and the device status after it.
Run in a process whose ops module loaded either build of the library."""
import numpy as np
import torch

BF, F = torch.bfloat16, torch.float32


def _np(t):
    t = t.detach()
    return (t.view(torch.int16) if t.dtype == BF else t).cpu().numpy().copy()


def _rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def run(ops):
    """Returns {case name: (list of output arrays, device status after it)}."""
    out = {}

    def rec(name, *tensors):
        torch.cuda.synchronize()
        out[name] = ([_np(t) for t in tensors], ops.device_status())

    for dtype in (BF, F):
        for y_dtype in (BF, F):
            for m, n in ((1, 1), (3, 40), (700, 33), (3, 257), (170, 1003), (2000, 1032), (1900, 1031), (2, 4099), (1000, 2051), (3, 8200),
                         (900, 8195), (2, 16384), (2, 17000)):
                wide = _rand((m, n + 9), dtype, m + n)
                w, b = _rand((n,), F, 1), _rand((n,), F, 2)
                for tag, x in (("whole", wide[:, :n].contiguous()), ("off", wide[:, 1:n + 1]), ("far", wide[:, 8:n + 8])):
                    y, stats = ops.layer_norm_saving(x, w, b, dtype=y_dtype)
                    rec(f"norm_{tag}_{m}x{n}_{dtype}_{y_dtype}", y, stats, ops.layer_norm(x, w.to(BF), None, dtype=y_dtype))
                    dy = _rand((m, n), y_dtype, 3)
                    rec(f"norm_back_{tag}_{m}x{n}_{dtype}_{y_dtype}", *ops.layer_norm_backward(dy, x, stats, w),
                        ops.layer_norm_backward(dy, x, stats, None)[0])
        for m, n, k, how in ((5, 1, 1, {}), (9, 20, 3, {}), (9, 64, 6, {}), (9, 162, 6, dict(groups=9, kept=3)), (9, 100, 8, dict(groups=4, kept=2, group_best=2)),
                             (9, 256, 8, dict(groups=8, kept=4, group_best=2)), (9, 512, 32, {}), (9, 500, 4, dict(groups=2, kept=1, group_best=2))):
            wide = _rand((m, n + 3), dtype, n)
            near = torch.round(wide.float() * 2).to(dtype)      # many ties: the paths in 64 bits
            for tag, x in (("whole", wide[:, :n].contiguous()), ("off", wide[:, 1:n + 1]), ("near", near[:, :n])):
                for score in ("softmax", "sigmoid"):
                    for bias in (None, _rand((n,), F, 5) * 1e-7, _rand((n + 1,), F, 5)[1:].contiguous()):
                        for re in (False, True):
                            w, e = ops.route(x, k, bias, score, renormalise=re, **how)
                            rec(f"route_{tag}_{n}_{dtype}_{score}_{re}_{bias is None}_{0 if bias is None else float(bias.abs().max()) < 1e-3}", w, e,
                                ops.route_backward(_rand((m, k), F, 6), x, e, score, re))
        for m, k, n, cols in ((1, 1, 1, 1), (17, 3, 5, 33), (40, 8, 256, 1024), (300, 9, 31, 520), (700, 8, 64, 2056), (2500, 2, 8, 264), (2500, 1, 8, 512),
                              (700, 2, 8, 4104), (2500, 4, 8, 260), (5, 17, 8, 4096), (20, 2, 8, 1003)):
            g = torch.Generator().manual_seed(m)
            e = torch.randint(-1, n, (m, k), generator=g).to(torch.int32).cuda()
            p = ops.expert_plan(e, n)
            rec(f"plan_{m}x{k}of{n}_{dtype}_{cols}", p.offsets, p.rows)
            w = _rand((m, k), F, 1)
            for tag, cut in (("whole", slice(0, cols)), ("off", slice(1, cols + 1)), ("far", slice(8, cols + 8))):
                x, ys = _rand((m, cols + 9), dtype, 2)[:, cut], _rand((m * k, cols + 9), dtype, 3)[:, cut]
                dy, add = _rand((m, cols + 9), dtype, 4)[:, cut], _rand((m, cols + 9), dtype, 5)[:, cut]
                rec(f"rows_{tag}_{m}x{k}of{n}x{cols}_{dtype}", ops.expert_dispatch(x, p), ops.expert_combine(ys, p, w, add), ops.expert_combine(ys, p),
                    *ops.expert_combine_backward(dy, ys, p, w))
    return out


if __name__ == "__main__":
    import sys
    from quantised_linear_layers_gb300 import ops
    res = run(ops)
    arrays = {}
    for name, (arrs, st) in res.items():
        arrays[f"{name}__status"] = np.array([st])
        for i, arr in enumerate(arrs):
            arrays[f"{name}__{i}"] = arr
    np.savez(sys.argv[1], **arrays)
    print("flag", int(ops.load_library().ql_bounds_checked()))
