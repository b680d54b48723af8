"""4-bit calls of experts that leave rows out, of many experts and of tensors with
dimensions of size one, for the bounds-checked build: each call's outputs and
the device status after it. Run in a process whose ops module loaded either
build of the library."""
import numpy as np
import torch

from fp4_bounds_cases import _acts, _np


def run(ops):
    """Returns {case name: (list of output arrays, device status after it)}."""
    out = {}

    def rec(name, tensors):
        torch.cuda.synchronize()
        out[name] = ([_np(t) for t in tensors], ops.device_status())

    sets = {"padded": (133, [3, 40, 40, 120]), "few": (16, [1, 3, 3, 12]), "none": (40, [7, 7, 7, 7]),
            "many": (90, [5] + [5 + i // 2 for i in range(1, 101)])}
    for fmt in (0, 1):
        own = ops.FP4_OWN_SCALE if fmt == 0 else None
        for name, (m, offs) in sets.items():
            off, e = torch.tensor(offs, dtype=torch.int32, device="cuda"), len(offs) - 1
            for n, k in ((136, 96), (131, 67)):
                x, dy = _acts(m, k, 3), _acts(m, n, 4)
                x[:offs[0]], dy[offs[-1]:] = float("nan"), float("inf")
                wr, wc = ops.fp4_cast_dual(torch.stack([_acts(n, k, 5 + i) for i in range(e)]), fmt, own)
                for path in (0, 2, 3):
                    ops.set_gemm_path(path)
                    try:
                        y, saved = ops.fp4_linear_saving(x, wr, own, off)
                        dx, dw = ops.fp4_linear_backward(dy, wc, saved, own, off)
                        f = ops.gemm_fp4_nt_ragged(ops.fp4_cast(x, fmt, own, off), wr, dtype=torch.float32)
                        rec(f"step_{name}_{n}x{k}_p{path}_f{fmt}", [y, dx, dw, f, ops.fp4_linear(x, wr, own, off)])
                    finally:
                        ops.set_gemm_path(0)
    off = torch.tensor([5, 700, 1100], dtype=torch.int32, device="cuda")
    for k, dtype in ((1024, torch.bfloat16), (1031, torch.bfloat16), (1031, torch.float32)):
        x = _acts(1200, k + 8, 1, dtype)
        for name, v in (("rows", x), ("off", x[:, 3:]), ("wide", x[:, 8:])):
            scales = [ops.fp4_cast(v, 0, ops.FP4_OWN_SCALE, off).scale, ops.fp4_tensor_scale(v),
                      ops.fp4_cast(v[:300], 0, ops.FP4_OWN_SCALE, off[:2]).scale]
            rec(f"scale_{name}_{k}_{'bf16' if dtype == torch.bfloat16 else 'f32'}", scales)
    base = _acts(1, 4 * 64, 2)
    for name, v in (("rows", base.view(1, 4, 64).transpose(0, 1)), ("turned", base.view(4, 64, 1).transpose(1, 2)),
                    ("column", base.view(4, 64, 1)), ("row", base.as_strided((1, 1, 256), (1, 4096, 1)))):
        a = ops.fp4_cast(v, 0, ops.FP4_OWN_SCALE)
        both = ops.fp4_cast_dual(v, 0, ops.FP4_OWN_SCALE)
        rec(f"one_{name}", [ops.fp4_tensor_scale(v), a.scale, a.q] + [c.q for c in both])
    return out


if __name__ == "__main__":
    import sys
    from quantised_linear_layers_gb300 import ops
    arrays = {}
    for name, (arrs, st) in run(ops).items():
        arrays[f"{name}__status"] = np.array([st])
        for i, arr in enumerate(arrs):
            arrays[f"{name}__{i}"] = arr
    np.savez(sys.argv[1], **arrays)
    print("flag", int(ops.load_library().ql_bounds_checked()))
