"""Small 4-bit cases over every kernel and form, for the bounds-checked build:
each call's outputs (as numpy arrays) and the device status after it. Run in a
process whose ops module loaded either build of the library."""
import numpy as np
import torch


def _np(t):
    t = t.detach()
    return (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy().copy()


def _acts(m, k, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((m, k), generator=g).to(dtype).cuda()


def run(ops):
    """Returns {case name: (list of output arrays, device status after it)}."""
    out = {}

    def rec(name, tensors):
        torch.cuda.synchronize()
        out[name] = ([_np(t) for t in tensors], ops.device_status())

    offs = torch.tensor([0, 0, 70, 71, 130], dtype=torch.int32, device="cuda")
    for fmt in (0, 1):
        for dtype in (torch.bfloat16, torch.float32):
            tag = f"f{fmt}_{'bf16' if dtype == torch.bfloat16 else 'f32'}"
            for m, k in ((1, 1), (130, 520), (7, 1031), (129, 64)):
                x = _acts(m, k, m + k, dtype)
                for name, v in (("rows", x), ("off", x[:, 1:]), ("wide", x[:, ::2]), ("turned", x.t())):
                    if v.shape[1] == 0:
                        continue
                    scale = ops.FP4_OWN_SCALE if fmt == 0 else None
                    a = ops.fp4_cast(v, fmt, scale)
                    # codes past the last column's byte and scale rows past the last row are not written
                    rec(f"cast_{name}_{m}x{k}_{tag}", [a.q[:, :(v.shape[1] + 1) // 2]])
                    rec(f"read_{name}_{m}x{k}_{tag}", [ops.fp4_dequant(a), ops.fp4_dequant(a, torch.float32)])
                    if v.stride(1) == 1:
                        r, c = ops.fp4_cast_dual(v, fmt, scale)
                        rec(f"dual_{name}_{m}x{k}_{tag}", [ops.fp4_dequant(r), ops.fp4_dequant(c)])
            x, w = _acts(9, 515, 1, dtype), _acts(300, 515, 2)
            wq = ops.fp4_cast(w, fmt)
            for m in (1, 8, 9):
                rec(f"linear_{m}_{tag}", [ops.fp4_linear(x[:m], wq), ops.fp4_linear(x[:m, :512], ops.fp4_cast(w[:, :512], fmt))])
        w = _acts(300, 4099, 2)
        wq = ops.fp4_cast(w, fmt)
        for m in (1, 40, 130, 300):
            a = ops.fp4_cast(_acts(m, 4099, m), fmt)
            for path in (0, 2, 3):
                ops.set_gemm_path(path)
                try:
                    d = torch.ones((m, 300), device="cuda")
                    ops.gemm_fp4_nt(a, wq, out=d, accumulate=True)
                    wide = torch.zeros((m, 310), dtype=torch.bfloat16, device="cuda")
                    ops.gemm_fp4_nt(a, wq, out=wide[:, 3:303])
                    rec(f"gemm_{m}_p{path}_f{fmt}", [ops.gemm_fp4_nt(a, wq), d, wide])
                finally:
                    ops.set_gemm_path(0)
        x, dy = _acts(133, 200, 3), _acts(133, 260, 4)
        we = torch.stack([_acts(260, 200, 5 + e) for e in range(4)])
        wr = ops.fp4_cast_dual(we, fmt)[0]
        ar, ac = ops.fp4_cast_dual(x, fmt, None, offs)
        yc = ops.fp4_cast_dual(dy, fmt, None, offs, rows=False)[1]
        for path in (0, 2, 3):
            ops.set_gemm_path(path)
            try:
                o = torch.zeros((133, 260), dtype=torch.bfloat16, device="cuda")
                ops.gemm_fp4_nt_ragged(ar, wr, out=o)
                o2 = torch.zeros((133, 260), dtype=torch.bfloat16, device="cuda")
                ops.gemm_fp4_nt_ragged(ops.fp4_cast(x, fmt, offsets=offs), wr, out=o2)
                rec(f"experts_p{path}_f{fmt}", [o, o2, ops.gemm_fp4_wgrad_ragged(yc, ac)])
            finally:
                ops.set_gemm_path(0)
        few = torch.tensor([0, 2, 2, 3, 8], dtype=torch.int32, device="cuda")
        rec(f"experts_linear_f{fmt}", [ops.fp4_linear(x[:8], wr, offsets=few), ops.fp4_linear(x[:130], wr, offsets=offs)])
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
