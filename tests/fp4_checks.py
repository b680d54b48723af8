"""Inputs and the comparison with 64 bits that the 4-bit layers' tests share."""
import numpy as np
import torch

import fp4_reference as ref


def acts(*shape, seed, dtype=torch.bfloat16, mul=1.0):
    """Rows of different loudness, on the GPU."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-3, 4, (*shape[:-1], 1), generator=g).float())
    return (x * mul).to(dtype).cuda()


def np64(x):
    return x.detach().float().cpu().numpy().astype(np.float64)


def check(got, xv, wv, d0=None):
    """got = xv wv^T (+ d0) within fp4_reference.bound, or for bf16 the rounding of a value within it. Written so that
    a NaN is outside of every bound."""
    want, absum = ref.product(xv, wv)
    if d0 is not None:
        want, absum = want + d0, absum + np.abs(d0)
    is_bf16, got = got.dtype == torch.bfloat16, np64(got)
    e = ref.bound(absum, xv.shape[1])
    ok = (got >= ref.bf16(want - e)) & (got <= ref.bf16(want + e)) if is_bf16 else np.abs(got - want) <= e
    assert ok.all(), f"{int((~ok).sum())} of {ok.size} off: {got[~ok][:4]} for {want[~ok][:4]}, bound {e[~ok][:4]}"
