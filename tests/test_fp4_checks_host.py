"""The comparison of the 4-bit tests (fp4_checks.check) itself."""
import numpy as np
import pytest
import torch

from fp4_checks import check

BF16_UP = {torch.bfloat16: 2.0 ** -7, torch.float32: 2.0 ** -15}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bad", ["nan", "inf", "step"])
def test_check_rejects(dtype, bad):
    """One element that is NaN, infinite or a step of bf16 (fp32: of 2^-15, above
    the bound of 9 * 2^-23 of sum |x| |w|, about 130 beside a value of about 40) away."""
    rng = np.random.default_rng(0)
    x, w = rng.integers(-4, 5, (7, 64)) * 0.5, rng.integers(-4, 5, (9, 64)) * 0.5
    x[:, 0], w[:, 0] = 6, 6
    good = torch.from_numpy(x @ w.T).to(dtype)
    check(good, x, w)
    got = good.clone()
    got[3, 5] = {"nan": float("nan"), "inf": float("inf"), "step": float(good[3, 5]) * (1 + BF16_UP[dtype]) + 2.0 ** -9}[bad]
    with pytest.raises(AssertionError):
        check(got, x, w)
    got[3, 5] = good[3, 5]
    check(got, x, w)
