"""4-bit calls on tensors with a dimension of size one, whose stride says nothing:
torch calls such a tensor contiguous whatever it is. What lies behind each
tensor is in its allocation and large, so that a stride taken at its word shows
in the scale."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
from fp4_checks import acts, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantised_linear_layers_gb300 import build, ops as o
    build.build()
    o.load_library()
    return o


def inside(shape, stride, seed, dtype):
    """A view of this shape and stride over the start of a buffer, 1e6 in every element past its last."""
    last = sum((n - 1) * s for n, s in zip(shape, stride) if n > 1)
    buf = torch.full((64 * 1024,), 1e6, dtype=dtype, device="cuda")
    x = buf.as_strided(shape, stride)
    # rows of elements that lie one after the other, filled through the view itself
    x.copy_(acts(*shape, seed=seed, dtype=dtype).reshape(shape))
    assert last < 16 * 1024
    return x


# [batch, rows, columns]; strides of dimensions of size one are not those of a new tensor
VIEWS = [((4, 1, 64), (64, 256, 1)), ((4, 1, 64), (64, 1, 1)), ((1, 5, 64), (17, 64, 1)), ((4, 1, 33), (33, 132, 1)),
         ((4, 1, 64), (128, 4096, 1)), ((3, 7, 1), (7, 1, 7)), ((3, 7, 1), (7, 1, 4096)), ((1, 1, 64), (3, 4096, 1)),
         ((5, 1, 1), (1, 4096, 4096))]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape,stride", VIEWS, ids=["x".join(map(str, a)) + "_" + "_".join(map(str, b)) for a, b in VIEWS])
def test_batches_with_a_size_of_one(ops, shape, stride, dtype):
    x = inside(shape, stride, 3, dtype)
    want = ref.tensor_scale(np64(x))
    assert float(ops.fp4_tensor_scale(x)) == want
    plain = x.clone(memory_format=torch.contiguous_format).reshape(-1).clone().reshape(shape)
    a, b = ops.fp4_cast(x, 0, ops.FP4_OWN_SCALE), ops.fp4_cast(plain, 0, ops.FP4_OWN_SCALE)
    assert float(a.scale) == want and torch.equal(a.q, b.q)
    both = ops.fp4_cast_dual(x, 0, ops.FP4_OWN_SCALE)
    for got, exp in zip(both, ops.fp4_cast_dual(plain, 0, ops.FP4_OWN_SCALE)):
        assert float(got.scale) == want
        assert torch.equal(got.q[:, :(got.cols + 1) // 2], exp.q[:, :(got.cols + 1) // 2])


@pytest.mark.parametrize("shape,stride", [((1, 64), (4096, 1)), ((1, 64), (3, 1)), ((7, 1), (1, 4096)), ((1, 64), (1, 7))],
                         ids=["row", "row3", "column", "spread"])
def test_matrices_with_a_size_of_one(ops, shape, stride):
    x = inside(shape, stride, 5, torch.bfloat16)
    w = acts(48, shape[1], seed=2)
    plain = x.reshape(-1).clone().reshape(shape)
    wq = ops.fp4_cast(w, 0, ops.FP4_OWN_SCALE)
    assert float(ops.fp4_tensor_scale(x)) == ref.tensor_scale(np64(x))
    assert torch.equal(ops.fp4_linear(x, wq, ops.FP4_OWN_SCALE), ops.fp4_linear(plain, wq, ops.FP4_OWN_SCALE))
    assert torch.equal(ops.fp4_cast(x, 1).q, ops.fp4_cast(plain, 1).q)


def test_experts_of_one_output_feature(ops):
    """A weight [experts, 1, in] made by transposing [1, experts, in]."""
    from quantised_linear_layers_gb300 import fp4
    w = acts(1, 4, 64, seed=1).transpose(0, 1)
    assert w.is_contiguous() and w.stride(1) == 256
    got, want = fp4.FP4ExpertWeight(w), fp4.FP4ExpertWeight(w.reshape(-1).clone().reshape(4, 1, 64))
    assert float(got.w.scale) == float(want.w.scale) == ref.tensor_scale(np64(w))
    off = torch.tensor([0, 3, 3, 4, 9], dtype=torch.int32, device="cuda")
    x = acts(9, 64, seed=2)
    y, saved = fp4.experts_forward_saving(x, off, got)
    assert torch.equal(y, fp4.experts_forward(x, off, want, "own")) and np.isfinite(np64(y)).all()
    dx, dw = fp4.experts_backward(acts(9, 1, seed=3), off, got, saved)
    dx2, dw2 = fp4.experts_backward(acts(9, 1, seed=3), off, want, saved)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and dw.shape == (4, 1, 64)


def test_own_scale_of_interleaved_matrices(ops):
    """[batch, rows, columns] views whose rows follow one another, columns far apart."""
    big = acts(40, 3 * 7, seed=4)                    # [columns, batch * rows]
    x = big.view(40, 3, 7).permute(1, 2, 0)          # strides (7, 1, 21)
    a = ops.fp4_cast(x, 0, ops.FP4_OWN_SCALE)
    b = ops.fp4_cast(x.contiguous(), 0, ops.FP4_OWN_SCALE)
    assert float(a.scale) == ref.tensor_scale(np64(big)) and torch.equal(a.q, b.q)
