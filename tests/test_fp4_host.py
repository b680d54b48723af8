"""4-bit operators without a GPU: sizes, and the C entry points' refusals from
host checks alone; the numpy reference against closed forms."""
import ctypes

import numpy as np
import pytest

import fp4_reference as ref


@pytest.fixture(scope="module")
def L():
    from quantised_linear_layers_gb300 import build, ops
    build.build()
    return ops.load_library()


def test_sizes(L):
    assert L.fp4_scale_bytes(1, 1, 0, 0) == 512
    assert L.fp4_scale_bytes(128, 64, 0, 0) == 512 and L.fp4_scale_bytes(129, 65, 0, 0) == 4 * 512
    assert L.fp4_scale_bytes(128, 128, 1, 0) == 512 and L.fp4_scale_bytes(128, 129, 1, 0) == 2 * 512
    assert L.fp4_scale_bytes(300, 256, 0, 8) == (3 + 8) * 4 * 512
    assert L.fp4_scale_bytes(0, 64, 0, 0) == 0
    assert L.fp4_scale_bytes(-1, 64, 0, 0) == -1 and L.fp4_scale_bytes(1, 64, 2, 0) == -1
    assert L.fp4_column_extent(1, 0) == 128 and L.fp4_column_extent(129, 0) == 256
    assert [L.fp4_row_stride(k) for k in (0, 1, 32, 33, 64, 65, 128, 129, 256, 257, 2051)] == \
        [16, 16, 16, 32, 32, 48, 64, 128, 128, 256, 1152]
    # any split of 257 rows over 3 experts needs at most 1 + 1 + 2 multiples of 256, and a room for one more
    assert L.fp4_column_extent(257, 3) == 5 * 256
    assert all(sum(-(-c // 256) for c in (a, b, 257 - a - b)) <= 5 for a in range(0, 258, 37) for b in range(0, 258 - a, 29))


def test_refused_before_cuda(L):
    p, u = ctypes.c_void_p(64), ctypes.c_void_p(72)
    C = L.fp4_cast
    assert C(p, 0, 1, 4, 64, 0, 64, 1, 2, None, 0, p, 32, p, None, 0, None) == 1          # unknown format
    assert C(p, 5, 1, 4, 64, 0, 64, 1, 0, None, 0, p, 32, p, None, 0, None) == 1          # unknown type
    assert C(p, 0, 1, -4, 64, 0, 64, 1, 0, None, 0, p, 32, p, None, 0, None) == 1         # negative size
    assert C(None, 0, 1, 4, 64, 0, 64, 1, 0, None, 0, p, 32, p, None, 0, None) == 1       # null input
    assert C(p, 0, 1, 4, 64, 0, 64, 1, 0, None, 0, None, 32, p, None, 0, None) == 1       # null codes
    assert C(p, 0, 1, 4, 64, 0, 64, 1, 0, None, 0, p, 16, p, None, 0, None) == 1          # codes' rows too short
    assert C(p, 0, 1, 4, 64, 0, 64, 1, 0, None, 0, p, 40, p, None, 0, None) == 3          # row stride not of 16 bytes
    assert C(p, 0, 1, 4, 64, 0, 64, 1, 0, None, 0, u, 32, p, None, 0, None) == 3          # misaligned codes
    assert C(p, 0, 1, 4, 64, 0, 64, 1, 0, None, 0, p, 32, u, None, 0, None) == 3          # misaligned scales
    assert C(p, 0, 2, 4, 64, 0, 64, 1, 0, None, 0, p, 32, p, p, 2, None) == 1             # offsets with a batch
    assert C(p, 0, 1, 4, 64, 0, 64, 1, 0, None, 0, p, 32, p, p, 0, None) == 1             # no experts
    assert C(p, 0, 1, 4, 64, 0, 64, 1, 0, None, 0, p, 32, p, p, 513, None) == 2           # too many
    assert C(p, 0, 1, 1 << 31, 64, 0, 64, 1, 0, None, 0, p, 32, p, None, 0, None) == 2
    assert C(p, 0, 1 << 30, 1, 64, 64, 64, 1, 0, None, 0, p, 32, p, None, 0, None) == 2    # more scale blocks than a grid has
    assert C(None, 0, 1, 0, 64, 0, 64, 1, 0, None, 0, None, 32, None, None, 0, None) == 0  # nothing to do
    assert C(p, 0, 1, 4, 64, 0, 64, 1, 0, None, 1, p, 32, p, None, 0, None) == 1       # own scale, nowhere to put it
    assert C(p, 0, 1, 4, 64, 0, 64, 1, 1, p, 1, p, 32, p, None, 0, None) == 1          # MX has none
    D = L.fp4_cast_dual
    assert D(p, 0, 1, 4, 64, 0, 64, 0, None, 0, p, 32, None, p, 64, p, None, 0, None) == 1  # codes without scales
    assert D(p, 0, 1, 4, 64, 0, 64, 0, None, 0, p, 32, p, p, 48, p, None, 0, None) == 1     # columns too short
    assert D(p, 0, 1, 4, 64, 0, 64, 7, None, 0, p, 32, p, p, 64, p, None, 0, None) == 1
    assert D(p, 0, 0, 4, 64, 0, 64, 0, None, 0, p, 32, p, p, 64, p, None, 0, None) == 0
    Q = L.fp4_dequant
    assert Q(p, 32, p, 3, None, 4, 64, p, 0, 64, None) == 1
    assert Q(p, 32, p, 0, None, 4, 64, p, 0, 63, None) == 1
    assert Q(p, 32, p, 0, None, 4, 64, p, 7, 64, None) == 1
    G = L.gemm_fp4_nt
    assert G(p, 32, p, None, p, 32, p, None, 2, p, 0, 8, 4, 8, 64, 0, None) == 1         # unknown format
    assert G(p, 32, p, None, p, 32, p, None, 0, p, 0, 7, 4, 8, 64, 0, None) == 1         # D's rows too short
    assert G(p, 32, p, None, p, 32, p, None, 0, p, 0, 8, 4, 8, 64, 1, None) == 1         # bf16 accumulation
    assert G(p, 32, p, None, p, 32, p, None, 0, None, 0, 8, 4, 8, 64, 0, None) == 1
    assert G(p, 32, None, None, p, 32, p, None, 0, p, 0, 8, 4, 8, 64, 0, None) == 1
    assert G(u, 32, p, None, p, 32, p, None, 0, p, 0, 8, 4, 8, 64, 0, None) == 3
    assert G(p, 32, p, None, p, 40, p, None, 0, p, 0, 8, 4, 8, 64, 0, None) == 3
    assert G(None, 32, None, None, p, 32, p, None, 0, p, 0, 8, 0, 8, 64, 0, None) == 0
    R = L.gemm_fp4_nt_ragged
    assert R(p, 32, p, None, p, 32, p, None, 0, p, 0, 8, None, 2, 4, 8, 64, None) == 1   # no offsets
    assert R(p, 32, p, None, p, 32, p, None, 0, p, 0, 8, p, 0, 4, 8, 64, None) == 1
    assert R(p, 32, p, None, p, 32, p, None, 0, p, 0, 8, p, 600, 4, 8, 64, None) == 2
    assert R(p, 32, p, None, p, 32, p, None, 0, p, 0, 8, p, 2, 4, 8, 0, None) == 2       # k == 0
    F = L.fp4_linear
    assert F(p, 0, 64, None, 0, p, 32, p, None, 2, p, 8, None, 0, 4, 8, 64, None, 0, None) == 1     # unknown format
    assert F(p, 0, 64, None, 0, p, 32, p, None, 0, p, 8, None, 0, 4, 0, 64, None, 0, None) == 0     # nothing to do
    assert F(p, 0, 64, None, 0, p, 32, p, None, 0, p, 8, None, 0, -4, 8, 64, None, 0, None) == 1    # negative size
    assert F(p, 0, 64, None, 1, p, 32, p, None, 0, p, 8, None, 0, 4, 8, 64, None, 0, None) == 1     # own scale, nowhere to put it
    assert F(p, 3, 64, None, 0, p, 32, p, None, 0, p, 8, None, 0, 4, 8, 64, None, 0, None) == 1     # unknown type
    assert F(p, 0, 64, None, 0, p, 32, p, None, 0, p, 7, None, 0, 4, 8, 64, None, 0, None) == 1     # D's rows too short
    assert F(None, 0, 64, None, 0, p, 32, p, None, 0, p, 8, None, 0, 4, 8, 64, None, 0, None) == 1
    assert F(p, 0, 64, None, 0, p, 40, p, None, 0, p, 8, None, 0, 4, 8, 64, None, 0, None) == 3
    assert F(p, 0, 64, None, 0, p, 32, p, None, 0, p, 8, p, 0, 4, 8, 64, None, 0, None) == 1        # offsets, no experts
    assert F(p, 0, 64, None, 0, p, 32, p, None, 0, p, 8, p, 600, 4, 8, 64, None, 0, None) == 2
    assert F(p, 0, 64, None, 0, p, 32, p, None, 0, p, 8, None, 0, 70, 8, 64, None, 0, None) == 1    # no workspace
    assert F(p, 0, 64, None, 0, p, 32, p, None, 0, p, 8, None, 0, 70, 8, 64, p, 10, None) == 1
    assert L.fp4_linear_workspace_size(8, 7168, 0, 0) == 0
    assert L.fp4_linear_workspace_size(70, 65, 0, 0) == 70 * 48 + 2 * 512
    W = L.gemm_fp4_wgrad_ragged
    assert W(p, 1024, p, None, p, 1024, p, None, 0, p, 8, None, 2, 4, 4, 8, 0, None) == 1
    assert W(p, 16, p, None, p, 1024, p, None, 0, p, 8, p, 2, 4, 4, 8, 0, None) == 1     # columns too short
    assert L.fp4_tensor_scale(p, 0, 4, 4, 4, 1, None, None) == 1


def test_reference_closed_forms():
    codes = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    row = np.array([codes + [-c for c in codes]])
    for fmt in (ref.NV, ref.MX):
        assert np.array_equal(ref.values(row, fmt), row)                    # scale 1: every code stands for itself
        assert np.array_equal(ref.values(row * 2.0 ** 5, fmt), row * 2.0 ** 5)
    mids = np.array([[6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] + [0] * 8])
    assert np.array_equal(ref.values(mids, ref.NV)[0, :8], [6, 0, 1, 1, 2, 2, 4, 4])    # ties to the even code
    assert ref.scales(np.array([[6.5]]), ref.MX)[0, 0] == 2 and ref.scales(np.array([[6.0]]), ref.MX)[0, 0] == 1
    assert ref.scales(np.array([[0.0]]), ref.NV)[0, 0] == 2.0 ** -9
    assert ref.scales(np.array([[6 * 1.0625]]), ref.NV)[0, 0] == 1.0        # E4M3 tie to even: 1, not 1.125
    assert ref.tensor_scale(np.array([[2688.0]])) == 1 and ref.tensor_scale(np.array([[2689.0]])) == 2
    assert np.isnan(ref.values(np.array([[1.0, np.inf]]), ref.NV)).all()


def test_module_fails_loudly_when_missing(monkeypatch, tmp_path):
    from quantised_linear_layers_gb300 import ops
    monkeypatch.setattr(ops, "_fp4", None)
    monkeypatch.setattr(ops, "_HERE", str(tmp_path))
    with pytest.raises(RuntimeError, match="_fp4.so not found"):
        ops._load_fp4()


def test_module_refuses_host_tensors():
    import torch
    from quantised_linear_layers_gb300 import ops
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: ops.fp4_cast(x), lambda: ops.fp4_cast_dual(x), lambda: ops.fp4_tensor_scale(x),
                 lambda: ops.fp4_dequant(x), lambda: ops.gemm_fp4_nt(x, x), lambda: ops.fp4_linear(x, x),
                 lambda: ops.fp4_cast(x, 7), lambda: ops.fp4_dequant(x, torch.float16)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ops._load_fp4().gemm(x)
