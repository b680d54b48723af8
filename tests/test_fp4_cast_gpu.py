"""4-bit casts on the GPU, every code and scale against the numpy definition
(exact: no tolerance)."""
import numpy as np
import pytest
import torch

import fp4_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantised_linear_layers_gb300 import build, ops as o
    build.build()
    o.load_library()
    return o


def acts(m, k, seed, dtype=torch.float32, spread=6):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, k), generator=g) * torch.exp2(torch.randint(-spread, spread + 1, (m, 1), generator=g).float())
    x *= 1 + 15 * (torch.rand((1, k), generator=g) < 0.02)
    return x.to(dtype)


def np64(x):
    return x.detach().float().cpu().numpy().astype(np.float64)


def unpack(a, t=1.0, **kw):
    return ref.unpack(a.q.cpu().numpy(), a.sf.cpu().numpy(), a.fmt, a.rows, a.cols, t, **kw)


def same(got, want):
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    bad = got[ok] != want[ok]
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} differ: {got[ok][bad][:4]} for {want[ok][bad][:4]}"


SHAPES = [(1, 1), (1, 16), (1, 7168), (3, 33), (5, 15), (33, 31), (128, 64), (130, 520), (257, 1031), (31, 513)]


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k", SHAPES)
def test_rows(ops, m, k, dtype, fmt):
    x = acts(m, k, 11 * m + k, dtype).cuda()
    for t in ([None, ops.fp4_tensor_scale(x), torch.tensor([0.37], device="cuda")] if fmt == 0 else [None]):
        tv = 1.0 if t is None else float(t)
        if t is not None and tv != float(np.float32(0.37)):
            assert tv == ref.tensor_scale(np64(x))
        a = ops.fp4_cast(x, fmt, t)
        want = ref.values(np64(x), fmt, tv)
        same(unpack(a, tv), want)
        same(np64(ops.fp4_dequant(a, torch.float32)), want.astype(np.float32).astype(np.float64))
        same(np64(ops.fp4_dequant(a)), np64(torch.from_numpy(want.astype(np.float32)).bfloat16()))


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_strides(ops, dtype, fmt):
    big = acts(200, 700, 5, dtype).cuda()
    views = [big.t(), big[:, 1:334], big[::3, 8:520], big[5:, ::2], big[:, :64].t(), big[7:8].expand(9, 700)]
    for x in views:
        same(unpack(ops.fp4_cast(x, fmt)), ref.values(np64(x), fmt))
        if fmt == 0:
            assert float(ops.fp4_tensor_scale(x)) == ref.tensor_scale(np64(x))


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
def test_halfway_cases_and_scale_edges(ops, fmt):
    """Rows of exact multiples of the group's scale at and beside the midpoints of E2M1, with the largest element at
    and beside the values where the scale changes."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for s in (1.0, 1.125, 1.875, 2.0 ** -9, 3 * 2.0 ** -9, 448.0, 0.0625):
        for lead in (6.0, 6.0 * (1 - 2.0 ** -8), 6.0 * (1 + 2.0 ** -7), 3.0, 4.0):
            row = np.zeros(32)
            row[0] = lead * s
            row[1:8], row[8:15] = mids * s, -mids * s
            row[16] = lead * s
            row[17:24] = mids * s
            rows.append(row)
    x = torch.tensor(np.array(rows), dtype=torch.float32)
    for v in (x, x.bfloat16(), torch.nextafter(x, torch.full_like(x, 1e9)), torch.nextafter(x, torch.zeros_like(x))):
        same(unpack(ops.fp4_cast(v.cuda(), fmt)), ref.values(np64(v), fmt))


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_zero_tiny_huge_and_non_finite(ops, dtype, fmt):
    x = torch.zeros((8, 96), dtype=torch.float32)
    x[1] = 1e-38 * torch.arange(96)
    x[2] = 1e-40
    x[3] = torch.finfo(torch.bfloat16).max * torch.linspace(-1, 1, 96)
    x[4] = 1.0
    x[4, 40] = float("nan")
    x[5] = -2.0
    x[5, 95] = float("inf")
    x[6] = -0.0
    x[7] = 1e30 * torch.linspace(0, 1, 96)
    x = x.to(dtype).cuda()
    a = ops.fp4_cast(x, fmt)
    same(unpack(a), ref.values(np64(x), fmt))
    got = np64(ops.fp4_dequant(a, torch.float32))
    want = ref.values(np64(x), fmt)
    same(got, np.where(np.isnan(want), np.nan, want.astype(np.float32)))
    if fmt == 0:
        assert np.isnan(float(ops.fp4_tensor_scale(x)))
        assert float(ops.fp4_tensor_scale(x[:4])) == ref.tensor_scale(np64(x[:4]))
        assert float(ops.fp4_tensor_scale(torch.zeros((3, 5), device="cuda"))) == 2.0 ** -80


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 130), (127, 33), (128, 128), (129, 257), (300, 520), (64, 1000)])
def test_both_ways(ops, m, k, dtype, fmt):
    x = acts(m, k, m + 7 * k, dtype).cuda()
    t = ops.fp4_tensor_scale(x) if fmt == 0 else None
    tv = 1.0 if t is None else float(t)
    rows, cols = ops.fp4_cast_dual(x, fmt, t)
    same(unpack(rows, tv), ref.values(np64(x), fmt, tv))
    same(unpack(cols, tv), ref.values(np64(x).T, fmt, tv))
    none, cols2 = ops.fp4_cast_dual(x, fmt, t, rows=False)
    assert none is None and torch.equal(cols2.q, cols.q)
    same(unpack(ops.fp4_cast(x.t(), fmt, t), tv), ref.values(np64(x).T, fmt, tv))       # a transposed view
    if dtype == torch.bfloat16 and k > 8:                       # rows that do not start on 16 bytes
        y = x[:, 1:]
        rows, cols = ops.fp4_cast_dual(y, fmt, t)
        same(unpack(rows, tv), ref.values(np64(y), fmt, tv))
        same(unpack(cols, tv), ref.values(np64(y).T, fmt, tv))


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
def test_batch(ops, fmt):
    w = torch.stack([acts(130, 200, s, torch.bfloat16) for s in range(3)]).cuda()
    t = ops.fp4_tensor_scale(w) if fmt == 0 else None
    tv = 1.0 if t is None else float(t)
    a, at = ops.fp4_cast_dual(w, fmt, t)
    b = ops.fp4_cast(w, fmt, t)
    for c, n, k, src in ((a, 130, 200, w), (b, 130, 200, w), (at, 200, 130, w.transpose(1, 2))):
        blocks = -(-n // 128) * -(-k // (4 * ref.GROUP[fmt])) * 512
        for i in range(3):
            got = ref.unpack(c.q.cpu().numpy()[i * n:], c.sf.cpu().numpy()[i * blocks:], fmt, n, k, tv)
            same(got, ref.values(np64(src[i]), fmt, tv))


OFFSETS = [[0, 5], [0, 0, 130, 130, 131, 300], [0, 256, 512, 513], [3, 40, 40, 200], [0, 1, 2, 3, 4, 5, 6, 7, 8, 9]]


@pytest.mark.parametrize("fmt", [0, 1], ids=["nv", "mx"])
@pytest.mark.parametrize("offs", OFFSETS, ids=[str(len(o) - 1) + "_" + str(o[-1]) for o in OFFSETS])
def test_by_expert(ops, offs, fmt):
    m, k = offs[-1] + 3, 200                                     # the last rows belong to nobody
    x = acts(m, k, 3, torch.bfloat16).cuda()
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    where = ref.expert_sf_rows(offs)
    rows_of = np.array(sorted(where))
    for a in (ops.fp4_cast(x, fmt, offsets=off), ops.fp4_cast_dual(x, fmt, offsets=off)[0]):
        got = ref.unpack(a.q.cpu().numpy()[rows_of], a.sf.cpu().numpy(), fmt, len(rows_of), k,
                         sf_rows=[where[r] for r in rows_of])
        same(got, ref.values(np64(x)[rows_of], fmt))
    cols = ops.fp4_cast_dual(x, fmt, offsets=off)[1]
    extent = int(ops.load_library().fp4_column_extent(m, len(offs) - 1))
    got = ref.unpack(cols.q.cpu().numpy(), cols.sf.cpu().numpy(), fmt, k, extent)
    at = 0
    for lo, hi in zip(offs[:-1], offs[1:]):
        n = -(-(hi - lo) // 256) * 256
        want = np.zeros((k, n))
        want[:, :hi - lo] = ref.values(np64(x)[lo:hi].T, fmt) if hi > lo else 0
        same(got[:, at:at + n], want)
        at += n


def test_a_scale_far_too_small(ops):
    """amax / (6 t) beyond fp32 makes its group NaN and no other; beyond the largest group scale it saturates."""
    x = torch.ones((2, 64), device="cuda")
    x[0, 20], x[1, 40] = 1e30, 1e10
    t = torch.tensor([2.0 ** -60], device="cuda")
    got = np64(ops.fp4_dequant(ops.fp4_cast(x, 0, t), torch.float32))
    assert np.isnan(got[0, 16:32]).all() and np.isfinite(got[0, :16]).all() and np.isfinite(got[0, 32:]).all()
    assert got[1, 40] == 6 * 448 * 2.0 ** -60 and got[0, 0] == 6 * 448 * 2.0 ** -60


@pytest.mark.parametrize("m,k", [(1, 1), (3, 33), (130, 520), (1031, 1031), (1024, 2048)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_own_scale(ops, m, k, dtype):
    """A scale made in the call is fp4_tensor_scale's, on both sides of the size where that changes its form, and is the
    casts' own: another call does not change it."""
    x = acts(m, k, m * k, dtype).cuda()
    t = ops.fp4_tensor_scale(x)
    assert float(t) == ref.tensor_scale(np64(x))
    a, (r, c) = ops.fp4_cast(x, 0, ops.FP4_OWN_SCALE), ops.fp4_cast_dual(x, 0, ops.FP4_OWN_SCALE)
    big = ops.fp4_cast_dual(x * 64, 0, ops.FP4_OWN_SCALE)[0]
    for v in (a, r, c):
        assert float(v.scale) == float(t)
    assert float(big.scale) == 64 * float(t)
    want = ops.fp4_dequant(ops.fp4_cast(x, 0, t), torch.float32)
    assert torch.equal(ops.fp4_dequant(a, torch.float32), want) and torch.equal(ops.fp4_dequant(r, torch.float32), want)
    w = torch.stack([x, 2 * x])
    assert float(ops.fp4_cast(w, 0, ops.FP4_OWN_SCALE).scale) == 2 * float(t)


def test_past_31_bits(ops):
    """More than 2^31 elements: the last rows' codes and scales."""
    m, k = 300_001, 7184
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    x[-130:] = acts(130, k, 9, torch.bfloat16).cuda()
    a = ops.fp4_cast(x, 0)
    tail = ops.fp4_dequant(a)[-130:]
    same(np64(tail), ref.values(np64(x[-130:]), 0))
