"""Thin ctypes binding over libqlinear.so (include/qlinear.h).

Argument marshalling only: every step of the cast and the GEMM runs in the
library's CUDA kernels. torch supplies device memory and the current stream.
If the library is missing or cannot be loaded every op raises; there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# QL_LIBRARY selects another build of the library (the bounds-checked
# libqlinear_bounds.so, for instance); the default is the product build.
LIB_PATH = os.environ.get("QL_LIBRARY") or os.path.join(_HERE, "libqlinear.so")

QL_BF16, QL_F32 = 0, 1
SF_FP32, SF_UE8M0, SF_PACKED_UE8M0 = 0, 1, 2
CAST_RECIP_OF_SCALE = 0x100
FP4_NV, FP4_MX = 0, 1
SCORES = {"softmax": 0, "sigmoid": 1}     # of a router, as expert_route takes them
FP4_OWN_SCALE = "own"       # as a tensor scale: fp4_tensor_scale of the tensor itself

_lock = threading.Lock()
_lib = None

_i64, _vp, _int, _sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t

_SIGS = {
    "fp8_cast_per_token": [_vp, _int, _i64, _i64, _i64, _i64, _int, _int, _vp, _i64, _i64, _vp, _i64, _i64, _vp],
    "fp8_cast_per_block": [_vp, _int, _i64, _i64, _i64, _i64, _int, _vp, _i64, _i64, _vp, _i64, _i64, _vp],
    "fp8_cast_per_token_dual": [_vp, _int, _i64, _i64, _i64, _int, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _vp,
                                _i64, _i64, _vp],
    "fp8_cast_per_block_dual": [_vp, _int, _i64, _i64, _i64, _i64, _int, _vp, _i64, _i64, _vp, _i64, _i64,
                                _vp, _i64, _i64, _vp],
    "gemm_fp8_nt_bf16": [_vp, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _int, _vp, _i64,
                         _i64, _i64, _i64, _vp, _sz, _vp],
    "gemm_fp8_wgrad_fp32": [_vp, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _int, _vp, _i64,
                            _i64, _i64, _i64, _int, _vp, _sz, _vp],
    "m_grouped_gemm_fp8_nt_bf16_contiguous": [_vp, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _i64,
                                              _int, _vp, _i64, _vp, _int, _i64, _i64, _i64, _vp],
    "ql_get_m_alignment_for_contiguous_layout": [],
    "gemm_fp8_nt_fp8out": [_vp, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _int, _vp, _i64, _vp, _i64,
                           _i64, _int, _int, _i64, _i64, _i64, _vp],
    "gemm_fp8_wgrad_fp32_mn": [_vp, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _int, _vp, _i64,
                               _i64, _i64, _i64, _int, _vp],
    "gemm_fp8_nn_bf16": [_vp, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _int, _vp, _i64,
                         _i64, _i64, _i64, _vp],
    "fp4_scale_bytes": [_i64, _i64, _int, _int],
    "fp4_row_stride": [_i64],
    "fp4_column_extent": [_i64, _int],
    "fp4_tensor_scale": [_vp, _int, _i64, _i64, _i64, _i64, _vp, _vp],
    "fp4_cast": [_vp, _int, _i64, _i64, _i64, _i64, _i64, _i64, _int, _vp, _int, _vp, _i64, _vp, _vp, _int, _vp],
    "fp4_cast_dual": [_vp, _int, _i64, _i64, _i64, _i64, _i64, _int, _vp, _int, _vp, _i64, _vp, _vp, _i64, _vp, _vp,
                      _int, _vp],
    "fp4_dequant": [_vp, _i64, _vp, _int, _vp, _i64, _i64, _vp, _int, _i64, _vp],
    "gemm_fp4_nt": [_vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _int, _vp, _int, _i64, _i64, _i64, _i64, _int, _vp],
    "gemm_fp4_nt_ragged": [_vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _int, _vp, _int, _i64, _vp, _int, _i64, _i64,
                           _i64, _vp],
    "fp4_linear_workspace_size": [_i64, _i64, _int, _int],
    "fp4_linear": [_vp, _int, _i64, _vp, _int, _vp, _i64, _vp, _vp, _int, _vp, _i64, _vp, _int, _i64, _i64, _i64, _vp, _sz, _vp],
    "gemm_fp4_wgrad_ragged": [_vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _int, _vp, _i64, _vp, _int, _i64, _i64, _i64,
                              _int, _vp],
    "layer_norm": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _int, ctypes.c_float, _vp, _int, _i64, _vp, _vp, _vp],
    "layer_norm_backward_workspace_size": [_i64, _i64],
    "layer_norm_backward": [_vp, _int, _i64, _vp, _int, _i64, _vp, _vp, _vp, _int, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _sz,
                            _vp],
    "expert_route": [_vp, _int, _i64, _int, _i64, _vp, _int, _int, _int, _int, _int, _int, ctypes.c_float, _vp, _vp, _vp],
    "expert_route_backward": [_vp, _vp, _int, _i64, _int, _i64, _vp, _int, _int, _int, ctypes.c_float, _vp, _i64, _vp],
    "expert_plan_workspace_size": [_i64, _int],
    "expert_plan": [_vp, _i64, _int, _vp, _vp, _vp, _sz, _vp],
    "expert_dispatch": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _int, _int, _vp, _i64, _vp],
    "expert_combine": [_vp, _int, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, _i64, _vp],
    "expert_combine_backward": [_vp, _int, _i64, _vp, _i64, _vp, _vp, _int, _vp, _i64, _i64, _int, _vp, _i64, _vp, _vp],
    "ql_cast_gemm_host_workspace_size": [_i64, _i64, _i64, _int],
    "ql_cast_gemm_host": [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _int, _vp, _i64, _i64, _i64, _i64, _i64,
                          _vp, _sz, _vp],
    "ql_cast_gemm_host_noalloc": [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _int, _vp, _i64, _i64, _i64, _i64, _i64,
                                  _vp],
    "ql_gemm_workspace_size": [_i64, _i64, _i64],
    "ql_set_num_sms": [_int],
    "ql_get_num_sms": [],
    "ql_binary_version": [],
    "ql_set_wait_limit_ms": [_int],
    "ql_set_gemm_block_n": [_int],
    "ql_set_gemm_path": [_int],
    "ql_test_stall_gemm_producer": [_int],
    "ql_device_status": [_vp],
    "ql_device_status_detail": [_vp, _vp, _vp],
    "ql_bounds_checked": [],
    "ql_status_string": [_int],
}


class QLError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {msg}")
        self.status = status


def load_library(path: str = LIB_PATH):
    """Load libqlinear.so (raises if it is missing: no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"libqlinear.so not found at {path}; run quantised_linear_layers_gb300.build.build()")
            lib = ctypes.CDLL(path)
            for name, args in _SIGS.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = _int
            lib.ql_status_string.restype = ctypes.c_char_p
            lib.ql_gemm_workspace_size.restype = _sz
            lib.ql_cast_gemm_host_workspace_size.restype = _sz
            lib.fp4_linear_workspace_size.restype = _sz
            lib.layer_norm_backward_workspace_size.restype = _sz
            lib.expert_plan_workspace_size.restype = _sz
            lib.fp4_scale_bytes.restype = _i64
            lib.fp4_row_stride.restype = _i64
            lib.fp4_column_extent.restype = _i64
            _lib = lib
    return _lib


def _check(fn: str, status: int) -> None:
    if status != 0:
        msg = load_library().ql_status_string(status).decode()
        raise QLError(fn, status, msg)


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _dtype_code(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return QL_BF16
    if x.dtype == torch.float32:
        return QL_F32
    raise TypeError(f"input must be bfloat16 or float32, got {x.dtype}")


def _bytes8(t: torch.Tensor) -> torch.Tensor:
    if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError(f"expected an E4M3 (float8_e4m3fn or uint8) tensor, got {t.dtype}")
    return t


def _ceil(a: int, b: int) -> int:
    return -(-a // b)


def sf_shape(n: int, gran_k: int, fmt: int) -> int:
    """Number of scale columns per row: groups, or int32 words for packed UE8M0."""
    g = _ceil(n, gran_k)
    return _ceil(g, 4) if (fmt & 0xFF) == SF_PACKED_UE8M0 else g


def empty_sf(m: int, cols: int, fmt: int, device, mn_major: bool = False) -> torch.Tensor:
    """Scale tensor [m, cols]; mn_major gives the M-major, TMA-aligned layout
    (stride (1, align(m, 4)))."""
    dt = torch.int32 if (fmt & 0xFF) == SF_PACKED_UE8M0 else torch.float32
    if not mn_major:
        return torch.empty((m, cols), dtype=dt, device=device)
    ld = _ceil(max(m, 1), 4) * 4
    return torch.empty((cols, ld), dtype=dt, device=device).t()[:m]


def fp8_cast_per_token(x: torch.Tensor, gran_k: int = 128, fmt: int = SF_FP32, recip: bool = False,
                       out: torch.Tensor | None = None, out_sf: torch.Tensor | None = None,
                       sf_mn_major: bool = False):
    """Per-token FP8 cast of a 2-D bf16/fp32 tensor (any strides).

    Returns (data float8_e4m3fn [m, n], scales). ``out`` / ``out_sf`` may be
    views of larger buffers; only their elements are written."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    m, n = x.shape
    if out is None:
        out = torch.empty((m, n), dtype=torch.float8_e4m3fn, device=x.device)
    if out_sf is None:
        out_sf = empty_sf(m, sf_shape(n, gran_k, fmt), fmt, x.device, sf_mn_major)
    _bytes8(out)
    code = fmt | (CAST_RECIP_OF_SCALE if recip else 0)
    st = load_library().fp8_cast_per_token(
        x.data_ptr(), _dtype_code(x), m, n, x.stride(0), x.stride(1), gran_k, code,
        out.data_ptr(), out.stride(0), out.stride(1), out_sf.data_ptr(), out_sf.stride(0), out_sf.stride(1),
        _stream(x))
    _check("fp8_cast_per_token", st)
    return out, out_sf


def fp8_cast_per_block(x: torch.Tensor, fmt: int = SF_FP32, recip: bool = False,
                       out: torch.Tensor | None = None, out_sf: torch.Tensor | None = None):
    """128x128 block FP8 cast. Returns (data [m, n], scales fp32 [ceil(m/128), ceil(n/128)],
    or int32 words [ceil(m/128), ceil(ceil(n/128)/4)] packed along the column blocks
    for SF_PACKED_UE8M0). ``out`` / ``out_sf`` may be transposed views (e.g.
    ``wt.t()``) to write W^T's cast."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    m, n = x.shape
    if out is None:
        out = torch.empty((m, n), dtype=torch.float8_e4m3fn, device=x.device)
    if out_sf is None:
        cols = _ceil(n, 128)
        if fmt == SF_PACKED_UE8M0:
            out_sf = torch.empty((_ceil(m, 128), _ceil(cols, 4)), dtype=torch.int32, device=x.device)
        else:
            out_sf = torch.empty((_ceil(m, 128), cols), dtype=torch.float32, device=x.device)
    _bytes8(out)
    code = fmt | (CAST_RECIP_OF_SCALE if recip else 0)
    st = load_library().fp8_cast_per_block(
        x.data_ptr(), _dtype_code(x), m, n, x.stride(0), x.stride(1), code,
        out.data_ptr(), out.stride(0), out.stride(1), out_sf.data_ptr(), out_sf.stride(0), out_sf.stride(1),
        _stream(x))
    _check("fp8_cast_per_block", st)
    return out, out_sf


def fp8_cast_per_token_dual(x: torch.Tensor, fmt: int = SF_FP32, recip: bool = False):
    """Both per-token casts of x [T, C] from one read (1x128 groups): returns
    (q_rows [T, C], s_rows [T, ceil(C/128)] M-major) = fp8_cast_per_token(x)
    and (q_cols [T, C], s_cols [C, ceil(T/128)] M-major), the cast of x^T kept
    in x's layout (the MN-major weight-gradient operand). E4M3 rows start on
    16-byte boundaries; their padding is never written or read."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with contiguous rows")
    t, c = x.shape
    ld = _ceil(max(c, 1), 16) * 16
    q_rows = torch.empty((t, ld), dtype=torch.float8_e4m3fn, device=x.device)[:, :c]
    q_cols = torch.empty((t, ld), dtype=torch.float8_e4m3fn, device=x.device)[:, :c]
    s_rows = empty_sf(t, sf_shape(c, 128, fmt), fmt, x.device, mn_major=True)
    s_cols = empty_sf(c, sf_shape(t, 128, fmt), fmt, x.device, mn_major=True)
    code = fmt | (CAST_RECIP_OF_SCALE if recip else 0)
    st = load_library().fp8_cast_per_token_dual(
        x.data_ptr(), _dtype_code(x), t, c, x.stride(0), code,
        q_rows.data_ptr(), q_rows.stride(0), s_rows.data_ptr(), s_rows.stride(0), s_rows.stride(1),
        q_cols.data_ptr(), q_cols.stride(0), s_cols.data_ptr(), s_cols.stride(0), s_cols.stride(1), _stream(x))
    _check("fp8_cast_per_token_dual", st)
    return q_rows, s_rows, q_cols, s_cols


def fp8_cast_per_block_dual(x: torch.Tensor, fmt: int = SF_FP32, recip: bool = False):
    """fp8_cast_per_block plus, from the same pass, the scale grid of the
    transposed cast (equal to fp8_cast_per_block(x.t())'s scales): returns
    (data [m, n], scales of x, scales of x^T). With the data read MN-major,
    the second grid is the data-gradient operand of gemm_fp8_nn_bf16. The
    data's rows start on 16-byte boundaries (the GEMMs' operand rows must),
    whatever n is; the padding bytes are never written or read."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    m, n = x.shape
    ld = _ceil(max(n, 1), 16) * 16
    out = torch.empty((m, ld), dtype=torch.float8_e4m3fn, device=x.device)[:, :n]
    rb, cb = _ceil(m, 128), _ceil(n, 128)
    if fmt == SF_PACKED_UE8M0:
        out_sf = torch.empty((rb, _ceil(cb, 4)), dtype=torch.int32, device=x.device)
        out_sf_t = torch.empty((cb, _ceil(rb, 4)), dtype=torch.int32, device=x.device)
    else:
        out_sf = torch.empty((rb, cb), dtype=torch.float32, device=x.device)
        out_sf_t = torch.empty((cb, rb), dtype=torch.float32, device=x.device)
    code = fmt | (CAST_RECIP_OF_SCALE if recip else 0)
    st = load_library().fp8_cast_per_block_dual(
        x.data_ptr(), _dtype_code(x), m, n, x.stride(0), x.stride(1), code,
        out.data_ptr(), out.stride(0), out.stride(1), out_sf.data_ptr(), out_sf.stride(0), out_sf.stride(1),
        out_sf_t.data_ptr(), out_sf_t.stride(0), out_sf_t.stride(1), _stream(x))
    _check("fp8_cast_per_block_dual", st)
    return out, out_sf, out_sf_t


def _gemm_args(a, sfa, b, sfb):
    _bytes8(a)
    _bytes8(b)
    if a.dim() != 2 or b.dim() != 2 or a.stride(1) != 1 or b.stride(1) != 1:
        raise ValueError("a and b must be 2-D with contiguous K")
    if a.shape[1] != b.shape[1]:
        raise ValueError("a and b must share K")
    return a.shape[0], b.shape[0], a.shape[1]


def gemm_fp8_nt_bf16(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor,
                     fmt: int = SF_FP32, out: torch.Tensor | None = None) -> torch.Tensor:
    """D = A B^T, bf16 [m, n]: A [m, k] with 1x128 scales sfa [m, ceil(k/128)],
    B [n, k] with 128x128 scales sfb [ceil(n/128), ceil(k/128)] (packed UE8M0:
    int32 words along K)."""
    m, n, k = _gemm_args(a, sfa, b, sfb)
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    if out.dtype != torch.bfloat16 or out.stride(1) != 1:
        raise ValueError("out must be bf16 with contiguous rows")
    st = load_library().gemm_fp8_nt_bf16(
        a.data_ptr(), a.stride(0), sfa.data_ptr(), sfa.stride(0), sfa.stride(1),
        b.data_ptr(), b.stride(0), sfb.data_ptr(), sfb.stride(0), sfb.stride(1),
        fmt, out.data_ptr(), out.stride(0), m, n, k, None, 0, _stream(a))
    _check("gemm_fp8_nt_bf16", st)
    return out


def gemm_fp8_nt_fp8out(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor,
                       fmt: int = SF_FP32, gran_k: int = 128, out_fmt: int = SF_FP32, recip: bool = False,
                       out: torch.Tensor | None = None, out_sf: torch.Tensor | None = None,
                       sf_mn_major: bool = False):
    """D = A B^T cast per token inside the GEMM: returns (E4M3 [m, n], scales),
    equal to fp8_cast_per_token(gemm_fp8_nt_bf16(...), gran_k, out_fmt)."""
    m, n, k = _gemm_args(a, sfa, b, sfb)
    if out is None:
        out = torch.empty((m, n), dtype=torch.float8_e4m3fn, device=a.device)
    _bytes8(out)
    if out.stride(1) != 1:
        raise ValueError("out must have contiguous rows")
    if out_sf is None:
        out_sf = empty_sf(m, sf_shape(n, gran_k, out_fmt), out_fmt, a.device, mn_major=sf_mn_major)
    code = out_fmt | (CAST_RECIP_OF_SCALE if recip else 0)
    st = load_library().gemm_fp8_nt_fp8out(
        a.data_ptr(), a.stride(0), sfa.data_ptr(), sfa.stride(0), sfa.stride(1),
        b.data_ptr(), b.stride(0), sfb.data_ptr(), sfb.stride(0), sfb.stride(1),
        fmt, out.data_ptr(), out.stride(0), out_sf.data_ptr(), out_sf.stride(0), out_sf.stride(1),
        gran_k, code, m, n, k, _stream(a))
    _check("gemm_fp8_nt_fp8out", st)
    return out, out_sf


def gemm_fp8_wgrad_fp32(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor,
                        out: torch.Tensor | None = None, accumulate: bool = False,
                        fmt: int = SF_FP32) -> torch.Tensor:
    """D (+)= A B^T, fp32 [m, n]: both operands with 1x128 per-row scales along K."""
    m, n, k = _gemm_args(a, sfa, b, sfb)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an existing out")
        out = torch.empty((m, n), dtype=torch.float32, device=a.device)
    if out.dtype != torch.float32 or out.stride(1) != 1:
        raise ValueError("out must be fp32 with contiguous rows")
    st = load_library().gemm_fp8_wgrad_fp32(
        a.data_ptr(), a.stride(0), sfa.data_ptr(), sfa.stride(0), sfa.stride(1),
        b.data_ptr(), b.stride(0), sfb.data_ptr(), sfb.stride(0), sfb.stride(1),
        fmt, out.data_ptr(), out.stride(0), m, n, k, int(bool(accumulate)), None, 0, _stream(a))
    _check("gemm_fp8_wgrad_fp32", st)
    return out


def m_grouped_gemm_fp8_nt_bf16_contiguous(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor,
                                          sfb: torch.Tensor, m_indices: torch.Tensor, fmt: int = SF_FP32,
                                          out: torch.Tensor | None = None) -> torch.Tensor:
    """Grouped D = A B_e^T over the contiguous layout: A [m, k] (m a multiple of
    128) with 1x128 scales, B [G, n, k] with scales sfb [G, ceil(n/128),
    ceil(k/128)], m_indices int32 [m] (expert per row, -1 for padding rows,
    which are left unwritten in ``out``)."""
    _bytes8(a)
    _bytes8(b)
    if a.dim() != 2 or b.dim() != 3 or a.stride(1) != 1 or b.stride(2) != 1:
        raise ValueError("a must be [m, k] and b [G, n, k], both with contiguous K")
    if b.stride(0) != b.shape[1] * b.stride(1):
        raise ValueError("b's experts must be stacked without gaps (stride(0) == n * stride(1))")
    if a.shape[1] != b.shape[2] or sfb.dim() != 3 or sfb.shape[0] != b.shape[0]:
        raise ValueError("shapes of a, b and sfb do not agree")
    if m_indices.dtype != torch.int32 or m_indices.dim() != 1 or m_indices.shape[0] != a.shape[0] \
            or not m_indices.is_contiguous() or m_indices.device != a.device:
        raise ValueError("m_indices must be a contiguous int32 [m] tensor on a's device")
    m, k = a.shape
    G, n = b.shape[0], b.shape[1]
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    if out.dtype != torch.bfloat16 or out.stride(1) != 1:
        raise ValueError("out must be bf16 with contiguous rows")
    st = load_library().m_grouped_gemm_fp8_nt_bf16_contiguous(
        a.data_ptr(), a.stride(0), sfa.data_ptr(), sfa.stride(0), sfa.stride(1),
        b.data_ptr(), b.stride(1), sfb.data_ptr(), sfb.stride(0), sfb.stride(1), sfb.stride(2),
        fmt, out.data_ptr(), out.stride(0), m_indices.data_ptr(), G, m, n, k, _stream(a))
    _check("m_grouped_gemm_fp8_nt_bf16_contiguous", st)
    return out


def get_m_alignment_for_contiguous_layout() -> int:
    return int(load_library().ql_get_m_alignment_for_contiguous_layout())


def gemm_fp8_wgrad_fp32_mn(a_t: torch.Tensor, sfa: torch.Tensor, b_t: torch.Tensor, sfb: torch.Tensor,
                           out: torch.Tensor | None = None, accumulate: bool = False,
                           fmt: int = SF_FP32) -> torch.Tensor:
    """D [m, n] (+)= A B^T, fp32, with both operands given K-outer: a_t [k, m]
    and b_t [k, n] (contiguous rows); sfa [m, ceil(k/128)], sfb [n, ceil(k/128)]."""
    _bytes8(a_t)
    _bytes8(b_t)
    if a_t.dim() != 2 or b_t.dim() != 2 or a_t.stride(1) != 1 or b_t.stride(1) != 1:
        raise ValueError("a_t and b_t must be 2-D with contiguous rows")
    if a_t.shape[0] != b_t.shape[0]:
        raise ValueError("a_t and b_t must share K (their first dimension)")
    k, m = a_t.shape
    n = b_t.shape[1]
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an existing out")
        out = torch.empty((m, n), dtype=torch.float32, device=a_t.device)
    if out.dtype != torch.float32 or out.stride(1) != 1:
        raise ValueError("out must be fp32 with contiguous rows")
    st = load_library().gemm_fp8_wgrad_fp32_mn(
        a_t.data_ptr(), a_t.stride(0), sfa.data_ptr(), sfa.stride(0), sfa.stride(1),
        b_t.data_ptr(), b_t.stride(0), sfb.data_ptr(), sfb.stride(0), sfb.stride(1),
        fmt, out.data_ptr(), out.stride(0), m, n, k, int(bool(accumulate)), _stream(a_t))
    _check("gemm_fp8_wgrad_fp32_mn", st)
    return out


def gemm_fp8_nn_bf16(a: torch.Tensor, sfa: torch.Tensor, b_kn: torch.Tensor, sfb: torch.Tensor,
                     fmt: int = SF_FP32, out: torch.Tensor | None = None) -> torch.Tensor:
    """D = A B, bf16 [m, n]: A [m, k] with 1x128 scales, B given as [k, n]
    (contiguous rows) with 128x128 scales sfb [ceil(n/128), ceil(k/128)] (any strides)."""
    _bytes8(a)
    _bytes8(b_kn)
    if a.dim() != 2 or b_kn.dim() != 2 or a.stride(1) != 1 or b_kn.stride(1) != 1:
        raise ValueError("a and b_kn must be 2-D with contiguous rows")
    if a.shape[1] != b_kn.shape[0]:
        raise ValueError("a [m, k] and b_kn [k, n] must share K")
    m, k = a.shape
    n = b_kn.shape[1]
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    if out.dtype != torch.bfloat16 or out.stride(1) != 1:
        raise ValueError("out must be bf16 with contiguous rows")
    st = load_library().gemm_fp8_nn_bf16(
        a.data_ptr(), a.stride(0), sfa.data_ptr(), sfa.stride(0), sfa.stride(1),
        b_kn.data_ptr(), b_kn.stride(0), sfb.data_ptr(), sfb.stride(0), sfb.stride(1),
        fmt, out.data_ptr(), out.stride(0), m, n, k, _stream(a))
    _check("gemm_fp8_nn_bf16", st)
    return out


def cast_gemm_host_workspace_size(n: int, k: int, chunk_rows: int, fmt: int) -> int:
    return int(load_library().ql_cast_gemm_host_workspace_size(n, k, chunk_rows, fmt))


def cast_gemm_host(x_host: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor, fmt: int, out_host: torch.Tensor,
                   chunk_rows: int, workspace: torch.Tensor) -> torch.Tensor:
    """out_host [m, n] = bf16(cast_per_token(x_host) @ b^T) with x_host / out_host
    bf16 tensors in host memory (pinned for overlap), b / sfb on the device and
    a device workspace of cast_gemm_host_workspace_size bytes; copies and
    kernels of successive row chunks overlap. Stream-ordered on the current stream."""
    if x_host.device.type != "cpu" or out_host.device.type != "cpu":
        raise ValueError("x_host and out_host must be host tensors")
    if x_host.dtype != torch.bfloat16 or out_host.dtype != torch.bfloat16:
        raise ValueError("x_host and out_host must be bf16")
    if x_host.stride(1) != 1 or out_host.stride(1) != 1 or b.stride(1) != 1:
        raise ValueError("rows must be contiguous")
    _bytes8(b)
    m, k = x_host.shape
    n = b.shape[0]
    if b.shape[1] != k or tuple(out_host.shape) != (m, n):
        raise ValueError("shapes of x_host, b and out_host do not agree")
    if not workspace.is_cuda or workspace.device != b.device:
        raise ValueError("workspace must be device memory on b's device")
    st = load_library().ql_cast_gemm_host(
        x_host.data_ptr(), x_host.stride(0), b.data_ptr(), b.stride(0), sfb.data_ptr(), sfb.stride(0), sfb.stride(1),
        fmt, out_host.data_ptr(), out_host.stride(0), m, n, k, chunk_rows,
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(b))
    _check("ql_cast_gemm_host", st)
    return out_host


# ---------------------------------------------------------------------------
# Microscaled 4-bit floating point
# ---------------------------------------------------------------------------
class FP4Tensor:
    """A matrix (or a batch of them) in 4 bits, as a cast left it: codes and scale
    blocks in one buffer ``buf`` (``q``: uint8, batch * rows rows of stride ld; ``sf``), the
    tensor's scale ``scale`` (fp32 [1], or None for 1), its format and its sizes;
    ``cols`` is the reduction axis. ``offsets`` are the row ranges of the experts
    it was cast by (``by_cols``: its columns are the experts' rows, each from a
    multiple of 256 on). The layouts are in include/qlinear.h."""

    __slots__ = ("buf", "ld", "fmt", "batch", "rows", "cols", "offsets", "by_cols", "device_index", "q_ptr", "sf_ptr",
                 "scale_ptr", "_scale")

    def __init__(self, buf, ld, scale, fmt, batch, rows, cols, offsets=None, by_cols=False):
        # scale: a tensor, None, FP4_OWN_SCALE (the last 16 bytes of buf) or the FP4Tensor that has it
        self.ld, self.fmt, self.batch, self.rows, self.cols, self.by_cols = ld, fmt, batch, rows, cols, by_cols
        self.buf, self.offsets, self.device_index = buf, offsets, buf.get_device()
        self.q_ptr = q = buf.data_ptr()
        self.sf_ptr = q + batch * rows * ld
        self._scale = scale
        if scale is None:
            self.scale_ptr = None
        elif scale is FP4_OWN_SCALE:
            self.scale_ptr = q + buf.numel() - 16
        else:
            self.scale_ptr = scale.scale_ptr if type(scale) is FP4Tensor else scale.data_ptr()

    def __reduce__(self):        # a copy has addresses of its own
        return _fp4_tensor, (self.buf, self.ld, self._scale, self.fmt, self.batch, self.rows, self.cols, self.offsets,
                             self.by_cols)

    @property
    def scale(self) -> torch.Tensor | None:
        s = self._scale
        if s is FP4_OWN_SCALE:
            return self.buf[-16:-12].view(torch.float32)
        return s.scale if type(s) is FP4Tensor else s

    @property
    def q(self) -> torch.Tensor:
        n = self.batch * self.rows
        return self.buf[:n * self.ld].view(n, self.ld)[:, :self.ld if self.by_cols else (self.cols + 1) // 2]

    @property
    def sf(self) -> torch.Tensor:
        return self.buf[self.batch * self.rows * self.ld:]


def _fp4_tensor(buf, ld, scale, *rest):
    return FP4Tensor(buf, ld, FP4_OWN_SCALE if isinstance(scale, str) else scale, *rest)


_fp4 = None
_FP4_ENTRIES = ("fp4_tensor_scale", "fp4_cast", "fp4_cast_dual", "fp4_dequant", "fp4_linear", "fp4_linear_workspace_size",
                "fp4_row_stride", "gemm_fp4_nt", "gemm_fp4_nt_ragged", "gemm_fp4_wgrad_ragged")
_LAYER_ENTRIES = ("layer_norm", "layer_norm_backward", "layer_norm_backward_workspace_size", "expert_route",
                  "expert_route_backward", "expert_plan", "expert_plan_workspace_size", "expert_dispatch", "expert_combine",
                  "expert_combine_backward")


class ExpertPlan:
    """Where the rows of a batch go among its experts (``expert_plan``): ``offsets`` int32
    [experts + 1], as the 4-bit experts take them, and ``rows`` int32 [tokens, k], the
    place of each slot in the order by expert (-1: none)."""

    __slots__ = ("offsets", "rows")

    def __init__(self, offsets: torch.Tensor, rows: torch.Tensor):
        self.offsets, self.rows = offsets, rows


def _load_fp4():
    """The module of the calls over torch tensors (_fp4.so), bound to the loaded library's entry
    points (raises if either is missing: no fallback)."""
    global _fp4
    lib = load_library()
    with _lock:
        if _fp4 is None:
            import importlib.util
            path = os.path.join(_HERE, "_fp4.so")
            if not os.path.exists(path):
                raise RuntimeError(f"_fp4.so not found at {path}; run quantised_linear_layers_gb300.build.build()")
            spec = importlib.util.spec_from_file_location("quantised_linear_layers_gb300._fp4", path)
            mod = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(mod)
            mod.bind(tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _FP4_ENTRIES + _LAYER_ENTRIES),
                     FP4Tensor, FP4_OWN_SCALE, ExpertPlan, _check)
            _fp4 = mod
    return _fp4


def _hold_in_graph(obj, event: torch.cuda.Event) -> None:
    """Keeps obj alive for as long as the graph being captured, or an executable of it,
    and waits for the event behind the work that made it."""
    (_fp4 or _load_fp4()).hold_in_graph(obj, event.cuda_event)


def _drop_held() -> None:
    """Lets go of what only graphs held that are gone."""
    if _fp4 is not None:
        _fp4.drop_held()


def _is_bf16(dtype: torch.dtype) -> bool:
    if dtype is torch.bfloat16:
        return True
    if dtype is torch.float32:
        return False
    raise ValueError("dtype must be bfloat16 or float32")


def fp4_tensor_scale(x: torch.Tensor) -> torch.Tensor:
    """The FP4_NV scale of a tensor (any 2-D or 3-D strides, fp32 [1]): the least
    power of two t with max|x| <= 2688 t, at least 2^-80; a power of two leaves
    every group's scale s * t exact. NaN if x has an infinity or a NaN."""
    return (_fp4 or _load_fp4()).tensor_scale(x)


def fp4_cast(x: torch.Tensor, fmt: int = FP4_NV, tensor_scale: torch.Tensor | None = None,
             offsets: torch.Tensor | None = None) -> FP4Tensor:
    """Casts the rows of x [m, k] or [batch, m, k] (bf16 or fp32, any strides) to
    4 bits. ``tensor_scale`` (FP4_NV): one fp32 value on the device, None for 1,
    or FP4_OWN_SCALE for ``fp4_tensor_scale(x)``, made in the call (with offsets, of
    the experts' rows alone); FP4_MX has none and takes no notice of it. ``offsets`` (int32 [experts + 1]): x's rows are sorted by expert and the cast is the
    operand of ``gemm_fp4_nt_ragged``; rows of no expert are left out."""
    return (_fp4 or _load_fp4()).cast(x, fmt, tensor_scale, offsets)


def fp4_cast_dual(x: torch.Tensor, fmt: int = FP4_NV, tensor_scale: torch.Tensor | None = None,
                  offsets: torch.Tensor | None = None, rows: bool = True):
    """Casts x [m, k] or [batch, m, k] (contiguous rows) along its rows and along
    its columns from one read: (cast of x, cast of x^T). The second is the
    operand of products that sum over x's rows; with ``offsets`` each expert's rows
    are columns of their own there (``gemm_fp4_wgrad_ragged``). ``rows=False``
    leaves the first out (None). ``tensor_scale`` as in ``fp4_cast``."""
    return (_fp4 or _load_fp4()).cast_dual(x, fmt, tensor_scale, offsets, rows)


def fp4_dequant(a: FP4Tensor, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values [rows, cols] that a cast stands for (bf16 or fp32)."""
    return (_fp4 or _load_fp4()).dequant(a, out, _is_bf16(dtype))


def gemm_fp4_nt(x: FP4Tensor, w: FP4Tensor, out: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16,
                accumulate: bool = False) -> torch.Tensor:
    """D [m, n] (+)= X W^T of two row-wise casts of one format: X [m, k], W [n, k];
    D bf16 or fp32 (accumulate: fp32)."""
    return (_fp4 or _load_fp4()).gemm(x, w, out, _is_bf16(dtype), accumulate)


def gemm_fp4_nt_ragged(x: FP4Tensor, w: FP4Tensor, out: torch.Tensor | None = None,
                       dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Experts' products: rows offsets[e] .. offsets[e+1] of D [m, n] are those
    rows of X [m, k] times W[e]^T; X cast with the offsets, W [experts, n, k] cast
    as a batch. Rows of no expert are zero, or left unwritten in a given ``out``."""
    return (_fp4 or _load_fp4()).ragged(x, w, out, _is_bf16(dtype))


def gemm_fp4_wgrad_ragged(y: FP4Tensor, x: FP4Tensor, out: torch.Tensor | None = None,
                          accumulate: bool = False) -> torch.Tensor:
    """Experts' weight gradients D [experts, m, n] (+)= Y_e^T X_e, fp32, from the
    column-wise casts of Y [tokens, m] and X [tokens, n] by the same offsets. An
    expert without rows gets zeros."""
    return (_fp4 or _load_fp4()).wgrad(y, x, out, accumulate)


def fp4_linear(x: torch.Tensor, w: FP4Tensor, x_scale: torch.Tensor | None = None,
               offsets: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """The forward call, cast and product in one: D [m, n] bf16 = X W^T of
    x [m, k] (bf16 or fp32) and a cast W [n, k]; with ``offsets`` (int32
    [experts + 1]) by expert, W [experts, n, k]; rows of no expert are zero, or left
    unwritten in a given ``out``. Equal to ``fp4_cast`` followed by
    ``gemm_fp4_nt`` or ``gemm_fp4_nt_ragged``; up to 8 rows (16 with experts) take one launch.
    ``x_scale`` as ``fp4_cast``'s tensor_scale."""
    return (_fp4 or _load_fp4()).linear(x, w, x_scale, offsets, out)


def fp4_linear_saving(x: torch.Tensor, w: FP4Tensor, x_scale: torch.Tensor | None = None,
                      offsets: torch.Tensor | None = None):
    """``fp4_linear`` that also casts x along its columns from the same read:
    (D, cast of x^T), the second for ``fp4_linear_backward``."""
    return (_fp4 or _load_fp4()).linear_saving(x, w, x_scale, offsets)


def fp4_linear_backward(dy: torch.Tensor, wt: FP4Tensor | None, x_cols: FP4Tensor, dy_scale: torch.Tensor | None = None,
                        offsets: torch.Tensor | None = None, dw_out: torch.Tensor | None = None,
                        accumulate: bool = False):
    """(dX, dW) of ``fp4_linear_saving``'s product: dX [m, k] bf16 = dY W from the
    cast ``wt`` of W^T (None: no dX), dW [n, k] or [experts, n, k] fp32 (+)= dY^T X,
    with dY cast both ways from one read."""
    return (_fp4 or _load_fp4()).linear_backward(dy, wt, x_cols, dy_scale, offsets, dw_out, accumulate)


# ---------------------------------------------------------------------------
# Around the experts' products: layer norm, routing and the exchange of rows
# ---------------------------------------------------------------------------
def _refuse_forward_mode(what: str, *tensors: torch.Tensor | None) -> None:
    """The calls go past autograd, which would refuse (the level by itself first: it is quick)."""
    from torch.autograd import forward_ad
    if forward_ad._current_level >= 0 and any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError(f"{what} has no forward-mode derivatives")


def _type_code(dtype: torch.dtype | None) -> int:
    if dtype is None:
        return 2
    return QL_BF16 if _is_bf16(dtype) else QL_F32


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, eps: float = 1e-5,
               out: torch.Tensor | None = None, dtype: torch.dtype | None = None) -> torch.Tensor:
    """(x - mean) / sqrt(var + eps) * weight + bias over the rows of x [m, n] (bf16 or
    fp32), in fp32 and rounded once to ``dtype`` (default: out's or x's). weight and
    bias [n], bf16 or fp32, each may be None. out may be x, but not overlap it otherwise."""
    return (_fp4 or _load_fp4()).layer_norm(x, weight, bias, eps, out, _type_code(dtype), False)


def layer_norm_saving(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                      eps: float = 1e-5, out: torch.Tensor | None = None, dtype: torch.dtype | None = None):
    """``layer_norm`` that keeps its rows' statistics: (y, stats), stats fp32 [2, m]
    (mean, 1 / sqrt(var + eps)) for ``layer_norm_backward``."""
    return (_fp4 or _load_fp4()).layer_norm(x, weight, bias, eps, out, _type_code(dtype), True)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, stats: torch.Tensor, weight: torch.Tensor | None = None,
                        sums: bool | None = None):
    """(dx, dweight, dbias) of ``layer_norm_saving``: dx of x's type, dweight and dbias
    fp32 [n], which are None without ``sums`` (default: with a weight)."""
    return (_fp4 or _load_fp4()).layer_norm_backward(dy, x, stats, weight, weight is not None if sums is None else sums)


def _score_code(score: str) -> int:
    if score not in SCORES:
        raise ValueError(f"score must be one of {', '.join(SCORES)}")
    return SCORES[score]


def route(logits: torch.Tensor, k: int, bias: torch.Tensor | None = None, score: str = "softmax", groups: int = 1,
          kept: int = 1, group_best: int = 1, renormalise: bool = True, scale: float = 1.0):
    """Which k experts each token goes to: (weights fp32 [tokens, k], experts int32
    [tokens, k]) from logits [tokens, experts] (bf16 or fp32).

    Scores s are the ``score`` ("softmax" or "sigmoid") of a token's logits. Experts are
    chosen by s + bias (fp32 [experts], for balance) from the ``kept`` best of ``groups``
    equal runs of experts, where a group's score is the sum of its ``group_best`` (1 or
    2) largest; ties go to the lower index, as in 64 bits. Weights are s, or with
    ``renormalise`` its share among the token's chosen, times ``scale``. An expert with
    logit or bias -inf is out of reach; a token that reaches fewer than k has experts -1
    with weight 0 for the rest."""
    return (_fp4 or _load_fp4()).route(logits, k, bias, _score_code(score), groups, kept, group_best, renormalise, scale)


def route_backward(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, score: str = "softmax",
                   renormalise: bool = True, scale: float = 1.0) -> torch.Tensor:
    """dlogits (of the logits' type) from the gradient of ``route``'s weights. The choice
    has no gradient, nor has the bias."""
    return (_fp4 or _load_fp4()).route_backward(dweights, logits, experts, _score_code(score), renormalise, scale)


def expert_plan(experts: torch.Tensor, num_experts: int) -> ExpertPlan:
    """The order by expert of the slots of ``experts`` (int32 [tokens, k], -1: none), the
    slots of one expert in their own order: an ``ExpertPlan``. Everything stays on the
    device. An index outside [-1, num_experts) counts as -1 and shows in
    ``device_status``."""
    return (_fp4 or _load_fp4()).plan(experts, num_experts)


def expert_dispatch(x: torch.Tensor, plan: ExpertPlan, out: torch.Tensor | None = None) -> torch.Tensor:
    """xs [tokens * k, n]: x's rows sorted by expert, one for each slot; zeros past the
    last expert's. out may not overlap x. Its gradient is ``expert_combine(dxs, plan)``."""
    return (_fp4 or _load_fp4()).dispatch(x, plan, out)


def expert_combine(ys: torch.Tensor, plan: ExpertPlan, weights: torch.Tensor | None = None, add: torch.Tensor | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """y [tokens, n] = add + the sum over a token's slots of weights (fp32 [tokens, k],
    None: 1) times their rows of ys [tokens * k, n], in fp32 and rounded once to ys's
    type; slots of no expert count for nothing. out may be add, but not overlap it otherwise,
    nor ys."""
    return (_fp4 or _load_fp4()).combine(ys, plan, weights, add, out)


def expert_combine_backward(dy: torch.Tensor, ys: torch.Tensor, plan: ExpertPlan, weights: torch.Tensor):
    """(dys, dweights) of ``expert_combine``: dys [tokens * k, n] of ys's type, zeros
    past the last expert's rows; dweights fp32 [tokens, k]. The gradient of ``add`` is dy."""
    return (_fp4 or _load_fp4()).combine_backward(dy, ys, plan, weights)


def set_num_sms(n: int) -> None:
    _check("ql_set_num_sms", load_library().ql_set_num_sms(int(n)))


def get_num_sms() -> int:
    return int(load_library().ql_get_num_sms())


def set_gemm_block_n(bn: int) -> None:
    _check("ql_set_gemm_block_n", load_library().ql_set_gemm_block_n(int(bn)))


def set_gemm_path(path: int) -> None:
    """GEMM kernel choice (ql_set_gemm_path): 0 auto; CUDA-core promotion: 1
    (default kernel), 5 on CTA pairs, 6 on one SM per tile, 7 split-K over a
    cluster where a split applies; block-scaled MMA (UE8M0 formats): 2 on one
    SM per tile, 3 on CTA pairs, 4 split-K over a cluster where it applies."""
    _check("ql_set_gemm_path", load_library().ql_set_gemm_path(int(path)))


def test_stall_gemm_producer(enable: bool) -> None:
    """Failure-path test hook: GEMM producers issue no copies while enabled."""
    _check("ql_test_stall_gemm_producer", load_library().ql_test_stall_gemm_producer(int(bool(enable))))


def set_wait_limit_ms(ms: int) -> None:
    _check("ql_set_wait_limit_ms", load_library().ql_set_wait_limit_ms(int(ms)))


def device_status(device=None) -> int:
    """Synchronise the current stream and return (and clear) the device status code."""
    s = torch.cuda.current_stream(device).cuda_stream
    return int(load_library().ql_device_status(s))
