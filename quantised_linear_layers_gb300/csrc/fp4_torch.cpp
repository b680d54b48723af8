// The 4-bit calls as a Python module over torch tensors: argument checks,
// output and workspace allocation, and the C ABI's entry points
// (include/qlinear.h), which it is handed as addresses. At these sizes a call's
// host time is most of its cost; done in Python it was twice this.
//
// No arithmetic here. Errors: ValueError / TypeError for arguments, the
// binding's own error for a status of the library.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cuda_runtime_api.h>

#include <atomic>
#include <cstdint>
#include <exception>
#include <stdexcept>
#include <string>

#include "../../include/qlinear.h"

namespace {

struct Api {
    decltype(&::fp4_tensor_scale) tensor_scale;
    decltype(&::fp4_cast) cast;
    decltype(&::fp4_cast_dual) cast_dual;
    decltype(&::fp4_dequant) dequant;
    decltype(&::fp4_linear) linear;
    decltype(&::fp4_linear_workspace_size) linear_ws;
    decltype(&::fp4_row_stride) row_stride;
    decltype(&::gemm_fp4_nt) gemm;
    decltype(&::gemm_fp4_nt_ragged) ragged;
    decltype(&::gemm_fp4_wgrad_ragged) wgrad;
} api;

PyObject* g_class = nullptr;     // FP4Tensor
PyObject* g_own = nullptr;       // FP4_OWN_SCALE
PyObject* g_error = nullptr;     // callable(function name, status) that raises
PyObject *n_q, *n_sf, *n_scale, *n_ld, *n_fmt, *n_batch, *n_rows, *n_cols, *n_offsets, *n_by_cols, *n_device;

struct Raised {};                // a Python error is set

[[noreturn]] void value_error(const char* msg) { throw std::invalid_argument(msg); }

void status(const char* fn, ql_status s) {
    if (s == QL_OK) return;
    PyObject* r = PyObject_CallFunction(g_error, "si", fn, static_cast<int>(s));
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, fn);
    throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* msg) {
    if (!THPVariable_Check(o)) value_error(msg);
    return THPVariable_Unpack(o);
}
const at::Tensor& cuda_tensor(PyObject* o) {
    const at::Tensor& t = tensor(o, "x must be a CUDA tensor");
    if (!t.is_cuda()) value_error("x must be a CUDA tensor");
    return t;
}
ql_dtype dtype_code(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return QL_BF16;
    if (t.scalar_type() == at::kFloat) return QL_F32;
    PyErr_Format(PyExc_TypeError, "input must be bfloat16 or float32, got %s", c10::toString(t.scalar_type()));
    throw Raised{};
}
ql_stream_t stream_of(const at::Device& d) {
    return reinterpret_cast<ql_stream_t>(c10::cuda::getCurrentCUDAStream(d.index()).stream());
}
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int format(PyObject* o) {
    const long f = PyLong_AsLong(o);
    if (f == -1 && PyErr_Occurred()) throw Raised{};
    if (f != QL_FP4_NV && f != QL_FP4_MX) value_error("fmt must be FP4_NV or FP4_MX");
    return static_cast<int>(f);
}

// at::empty without the way through the dispatcher
at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType type, const at::Device& d) {
    return at::Tensor(at::detail::empty_cuda(shape, type, d, std::nullopt));
}
at::Tensor new_bytes(int64_t n, const at::Device& d) { return new_tensor({n}, at::kByte, d); }

// One cast input: sizes, strides and the experts.
struct Input {
    const at::Tensor* x;
    ql_dtype code;
    int64_t batch, m, k, sb, sm, sk;
    int experts;
    const int32_t* offsets;
    float* scale;        // given by the caller, or null
    bool own;            // made in the call
};

// Sizes and strides of a matrix or a batch. A dimension of size one may have any
// stride (torch calls [4, 1, 64] with strides (64, 256, 1) contiguous): it gets
// one that holds for whoever takes the batch's rows as one long matrix.
void layout(const at::Tensor& x, Input& in) {
    in.batch = x.dim() == 3 ? x.size(0) : 1;
    in.m = x.size(-2);
    in.k = x.size(-1);
    in.sb = in.batch > 1 ? x.stride(0) : 0;
    in.sm = in.m == 1 ? in.sb : x.stride(-2);
    in.sk = in.k == 1 ? 1 : x.stride(-1);
}

int experts_of(const at::Tensor& o, const at::Device& d) {
    if (o.scalar_type() != at::kInt || o.dim() != 1 || !o.is_contiguous() || o.size(0) < 2 || o.device() != d)
        value_error("offsets must be a contiguous int32 [experts + 1] tensor on x's device");
    return static_cast<int>(o.size(0) - 1);
}

Input input(PyObject* ox, int fmt, PyObject* oscale, PyObject* ooffsets) {
    const at::Tensor& x = cuda_tensor(ox);
    if (x.dim() != 2 && x.dim() != 3) value_error("x must be 2-D or a batch of 2-D matrices");
    Input in{};
    in.x = &x;
    layout(x, in);
    in.code = dtype_code(x);
    if (oscale != Py_None && fmt == QL_FP4_NV) {        // FP4_MX has none and takes no notice of one
        if (oscale == g_own) {
            in.own = true;
            // one matrix below the other, or (transposed views) one beside the other
            if (in.batch > 1 && in.sb != in.m * in.sm && !(in.sm == 1 && in.sb == in.k * in.sk))
                value_error("x's matrices must follow one another for a scale of their own");
        } else {
            const at::Tensor& s = tensor(oscale, "tensor_scale must be a tensor, FP4_OWN_SCALE or None");
            if (s.scalar_type() != at::kFloat || s.numel() != 1 || s.device() != x.device())
                value_error("tensor_scale must be one fp32 value on x's device");
            in.scale = s.data_ptr<float>();
        }
    }
    if (ooffsets != Py_None) {
        const at::Tensor& o = tensor(ooffsets, "offsets must be a contiguous int32 [experts + 1] tensor on x's device");
        in.experts = experts_of(o, x.device());
        if (x.dim() != 2) value_error("x must be 2-D with offsets");
        in.offsets = o.data_ptr<int32_t>();
    }
    return in;
}

// The layers' calls take x with any strides: `copy` holds one with contiguous
// rows where x's are not.
void contiguous_rows(Input& in, at::Tensor& copy) {
    if (in.sk == 1 || in.k <= 1) return;
    copy = in.x->contiguous();
    in.x = &copy;
    in.sm = copy.stride(-2);
    in.sk = 1;
}

// Device memory for the length of a call, from torch's allocator (no tensor
// around it: 1.0 us less).
c10::DataPtr scratch(int64_t n) { return c10::cuda::CUDACachingAllocator::get()->allocate(static_cast<size_t>(n)); }

// Codes, scale blocks and (last 16 bytes) a scale of one cast, in one buffer: a
// tensor for an FP4Tensor, or scratch.
enum class For { kResult, kCall };
struct Room {
    at::Tensor buf;
    c10::DataPtr mem;
    uint8_t* q;
    int64_t ld;
    uint8_t* sf;
    float* own;
};
Room room(int64_t batch, int64_t rows, int64_t ld, int64_t row_blocks, int64_t kcols, int fmt, const at::Device& d, For use) {
    Room r;
    const int64_t codes = batch * rows * ld;
    const int64_t bytes = codes + batch * row_blocks * ceil_div(kcols, fmt == QL_FP4_NV ? 64 : 128) * 512 + 16;
    if (use == For::kCall) {
        r.mem = scratch(bytes);
        r.q = static_cast<uint8_t*>(r.mem.get());
    } else {
        r.buf = new_bytes(bytes, d);
        r.q = r.buf.data_ptr<uint8_t>();
    }
    r.ld = ld;
    r.sf = r.q + codes;
    r.own = reinterpret_cast<float*>(r.q + bytes - 16);
    return r;
}
Room row_room(const Input& in, int fmt, For use) {
    return room(in.batch, in.m, api.row_stride(in.k), ceil_div(in.m, 128) + in.experts, in.k, fmt, in.x->device(), use);
}
Room column_room(const Input& in, int fmt, For use) {
    const int64_t m1 = in.m > 0 ? in.m : 1;
    const int64_t extent = in.experts > 0 ? (ceil_div(in.m, 256) + in.experts) * 256 : ceil_div(m1, 128) * 128;
    return room(in.batch, in.k, api.row_stride(extent), ceil_div(in.k, 128), in.experts > 0 ? extent : in.m, fmt, in.x->device(),
                use);
}

// FP4Tensor(buf, ld, scale, fmt, batch, rows, cols, offsets, by_cols)
PyObject* wrap(const Room& r, PyObject* scale, int fmt, int64_t batch, int64_t rows, int64_t cols, PyObject* offsets,
               bool by_cols) {
    if (fmt == QL_FP4_MX) scale = Py_None;
    PyObject* a[9] = {THPVariable_Wrap(r.buf), PyLong_FromLongLong(r.ld), scale, PyLong_FromLong(fmt),
                      PyLong_FromLongLong(batch), PyLong_FromLongLong(rows), PyLong_FromLongLong(cols), offsets,
                      by_cols ? Py_True : Py_False};
    PyObject* o = PyObject_Vectorcall(g_class, a, 9, nullptr);
    for (int i : {0, 1, 3, 4, 5, 6}) Py_XDECREF(a[i]);
    if (o == nullptr) throw Raised{};
    return o;
}

// An FP4Tensor as an operand.
struct Operand {
    uint8_t *q, *sf;
    float* scale;
    int64_t ld, batch, rows, cols;
    int fmt;
    bool by_cols;
    const at::Tensor* offsets;       // null: none
    at::Device device{at::kCUDA, 0};
};
int64_t int_attr(PyObject* o, PyObject* name) {
    PyObject* v = PyObject_GetAttr(o, name);
    if (v == nullptr) throw Raised{};
    const int64_t r = v == Py_None ? 0 : PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (r == -1 && PyErr_Occurred()) throw Raised{};
    return r;
}
Operand operand(PyObject* o) {
    if (Py_TYPE(o) != reinterpret_cast<PyTypeObject*>(g_class)) value_error("the operands must be FP4Tensors");
    Operand a;
    a.q = reinterpret_cast<uint8_t*>(int_attr(o, n_q));
    a.sf = reinterpret_cast<uint8_t*>(int_attr(o, n_sf));
    a.scale = reinterpret_cast<float*>(int_attr(o, n_scale));
    a.ld = int_attr(o, n_ld);
    a.fmt = static_cast<int>(int_attr(o, n_fmt));
    a.batch = int_attr(o, n_batch);
    a.rows = int_attr(o, n_rows);
    a.cols = int_attr(o, n_cols);
    a.by_cols = int_attr(o, n_by_cols) != 0;
    a.device = at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(int_attr(o, n_device)));
    PyObject* off = PyObject_GetAttr(o, n_offsets);
    if (off == nullptr) throw Raised{};
    a.offsets = off == Py_None ? nullptr : &THPVariable_Unpack(off);
    Py_DECREF(off);                  // the FP4Tensor keeps it
    return a;
}
void same_kind(const Operand& x, const Operand& w) {
    if (x.fmt != w.fmt) value_error("the operands' formats differ");
    if (x.cols != w.cols) value_error("the operands must share K");
    if (x.device != w.device) value_error("the operands must be on one device");
}

// The output: given (checked) or new. D's row stride is its second last stride.
// Rows that no expert has are left alone in a given one and zero in a new one.
struct Out {
    at::Tensor t;
    ql_dtype code;
    int64_t ld;
    int zero_rest;       // QL_FP4_ZERO_REST for a new one
};
Out output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const at::Device& d, bool accumulate) {
    Out r{};
    if (o == Py_None) {
        if (accumulate) value_error("accumulate needs an existing out");
        r.zero_rest = QL_FP4_ZERO_REST;
        r.t = new_tensor(shape, type, d);
    } else {
        r.t = tensor(o, "out must be a tensor");
        const bool type_ok = r.t.scalar_type() == at::kBFloat16 || r.t.scalar_type() == at::kFloat;
        // rows that overlap (an expanded tensor's) are no room for them
        if (!type_ok || r.t.sizes() != shape || r.t.device() != d || (r.t.size(-1) > 1 && r.t.stride(-1) != 1) ||
            (r.t.size(-2) > 1 && r.t.stride(-2) < r.t.size(-1)))
            value_error("out must be bf16 or fp32 of the result's shape with contiguous rows on the operands' device");
        if (accumulate && r.t.scalar_type() != at::kFloat) value_error("accumulate needs an fp32 out");
    }
    r.code = r.t.scalar_type() == at::kFloat ? QL_F32 : QL_BF16;
    const int64_t n = shape.back();
    r.ld = r.t.stride(-2) > n ? r.t.stride(-2) : n;
    return r;
}

// ---------------------------------------------------------------- launches
void launch_cast(const Input& in, int fmt, const Room& r) {
    status("fp4_cast", api.cast(in.x->data_ptr(), in.code, in.batch, in.m, in.k, in.sb, in.sm, in.sk, fmt,
                                in.own ? r.own : in.scale, in.own, r.q, r.ld, r.sf, in.offsets, in.experts,
                                stream_of(in.x->device())));
}
// rows: null to leave them out; the scale is in the columns' room
void launch_dual(const Input& in, int fmt, const Room* rows, const Room& cols) {
    if (in.sk != 1 && in.k > 1) value_error("x must have contiguous rows");
    status("fp4_cast_dual",
           api.cast_dual(in.x->data_ptr(), in.code, in.batch, in.m, in.k, in.sb, in.sm, fmt, in.own ? cols.own : in.scale,
                         in.own, rows ? rows->q : nullptr, rows ? rows->ld : 0, rows ? rows->sf : nullptr, cols.q, cols.ld,
                         cols.sf, in.offsets, in.experts, stream_of(in.x->device())));
}
Operand as_operand(const Input& in, int fmt, const Room& r, float* scale, bool columns) {
    Operand a;
    a.q = r.q;
    a.sf = r.sf;
    a.ld = r.ld;
    a.scale = scale;
    a.fmt = fmt;
    a.batch = in.batch;
    a.rows = columns ? in.k : in.m;
    a.cols = columns ? in.m : in.k;
    a.by_cols = columns && in.experts > 0;
    a.offsets = nullptr;
    a.device = in.x->device();
    return a;
}
void launch_gemm(const Operand& x, const Operand& w, const Out& d, bool accumulate) {
    status("gemm_fp4_nt", api.gemm(x.q, x.ld, x.sf, x.scale, w.q, w.ld, w.sf, w.scale, x.fmt, d.t.data_ptr(), d.code, d.ld,
                                   x.rows, w.rows, x.cols, accumulate, stream_of(x.device)));
}
void launch_ragged(const Operand& x, const Operand& w, const int32_t* offsets, const Out& d) {
    status("gemm_fp4_nt_ragged",
           api.ragged(x.q, x.ld, x.sf, x.scale, w.q, w.ld, w.sf, w.scale, x.fmt | d.zero_rest, d.t.data_ptr(), d.code, d.ld, offsets,
                      static_cast<int>(w.batch), x.rows, w.rows, x.cols, stream_of(x.device)));
}
void launch_wgrad(const Operand& y, const Operand& x, const int32_t* offsets, int experts, const Out& d, bool accumulate) {
    status("gemm_fp4_wgrad_ragged",
           api.wgrad(y.q, y.ld, y.sf, y.scale, x.q, x.ld, x.sf, x.scale, y.fmt, d.t.data_ptr<float>(), x.rows, offsets,
                     experts, y.cols, y.rows, x.rows, accumulate, stream_of(y.device)));
}
void check_fp32_whole(const Out& d) {
    if (d.code != QL_F32 || !d.t.is_contiguous()) value_error("out must be contiguous fp32");
}
// the weight of a forward or data-gradient product of x
void check_weight(const Input& in, const Operand& w) {
    if (in.x->dim() != 2 || in.k != w.cols || in.x->device() != w.device)
        value_error("x must be [m, k] with w's k, on w's device");
    if (w.offsets != nullptr || w.batch != (in.experts > 0 ? in.experts : 1))
        value_error("w must be the cast of one matrix, or of one per expert with offsets");
}

// ---------------------------------------------------------------- functions
using Args = PyObject* const*;

PyObject* f_tensor_scale(Args a) {
    const at::Tensor& x0 = cuda_tensor(a[0]);
    if (x0.dim() != 2 && x0.dim() != 3) value_error("x must be a 2-D or 3-D CUDA tensor");
    const ql_dtype code = dtype_code(x0);
    c10::cuda::CUDAGuard guard(x0.device());
    Input in{};
    layout(x0, in);
    at::Tensor x = x0;
    if (in.batch > 1 && in.sb != in.m * in.sm) {       // its rows do not follow one another: m > 1
        x = x0.contiguous();
        layout(x, in);
    }
    at::Tensor out = new_tensor({1}, at::kFloat, x.device());
    status("fp4_tensor_scale", api.tensor_scale(x.data_ptr(), code, in.batch * in.m, in.k, in.sm, in.sk,
                                                out.data_ptr<float>(), stream_of(x.device())));
    return THPVariable_Wrap(out);
}

// (x, fmt, tensor_scale, offsets)
PyObject* f_cast(Args a) {
    const int fmt = format(a[1]);
    Input in = input(a[0], fmt, a[2], a[3]);
    c10::cuda::CUDAGuard guard(in.x->device());
    const bool turned = in.sk != 1 && in.sm == 1 && in.m > 1;
    if (in.offsets == nullptr && turned && !(in.own && in.batch > 1 && in.sb != in.k * in.sk)) {
        // a transposed view: the column-wise cast of the matrix it views (whose scale
        // needs those matrices to follow one another)
        Input t = in;
        std::swap(t.m, t.k);
        std::swap(t.sm, t.sk);
        const Room r = column_room(t, fmt, For::kResult);
        launch_dual(t, fmt, nullptr, r);
        return wrap(r, a[2], fmt, in.batch, in.m, in.k, Py_None, false);
    }
    const Room r = row_room(in, fmt, For::kResult);
    launch_cast(in, fmt, r);
    return wrap(r, a[2], fmt, in.batch, in.m, in.k, a[3], false);
}

// (x, fmt, tensor_scale, offsets, rows)
PyObject* f_cast_dual(Args a) {
    const int fmt = format(a[1]);
    const Input in = input(a[0], fmt, a[2], a[3]);
    const bool rows = PyObject_IsTrue(a[4]) == 1;
    if (in.sk != 1 && in.k > 1) value_error("x must have contiguous rows");
    c10::cuda::CUDAGuard guard(in.x->device());
    const Room c = column_room(in, fmt, For::kResult);
    Room r;
    if (rows) r = row_room(in, fmt, For::kResult);
    launch_dual(in, fmt, rows ? &r : nullptr, c);
    PyObject* oc = wrap(c, a[2], fmt, in.batch, in.k, in.m, a[3], in.experts > 0);
    PyObject* orow = Py_None;
    if (rows) {
        try {
            orow = wrap(r, a[2] == Py_None ? Py_None : oc, fmt, in.batch, in.m, in.k, a[3], false);
        } catch (...) {
            Py_DECREF(oc);
            throw;
        }
    } else {
        Py_INCREF(orow);
    }
    PyObject* res = PyTuple_Pack(2, orow, oc);
    Py_DECREF(orow);
    Py_DECREF(oc);
    return res;
}

// (a, out, bf16)
PyObject* f_dequant(Args a) {
    const Operand x = operand(a[0]);
    if (x.batch != 1 || x.offsets != nullptr) value_error("fp4_dequant takes the cast of one matrix");
    c10::cuda::CUDAGuard guard(x.device);
    const Out d = output(a[1], {x.rows, x.cols}, PyObject_IsTrue(a[2]) ? at::kBFloat16 : at::kFloat, x.device, false);
    status("fp4_dequant", api.dequant(x.q, x.ld, x.sf, x.fmt, x.scale, x.rows, x.cols, d.t.data_ptr(), d.code, d.ld,
                                      stream_of(x.device)));
    return THPVariable_Wrap(d.t);
}

// (x, w, out, bf16, accumulate)
PyObject* f_gemm(Args a) {
    const Operand x = operand(a[0]), w = operand(a[1]);
    same_kind(x, w);
    if (x.batch != 1 || w.batch != 1 || x.offsets != nullptr || w.offsets != nullptr)
        value_error("gemm_fp4_nt takes casts of one matrix each");
    const bool acc = PyObject_IsTrue(a[4]) == 1;
    c10::cuda::CUDAGuard guard(x.device);
    const Out d = output(a[2], {x.rows, w.rows}, PyObject_IsTrue(a[3]) ? at::kBFloat16 : at::kFloat, x.device, acc);
    launch_gemm(x, w, d, acc);
    return THPVariable_Wrap(d.t);
}

// (x, w, out, bf16)
PyObject* f_ragged(Args a) {
    const Operand x = operand(a[0]), w = operand(a[1]);
    same_kind(x, w);
    if (x.offsets == nullptr || x.by_cols || w.offsets != nullptr || w.batch != x.offsets->size(0) - 1)
        value_error("x must be cast by expert and w hold one matrix per expert");
    c10::cuda::CUDAGuard guard(x.device);
    const Out d = output(a[2], {x.rows, w.rows}, PyObject_IsTrue(a[3]) ? at::kBFloat16 : at::kFloat, x.device, false);
    launch_ragged(x, w, x.offsets->data_ptr<int32_t>(), d);
    return THPVariable_Wrap(d.t);
}

// (y, x, out, accumulate)
PyObject* f_wgrad(Args a) {
    const Operand y = operand(a[0]), x = operand(a[1]);
    same_kind(y, x);
    if (!y.by_cols || !x.by_cols || y.offsets->sizes() != x.offsets->sizes())
        value_error("both operands must be column-wise casts by the same experts");
    const bool acc = PyObject_IsTrue(a[3]) == 1;
    const int experts = static_cast<int>(y.offsets->size(0) - 1);
    c10::cuda::CUDAGuard guard(y.device);
    const Out d = output(a[2], {experts, y.rows, x.rows}, at::kFloat, y.device, acc);
    check_fp32_whole(d);
    launch_wgrad(y, x, y.offsets->data_ptr<int32_t>(), experts, d, acc);
    return THPVariable_Wrap(d.t);
}

// (x, w, x_scale, offsets, out)
PyObject* f_linear(Args a) {
    const Operand w = operand(a[1]);
    Input in = input(a[0], w.fmt, a[2], a[3]);
    check_weight(in, w);
    c10::cuda::CUDAGuard guard(in.x->device());
    at::Tensor copy;
    contiguous_rows(in, copy);
    const Out d = output(a[4], {in.m, w.rows}, at::kBFloat16, w.device, false);
    if (d.code != QL_BF16) value_error("out must be bf16");
    const int64_t size = static_cast<int64_t>(api.linear_ws(in.m, in.k, w.fmt, in.experts));
    c10::DataPtr ws;
    uint8_t* p = nullptr;
    if (size > 0 || in.own) {
        ws = scratch(size + 16);       // the scale is at its end
        p = static_cast<uint8_t*>(ws.get());
    }
    status("fp4_linear", api.linear(in.x->data_ptr(), in.code, in.sm, in.own ? reinterpret_cast<float*>(p + size) : in.scale,
                                    in.own, w.q, w.ld, w.sf, w.scale, w.fmt | d.zero_rest, d.t.data_ptr(), d.ld, in.offsets,
                                    in.experts, in.m, w.rows, in.k, p, static_cast<size_t>(size), stream_of(w.device)));
    return THPVariable_Wrap(d.t);
}

// (x, w, x_scale, offsets): the product and the cast of x along its columns
PyObject* f_linear_saving(Args a) {
    const Operand w = operand(a[1]);
    Input in = input(a[0], w.fmt, a[2], a[3]);
    check_weight(in, w);
    c10::cuda::CUDAGuard guard(in.x->device());
    at::Tensor copy;
    contiguous_rows(in, copy);
    const Out d = output(Py_None, {in.m, w.rows}, at::kBFloat16, w.device, false);
    const Room c = column_room(in, w.fmt, For::kResult), r = row_room(in, w.fmt, For::kCall);
    launch_dual(in, w.fmt, &r, c);
    const Operand x = as_operand(in, w.fmt, r, in.own ? c.own : in.scale, false);
    if (in.offsets != nullptr) launch_ragged(x, w, in.offsets, d);
    else launch_gemm(x, w, d, false);
    PyObject* oc = wrap(c, a[2], w.fmt, 1, in.k, in.m, a[3], in.experts > 0);
    PyObject* od = THPVariable_Wrap(d.t);
    PyObject* res = PyTuple_Pack(2, od, oc);
    Py_DECREF(od);
    Py_DECREF(oc);
    return res;
}

// (dy, wt, x_cols, dy_scale, offsets, dw_out, accumulate): wt the cast of W^T,
// or None for no dX; x_cols from linear_saving
PyObject* f_linear_backward(Args a) {
    const bool need_dx = a[1] != Py_None;
    const Operand xc = operand(a[2]);
    Input in = input(a[0], xc.fmt, a[3], a[4]);
    const bool acc = PyObject_IsTrue(a[6]) == 1;
    Operand wt;
    if (need_dx) {
        wt = operand(a[1]);
        if (wt.fmt != xc.fmt) value_error("the operands' formats differ");
        check_weight(in, wt);
    }
    if (in.x->dim() != 2 || in.m != xc.cols || in.x->device() != xc.device || xc.batch != 1 ||
        xc.by_cols != (in.experts > 0) || (xc.offsets != nullptr) != (in.experts > 0) ||
        (in.experts > 0 && xc.offsets->size(0) - 1 != in.experts))
        value_error("dy must have the rows, experts and device of the forward call");
    c10::cuda::CUDAGuard guard(in.x->device());
    at::Tensor copy;
    contiguous_rows(in, copy);
    const Out dw = in.experts > 0 ? output(a[5], {in.experts, in.k, xc.rows}, at::kFloat, xc.device, acc)
                                  : output(a[5], {in.k, xc.rows}, at::kFloat, xc.device, acc);
    if (dw.code != QL_F32) value_error("dw_out must be fp32");
    if (in.experts > 0) check_fp32_whole(dw);
    Out dx;
    if (need_dx) dx = output(Py_None, {in.m, wt.rows}, at::kBFloat16, xc.device, false);
    const Room c = column_room(in, xc.fmt, For::kCall);
    Room r;
    if (need_dx) r = row_room(in, xc.fmt, For::kCall);
    launch_dual(in, xc.fmt, need_dx ? &r : nullptr, c);
    float* scale = in.own ? c.own : in.scale;
    if (need_dx) {
        const Operand dy = as_operand(in, xc.fmt, r, scale, false);
        if (in.offsets != nullptr) launch_ragged(dy, wt, in.offsets, dx);
        else launch_gemm(dy, wt, dx, false);
    }
    const Operand dyc = as_operand(in, xc.fmt, c, scale, true);
    if (in.offsets != nullptr) launch_wgrad(dyc, xc, in.offsets, in.experts, dw, acc);
    else launch_gemm(dyc, xc, dw, acc);
    PyObject* odx = need_dx ? THPVariable_Wrap(dx.t) : Py_NewRef(Py_None);
    PyObject* odw = THPVariable_Wrap(dw.t);
    PyObject* res = PyTuple_Pack(2, odx, odw);
    Py_DECREF(odx);
    Py_DECREF(odw);
    return res;
}

// Objects that graphs hold, and those whose graphs are gone: a list, since the
// runtime says so on a thread of its own, which may call neither Python nor CUDA.
struct Held {
    PyObject* object;
    Held* next;
};
std::atomic<Held*> g_dropped{nullptr};
void CUDART_CB graph_gone(void* p) {
    Held* h = static_cast<Held*>(p);
    h->next = g_dropped.load(std::memory_order_relaxed);
    while (!g_dropped.compare_exchange_weak(h->next, h, std::memory_order_release, std::memory_order_relaxed)) {
    }
}
void check_cuda(cudaError_t e) {
    if (e != cudaSuccess) throw std::runtime_error(cudaGetErrorString(e));
}

// (object, event): object is kept alive by the graph that the current stream
// captures into, and by every executable made from it; the host waits for the event
// behind the work that made it, which a capture cannot.
PyObject* f_hold(Args a) {
    void* event = PyLong_AsVoidPtr(a[1]);
    if (event == nullptr && PyErr_Occurred()) throw Raised{};
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    cudaGraph_t graph = nullptr;
    check_cuda(cudaStreamGetCaptureInfo(c10::cuda::getCurrentCUDAStream().stream(), &status, &id, &graph));
    if (status != cudaStreamCaptureStatusActive || graph == nullptr) value_error("the current stream captures no graph");
    if (event != nullptr) {
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;       // else a wait ends the capture
        check_cuda(cudaThreadExchangeStreamCaptureMode(&mode));
        cudaError_t e;
        Py_BEGIN_ALLOW_THREADS
        e = cudaEventSynchronize(static_cast<cudaEvent_t>(event));
        Py_END_ALLOW_THREADS
        check_cuda(cudaThreadExchangeStreamCaptureMode(&mode));
        check_cuda(e);
    }
    Held* h = new Held{Py_NewRef(a[0]), nullptr};
    cudaUserObject_t object;
    if (cudaError_t e = cudaUserObjectCreate(&object, h, graph_gone, 1, cudaUserObjectNoDestructorSync); e != cudaSuccess) {
        Py_DECREF(h->object);
        delete h;
        check_cuda(e);
    }
    if (cudaError_t e = cudaGraphRetainUserObject(graph, object, 1, cudaGraphUserObjectMove); e != cudaSuccess) {
        cudaUserObjectRelease(object, 1);
        check_cuda(e);
    }
    Py_RETURN_NONE;
}

// (): lets go of what only graphs held that are gone.
PyObject* f_drop(Args) {
    for (Held* h = g_dropped.exchange(nullptr, std::memory_order_acquire); h != nullptr;) {
        Held* next = h->next;
        Py_DECREF(h->object);
        delete h;
        h = next;
    }
    Py_RETURN_NONE;
}

template <PyObject* (*F)(Args), int N>
PyObject* entry(PyObject*, Args a, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(a);
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch != nullptr ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type != nullptr) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error in a 4-bit call");
    }
    return nullptr;
}

// (addresses, FP4Tensor, FP4_OWN_SCALE, error callable)
PyObject* bind(PyObject*, Args a, Py_ssize_t n) {
    if (n != 4 || !PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 10) {
        PyErr_SetString(PyExc_TypeError, "bind(addresses, class, own, error)");
        return nullptr;
    }
    void* p[10];
    for (int i = 0; i < 10; ++i) {
        p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[0], i));
        if (p[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    api.tensor_scale = reinterpret_cast<decltype(api.tensor_scale)>(p[0]);
    api.cast = reinterpret_cast<decltype(api.cast)>(p[1]);
    api.cast_dual = reinterpret_cast<decltype(api.cast_dual)>(p[2]);
    api.dequant = reinterpret_cast<decltype(api.dequant)>(p[3]);
    api.linear = reinterpret_cast<decltype(api.linear)>(p[4]);
    api.linear_ws = reinterpret_cast<decltype(api.linear_ws)>(p[5]);
    api.row_stride = reinterpret_cast<decltype(api.row_stride)>(p[6]);
    api.gemm = reinterpret_cast<decltype(api.gemm)>(p[7]);
    api.ragged = reinterpret_cast<decltype(api.ragged)>(p[8]);
    api.wgrad = reinterpret_cast<decltype(api.wgrad)>(p[9]);
    g_class = Py_NewRef(a[1]);
    g_own = Py_NewRef(a[2]);
    g_error = Py_NewRef(a[3]);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction cfunction(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}

PyMethodDef methods[] = {
    {"bind", cfunction(bind), METH_FASTCALL, nullptr},
    {"tensor_scale", cfunction(entry<f_tensor_scale, 1>), METH_FASTCALL, nullptr},
    {"cast", cfunction(entry<f_cast, 4>), METH_FASTCALL, nullptr},
    {"cast_dual", cfunction(entry<f_cast_dual, 5>), METH_FASTCALL, nullptr},
    {"dequant", cfunction(entry<f_dequant, 3>), METH_FASTCALL, nullptr},
    {"gemm", cfunction(entry<f_gemm, 5>), METH_FASTCALL, nullptr},
    {"ragged", cfunction(entry<f_ragged, 4>), METH_FASTCALL, nullptr},
    {"wgrad", cfunction(entry<f_wgrad, 4>), METH_FASTCALL, nullptr},
    {"linear", cfunction(entry<f_linear, 5>), METH_FASTCALL, nullptr},
    {"linear_saving", cfunction(entry<f_linear_saving, 4>), METH_FASTCALL, nullptr},
    {"hold_in_graph", cfunction(entry<f_hold, 2>), METH_FASTCALL, nullptr},
    {"drop_held", cfunction(entry<f_drop, 0>), METH_FASTCALL, nullptr},
    {"linear_backward", cfunction(entry<f_linear_backward, 7>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp4", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp4() {
    PyObject** names[] = {&n_q, &n_sf, &n_scale, &n_ld, &n_fmt, &n_batch, &n_rows, &n_cols, &n_offsets, &n_by_cols, &n_device};
    const char* text[] = {"q_ptr", "sf_ptr", "scale_ptr", "ld", "fmt", "batch", "rows", "cols", "offsets", "by_cols",
                          "device_index"};
    for (int i = 0; i < 11; ++i)
        if ((*names[i] = PyUnicode_InternFromString(text[i])) == nullptr) return nullptr;
    return PyModule_Create(&module);
}
