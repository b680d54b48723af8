// Layer norm, routing and the exchange with the experts as functions of the Python
// module (fp4_torch.cpp, which includes this file once inside its namespace, after its
// helpers).

struct LayerApi {
    decltype(&::layer_norm) norm;
    decltype(&::layer_norm_backward) norm_back;
    decltype(&::layer_norm_backward_workspace_size) norm_back_ws;
    decltype(&::expert_route) route;
    decltype(&::expert_route_backward) route_back;
    decltype(&::expert_plan) plan;
    decltype(&::expert_plan_workspace_size) plan_ws;
    decltype(&::expert_dispatch) dispatch;
    decltype(&::expert_combine) combine;
    decltype(&::expert_combine_backward) combine_back;
} layers;
constexpr int kLayerEntries = 10;

PyObject* g_plan_class = nullptr;        // ExpertPlan
PyObject *n_plan_rows, *n_plan_offsets;

void bind_layers(void* const* p) {
    layers.norm = reinterpret_cast<decltype(layers.norm)>(p[0]);
    layers.norm_back = reinterpret_cast<decltype(layers.norm_back)>(p[1]);
    layers.norm_back_ws = reinterpret_cast<decltype(layers.norm_back_ws)>(p[2]);
    layers.route = reinterpret_cast<decltype(layers.route)>(p[3]);
    layers.route_back = reinterpret_cast<decltype(layers.route_back)>(p[4]);
    layers.plan = reinterpret_cast<decltype(layers.plan)>(p[5]);
    layers.plan_ws = reinterpret_cast<decltype(layers.plan_ws)>(p[6]);
    layers.dispatch = reinterpret_cast<decltype(layers.dispatch)>(p[7]);
    layers.combine = reinterpret_cast<decltype(layers.combine)>(p[8]);
    layers.combine_back = reinterpret_cast<decltype(layers.combine_back)>(p[9]);
}

// A matrix with contiguous rows: the tensor itself, or a copy of it. Its row stride
// counts only where there is more than one row.
struct Matrix {
    at::Tensor t;
    ql_dtype code;
    int64_t m, n, ld;
};
Matrix matrix(PyObject* o, const char* msg, const at::Device* on = nullptr) {
    if (!THPVariable_Check(o)) value_error(msg);
    Matrix r;
    r.t = THPVariable_Unpack(o);
    if (!r.t.is_cuda() || r.t.dim() != 2 || (on != nullptr && r.t.device() != *on)) value_error(msg);
    r.code = dtype_code(r.t);
    r.m = r.t.size(0);
    r.n = r.t.size(1);
    if (r.n > 1 && r.t.stride(1) != 1) r.t = r.t.contiguous();
    r.ld = r.m > 1 ? r.t.stride(0) : r.n;
    return r;
}
// An output of these sizes: given or new.
Matrix result(PyObject* o, int64_t m, int64_t n, at::ScalarType type, const at::Device& d) {
    Matrix r;
    r.m = m;
    r.n = n;
    r.code = type == at::kFloat ? QL_F32 : QL_BF16;
    if (o == nullptr || o == Py_None) {
        r.t = new_tensor({m, n}, type, d);
        r.ld = n;
        return r;
    }
    r.t = tensor(o, "out must be a tensor");
    if (r.t.scalar_type() != type || r.t.dim() != 2 || r.t.size(0) != m || r.t.size(1) != n || r.t.device() != d ||
        (n > 1 && r.t.stride(1) != 1) || (m > 1 && r.t.stride(0) < n))
        value_error("out must be of the result's type and shape with contiguous rows on the inputs' device");
    r.ld = m > 1 ? r.t.stride(0) : n;
    return r;
}
// A given out is written while other rows are still read: it may not meet an input in memory, but
// (in_place) be it, with the same type and stride. Rows side by side in one buffer do not meet.
void refuse_overlap(const Matrix& out, const Matrix& in, bool in_place, const char* msg) {
    if (out.m == 0 || out.n == 0 || in.m == 0 || in.n == 0) return;
    const int64_t eo = out.code == QL_BF16 ? 2 : 4, ei = in.code == QL_BF16 ? 2 : 4;
    const int64_t po = reinterpret_cast<intptr_t>(out.t.data_ptr()), pi = reinterpret_cast<intptr_t>(in.t.data_ptr());
    const int64_t wo = out.n * eo, wi = in.n * ei;
    if (po + (out.m - 1) * out.ld * eo + wo <= pi || pi + (in.m - 1) * in.ld * ei + wi <= po) return;
    if (in_place && po == pi && out.code == in.code && out.m == in.m && out.n == in.n && out.ld == in.ld) return;
    const int64_t row = out.m > 1 ? out.ld * eo : in.ld * ei;
    if (row > 0 && (out.m == 1 || in.m == 1 || out.ld * eo == in.ld * ei)) {
        const int64_t d = ((pi - po) % row + row) % row;      // from a row of out to the next of in
        if (d >= wo && d + wi <= row) return;
    }
    value_error(msg);
}
// A given out has been written: autograd sees where it had saved it.
void count_write(PyObject* given, const Matrix& out) {
    if (given != Py_None && !out.t.is_inference()) out.t.unsafeGetTensorImpl()->bump_version();
}
// Two new tensors of one type that live and die together, in one storage: an allocation is a fifth
// of a small call's host time (a plan 4.7 -> 3.7 us). Of two types they could not be saved: torch
// refuses a storage that is read as both.
struct Two {
    at::Tensor a, b;
};
Two new_two(at::IntArrayRef a_shape, at::IntArrayRef b_shape, at::ScalarType type, const at::Device& d) {
    const int64_t room = (c10::multiply_integers(a_shape) + 3) / 4 * 4;
    Two r;
    r.a = new_tensor({room + c10::multiply_integers(b_shape)}, type, d);
    r.b = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(r.a.storage()), r.a.key_set(), r.a.dtype());
    r.b.unsafeGetTensorImpl()->set_storage_offset(room);
    r.b.unsafeGetTensorImpl()->set_sizes_contiguous(b_shape);
    r.a.unsafeGetTensorImpl()->set_sizes_contiguous(a_shape);
    return r;
}
bool cuda_contiguous(PyObject* o, at::ScalarType type, const at::Device& d) {
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.is_cuda() && t.scalar_type() == type && t.device() == d && t.is_contiguous();
}
// fp32 [m, k] or int32 [m, k]
const at::Tensor& table(PyObject* o, at::ScalarType type, int64_t m, int64_t k, const at::Device& d, const char* msg) {
    if (!cuda_contiguous(o, type, d)) value_error(msg);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.dim() != 2 || t.size(0) != m || (k >= 0 && t.size(1) != k)) value_error(msg);
    return t;
}
int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
int small_integer(PyObject* o) {
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) value_error("integer out of range");
    return static_cast<int>(v);
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v == 1;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(v);
}
PyObject* pair(PyObject* a, PyObject* b) {
    PyObject* r = PyTuple_Pack(2, a, b);
    Py_DECREF(a);
    Py_DECREF(b);
    return r;
}

// weight and bias of a norm over n columns, each may be None
struct Weights {
    const void *w = nullptr, *b = nullptr;
    ql_dtype code = QL_F32;
};
const void* weight_of(PyObject* o, int64_t n, const at::Device& d, Weights& r, bool first) {
    if (o == Py_None) return nullptr;
    const char* msg = "weight and bias must be contiguous [n] tensors of one type on x's device";
    const at::Tensor& t = tensor(o, msg);
    if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous() || t.device() != d) value_error(msg);
    const ql_dtype code = dtype_code(t);
    if (!first && r.w != nullptr && code != r.code) value_error(msg);
    r.code = code;
    return t.data_ptr();
}

// (x, weight, bias, eps, out, type, saving): type 0 bf16, 1 fp32, 2 that of out or x
PyObject* f_layer_norm(Args a) {
    const Matrix x = matrix(a[0], "x must be a 2-D CUDA tensor");
    const at::Device d = x.t.device();
    Weights w;
    w.w = weight_of(a[1], x.n, d, w, true);
    w.b = weight_of(a[2], x.n, d, w, false);
    const float eps = real(a[3]);
    const int64_t type = integer(a[5]);
    at::ScalarType out_type = type == 0 ? at::kBFloat16 : type == 1 ? at::kFloat : x.t.scalar_type();
    if (type == 2 && a[4] != Py_None) {
        out_type = tensor(a[4], "out must be a tensor").scalar_type();
        if (out_type != at::kBFloat16 && out_type != at::kFloat) value_error("out must be bfloat16 or float32");
    }
    const bool saving = truth(a[6]);
    c10::cuda::CUDAGuard guard(d);
    const Matrix y = result(a[4], x.m, x.n, out_type, d);
    if (a[4] != Py_None) refuse_overlap(y, x, true, "out must be x or away from it");
    at::Tensor stats;
    float* mean = nullptr;
    if (saving) {
        stats = new_tensor({2, x.m}, at::kFloat, d);
        mean = stats.data_ptr<float>();
    }
    status("layer_norm", layers.norm(x.t.data_ptr(), x.code, x.m, x.n, x.ld, w.w, w.b, w.code, eps, y.t.data_ptr(), y.code, y.ld,
                                     saving && x.m > 0 ? mean : nullptr, saving && x.m > 0 ? mean + x.m : nullptr, stream_of(d)));
    count_write(a[4], y);
    PyObject* oy = THPVariable_Wrap(y.t);
    return saving ? pair(oy, THPVariable_Wrap(stats)) : oy;
}

// (dy, x, stats, weight, sums): (dx, dweight, dbias), the last two None without sums
PyObject* f_layer_norm_backward(Args a) {
    const Matrix x = matrix(a[1], "x must be a 2-D CUDA tensor");
    const at::Device d = x.t.device();
    c10::cuda::CUDAGuard guard(d);
    const Matrix dy = matrix(a[0], "dy must be a matrix of x's shape on its device", &d);
    if (dy.m != x.m || dy.n != x.n) value_error("dy must be a matrix of x's shape on its device");
    const at::Tensor& stats = table(a[2], at::kFloat, 2, x.m, d, "stats must be those of the forward call");
    Weights w;
    w.w = weight_of(a[3], x.n, d, w, true);
    const bool sums = truth(a[4]);
    const Matrix dx = result(nullptr, x.m, x.n, x.t.scalar_type(), d);
    at::Tensor dw, db;
    c10::DataPtr ws;
    size_t size = 0;
    if (sums) {
        const Two two = new_two({x.n}, {x.n}, at::kFloat, d);
        dw = two.a;
        db = two.b;
        size = layers.norm_back_ws(x.m, x.n);
        if (size > 0) ws = scratch(static_cast<int64_t>(size));
    }
    const float* mean = stats.data_ptr<float>();
    status("layer_norm_backward",
           layers.norm_back(dy.t.data_ptr(), dy.code, dy.ld, x.t.data_ptr(), x.code, x.ld, mean, mean + x.m, w.w, w.code, x.m,
                            x.n, dx.t.data_ptr(), dx.ld, sums ? dw.data_ptr<float>() : nullptr,
                            sums ? db.data_ptr<float>() : nullptr, ws.get(), size, stream_of(d)));
    PyObject* r[3] = {THPVariable_Wrap(dx.t), sums ? THPVariable_Wrap(dw) : Py_NewRef(Py_None),
                      sums ? THPVariable_Wrap(db) : Py_NewRef(Py_None)};
    PyObject* res = PyTuple_Pack(3, r[0], r[1], r[2]);
    for (PyObject* o : r) Py_DECREF(o);
    return res;
}

// (logits, k, bias, score, groups, kept, group_best, renormalise, scale): (weights, experts)
PyObject* f_route(Args a) {
    const Matrix l = matrix(a[0], "logits must be a 2-D CUDA tensor");
    const at::Device d = l.t.device();
    const int k = small_integer(a[1]);
    const float* bias = nullptr;
    if (a[2] != Py_None) {
        if (!cuda_contiguous(a[2], at::kFloat, d) || THPVariable_Unpack(a[2]).dim() != 1 || THPVariable_Unpack(a[2]).size(0) != l.n)
            value_error("bias must be a contiguous fp32 [experts] tensor on the logits' device");
        bias = THPVariable_Unpack(a[2]).data_ptr<float>();
    }
    if (l.n < 1 || k < 1 || k > l.n) value_error("k must be between 1 and the number of experts");
    const int groups = small_integer(a[4]), kept = small_integer(a[5]), best = small_integer(a[6]);
    if (groups < 1 || l.n % groups != 0 || kept < 1 || kept > groups || best < 1 || best > 2)
        value_error("groups must divide the experts, kept be between 1 and groups, group_best 1 or 2");
    c10::cuda::CUDAGuard guard(d);
    const int experts = static_cast<int>(l.n < INT32_MAX ? l.n : INT32_MAX);
    const at::Tensor w = new_tensor({l.m, k}, at::kFloat, d), e = new_tensor({l.m, k}, at::kInt, d);
    status("expert_route", layers.route(l.t.data_ptr(), l.code, l.m, experts, l.ld, bias, k, small_integer(a[3]), groups, kept, best,
                                        truth(a[7]), real(a[8]), w.data_ptr<float>(), e.data_ptr<int32_t>(),
                                        stream_of(d)));
    return pair(THPVariable_Wrap(w), THPVariable_Wrap(e));
}

// (dweights, logits, experts, score, renormalise, scale): dlogits
PyObject* f_route_backward(Args a) {
    const Matrix l = matrix(a[1], "logits must be a 2-D CUDA tensor");
    const at::Device d = l.t.device();
    const at::Tensor& e = table(a[2], at::kInt, l.m, -1, d, "experts must be the contiguous int32 [tokens, k] of the forward call");
    const at::Tensor& dw = table(a[0], at::kFloat, l.m, e.size(1), d, "dweights must be contiguous fp32 of the experts' shape");
    c10::cuda::CUDAGuard guard(d);
    const Matrix o = result(nullptr, l.m, l.n, l.t.scalar_type(), d);
    const int experts = static_cast<int>(l.n < INT32_MAX ? l.n : INT32_MAX);
    status("expert_route_backward",
           layers.route_back(dw.data_ptr<float>(), l.t.data_ptr(), l.code, l.m, experts, l.ld, e.data_ptr<int32_t>(),
                             static_cast<int>(e.size(1)), small_integer(a[3]), truth(a[4]), real(a[5]),
                             o.t.data_ptr(), o.ld, stream_of(d)));
    return THPVariable_Wrap(o.t);
}

// (experts [tokens, k], number of experts): ExpertPlan(offsets, rows)
PyObject* f_plan(Args a) {
    const at::Tensor& e = tensor(a[0], "experts must be a contiguous int32 [tokens, k] CUDA tensor");
    if (!e.is_cuda() || e.scalar_type() != at::kInt || e.dim() != 2 || !e.is_contiguous() || e.size(1) < 1)
        value_error("experts must be a contiguous int32 [tokens, k] CUDA tensor");
    const at::Device d = e.device();
    const int experts = small_integer(a[1]);
    if (experts < 1) value_error("the number of experts must be positive");
    c10::cuda::CUDAGuard guard(d);
    const int64_t slots = e.numel();
    const size_t size = layers.plan_ws(slots, experts);
    c10::DataPtr ws;
    if (size > 0) ws = scratch(static_cast<int64_t>(size));
    const Two two = new_two({static_cast<int64_t>(experts) + 1}, e.sizes(), at::kInt, d);
    const at::Tensor &offsets = two.a, &rows = two.b;
    status("expert_plan", layers.plan(e.data_ptr<int32_t>(), slots, experts, offsets.data_ptr<int32_t>(), rows.data_ptr<int32_t>(),
                                      ws.get(), size, stream_of(d)));
    PyObject* args[2] = {THPVariable_Wrap(offsets), THPVariable_Wrap(rows)};
    PyObject* o = PyObject_Vectorcall(g_plan_class, args, 2, nullptr);
    Py_DECREF(args[0]);
    Py_DECREF(args[1]);
    if (o == nullptr) throw Raised{};
    return o;
}

struct Plan {
    at::Tensor rows, offsets;
    int64_t m, k;
    int experts;
};
Plan plan_of(PyObject* o, const at::Device& d) {
    if (Py_TYPE(o) != reinterpret_cast<PyTypeObject*>(g_plan_class)) value_error("plan must be an ExpertPlan");
    Plan r;
    PyObject* v = PyObject_GetAttr(o, n_plan_rows);
    if (v == nullptr) throw Raised{};
    const bool rows_ok = cuda_contiguous(v, at::kInt, d) && THPVariable_Unpack(v).dim() == 2;
    if (rows_ok) r.rows = THPVariable_Unpack(v);
    Py_DECREF(v);
    v = PyObject_GetAttr(o, n_plan_offsets);
    if (v == nullptr) throw Raised{};
    const bool offsets_ok = cuda_contiguous(v, at::kInt, d) && THPVariable_Unpack(v).dim() == 1 && THPVariable_Unpack(v).size(0) > 1;
    if (offsets_ok) r.offsets = THPVariable_Unpack(v);
    Py_DECREF(v);
    if (!rows_ok || !offsets_ok) value_error("the plan must be on the rows' device");
    r.m = r.rows.size(0);
    r.k = r.rows.size(1);
    r.experts = static_cast<int>(r.offsets.size(0) - 1);
    if (r.k > INT32_MAX) value_error("the plan has too many slots per token");
    return r;
}

// (x, plan, out): xs
PyObject* f_dispatch(Args a) {
    const Matrix x = matrix(a[0], "x must be a 2-D CUDA tensor");
    const at::Device d = x.t.device();
    const Plan p = plan_of(a[1], d);
    if (p.m != x.m) value_error("x must have the plan's tokens");
    c10::cuda::CUDAGuard guard(d);
    const Matrix o = result(a[2], p.m * p.k, x.n, x.t.scalar_type(), d);
    if (a[2] != Py_None) refuse_overlap(o, x, false, "out must be away from x");
    status("expert_dispatch", layers.dispatch(x.t.data_ptr(), x.code, x.m, x.n, x.ld, p.rows.data_ptr<int32_t>(), p.offsets.data_ptr<int32_t>(),
                                              p.experts, static_cast<int>(p.k), o.t.data_ptr(), o.ld, stream_of(d)));
    count_write(a[2], o);
    return THPVariable_Wrap(o.t);
}

// (ys, plan, weights, add, out): y
PyObject* f_combine(Args a) {
    const Matrix ys = matrix(a[0], "ys must be a 2-D CUDA tensor");
    const at::Device d = ys.t.device();
    const Plan p = plan_of(a[1], d);
    if (ys.m != p.m * p.k) value_error("ys must have a row for each of the plan's slots");
    const float* w = nullptr;
    if (a[2] != Py_None) w = table(a[2], at::kFloat, p.m, p.k, d, "weights must be contiguous fp32 of the plan's shape").data_ptr<float>();
    c10::cuda::CUDAGuard guard(d);
    Matrix add;
    if (a[3] != Py_None) {
        add = matrix(a[3], "add must be a matrix of the result's shape and type on its device", &d);
        if (add.m != p.m || add.n != ys.n || add.code != ys.code) value_error("add must be a matrix of the result's shape and type on its device");
    }
    const Matrix y = result(a[4], p.m, ys.n, ys.t.scalar_type(), d);
    if (a[4] != Py_None) {
        refuse_overlap(y, ys, false, "out must be away from ys");
        if (a[3] != Py_None) refuse_overlap(y, add, true, "out must be add or away from it");
    }
    status("expert_combine", layers.combine(ys.t.data_ptr(), ys.code, ys.ld, p.rows.data_ptr<int32_t>(), w,
                                            a[3] != Py_None ? add.t.data_ptr() : nullptr, a[3] != Py_None ? add.ld : 0, p.m, ys.n,
                                            static_cast<int>(p.k), y.t.data_ptr(), y.ld, stream_of(d)));
    count_write(a[4], y);
    return THPVariable_Wrap(y.t);
}

// (dy, ys, plan, weights): (dys, dweights)
PyObject* f_combine_backward(Args a) {
    const Matrix ys = matrix(a[1], "ys must be a 2-D CUDA tensor");
    const at::Device d = ys.t.device();
    c10::cuda::CUDAGuard guard(d);
    const Plan p = plan_of(a[2], d);
    const Matrix dy = matrix(a[0], "dy must be a matrix of the result's shape and type on its device", &d);
    if (ys.m != p.m * p.k) value_error("ys must have a row for each of the plan's slots");
    if (dy.m != p.m || dy.n != ys.n || dy.code != ys.code) value_error("dy must be a matrix of the result's shape and type on its device");
    const at::Tensor& w = table(a[3], at::kFloat, p.m, p.k, d, "weights must be contiguous fp32 of the plan's shape");
    const Matrix dys = result(nullptr, ys.m, ys.n, ys.t.scalar_type(), d);
    at::Tensor dw = new_tensor({p.m, p.k}, at::kFloat, d);
    status("expert_combine_backward",
           layers.combine_back(dy.t.data_ptr(), dy.code, dy.ld, ys.t.data_ptr(), ys.ld, p.rows.data_ptr<int32_t>(),
                               p.offsets.data_ptr<int32_t>(), p.experts, w.data_ptr<float>(), p.m, ys.n, static_cast<int>(p.k),
                               dys.t.data_ptr(), dys.ld, dw.data_ptr<float>(), stream_of(d)));
    return pair(THPVariable_Wrap(dys.t), THPVariable_Wrap(dw));
}
