// ew_torch.cpp -- the row operators' torch binding: argument checks, output
// allocation and the calls into libew.so, as a CPython extension.
//
// Small calls are bound by the host.  On a GB300's Arm cores a Python-level
// torch.empty takes 1.4 us and a foreign call with its 20 arguments 1.2 us;
// the 8-bit norm of 7 rows came to 19 us from Python through ctypes, 2.4 us of
// which are the kernel's.  rows.py holds the signatures and documentation and
// hands over to these functions, which take all arguments in order.
//
// Errors: ValueError and TypeError for what does not fit, and for the
// library's own status the callable given to set_check.
#include <array>
#include <cstdint>

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ew.h"

namespace {

using at::Tensor;

// A Python exception is set; ends the call.
struct Raised {};
#define REFUSE(type, ...)                  \
    do {                                   \
        PyErr_Format(type, __VA_ARGS__);   \
        throw Raised{};                    \
    } while (0)

PyObject *g_check = nullptr;  // check(status, name): raises the library's error

void check_status(ew_status status, const char *name) {
    if (status == EW_OK) return;
    PyObject *r = PyObject_CallFunction(g_check, "is", static_cast<int>(status), name);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", name, static_cast<int>(status));
    throw Raised{};
}

const Tensor &tensor(PyObject *o, const char *what) {
    if (!THPVariable_Check(o)) REFUSE(PyExc_TypeError, "%s: expected a tensor, got %s", what, Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}
int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

struct Device {
    c10::DeviceIndex index;
    // From the caching allocator without a way through the dispatcher, which takes 0.7 us a
    // tensor: a layer norm's call with its four outputs 6.0 us of host time, 8.4 by at::empty.
    Tensor empty(at::IntArrayRef sizes, at::ScalarType t) const {
        return at::detail::empty_cuda(sizes, t, c10::Device(c10::kCUDA, index), std::nullopt);
    }
    ew_stream_t stream() const {
        return reinterpret_cast<ew_stream_t>(c10::cuda::getCurrentCUDAStream(index).stream());
    }
};
Device device_of(const Tensor &t, const char *what) {
    if (!t.is_cuda()) REFUSE(PyExc_ValueError, "%s must be on a CUDA device", what);
    const Device d{t.get_device()};
    if (d.index != c10::cuda::current_device()) REFUSE(PyExc_ValueError, "%s must be on the current device", what);
    return d;
}
void check_device(const Tensor &t, const char *what, Device d) {
    if (!t.is_cuda() || t.get_device() != d.index)
        REFUSE(PyExc_ValueError, "%s must be on cuda:%d", what, static_cast<int>(d.index));
}

ew_dtype code_of(const Tensor &t, const char *what) {
    switch (t.scalar_type()) {
        case at::kFloat: return EW_F32;
        case at::kHalf: return EW_F16;
        case at::kBFloat16: return EW_BF16;
        default: REFUSE(PyExc_TypeError, "%s: unsupported dtype %s (float32, float16, bfloat16)", what, c10::toString(t.scalar_type()));
    }
}
ew_index index_of(const Tensor &t, const char *what) {
    if (t.scalar_type() == at::kInt) return EW_INDEX_I32;
    if (t.scalar_type() == at::kLong) return EW_INDEX_I64;
    REFUSE(PyExc_TypeError, "%s: int32 or int64, got %s", what, c10::toString(t.scalar_type()));
}

// A tensor as a matrix of its last dimension.
struct Matrix {
    void *p;
    int64_t rows, cols, stride;
};
Matrix matrix(const Tensor &t, const char *what, Device d) {
    check_device(t, what, d);
    const auto sizes = t.sizes();
    if (sizes.size() == 2) {
        const int64_t rows = sizes[0], cols = sizes[1], stride = t.stride(0), inner = t.stride(1);
        if (inner == 1 || cols <= 1) {
            if (stride >= cols && stride > 0) return {t.data_ptr(), rows, cols, stride};
            if (rows <= 1) return {t.data_ptr(), rows, cols, cols};  // the stride of a single row says nothing
        }
    } else if (!sizes.empty() && t.is_contiguous()) {
        const int64_t cols = sizes.back();
        return {t.data_ptr(), cols ? t.numel() / cols : 0, cols, cols};
    }
    REFUSE(PyExc_ValueError, "%s: a matrix needs a contiguous last dimension and rows that do not overlap", what);
}
Matrix matrix_like(const Tensor &t, const char *what, int64_t rows, int64_t cols, at::ScalarType type, Device d) {
    const Matrix m = matrix(t, what, d);
    if (m.rows != rows || m.cols != cols || t.scalar_type() != type)
        REFUSE(PyExc_ValueError, "%s: expected %lld x %lld of %s, got %lld x %lld of %s", what, static_cast<long long>(rows),
               static_cast<long long>(cols), c10::toString(type), static_cast<long long>(m.rows),
               static_cast<long long>(m.cols), c10::toString(t.scalar_type()));
    return m;
}
void *vector(const Tensor &t, const char *what, int64_t n, at::ScalarType type, Device d) {
    if (!t.is_cuda() || t.get_device() != d.index || t.scalar_type() != type || t.numel() != n || !t.is_contiguous())
        REFUSE(PyExc_ValueError, "%s: expected %lld contiguous elements of %s on cuda:%d", what, static_cast<long long>(n),
               c10::toString(type), static_cast<int>(d.index));
    return t.data_ptr();
}
float *floats(PyObject *o, const char *what, int64_t n, Device d) {
    return static_cast<float *>(vector(tensor(o, what), what, n, at::kFloat, d));
}
// A vector of ids.
struct Ids {
    ew_index type;
    const void *p;
};
Ids ids_of(PyObject *o, const char *what, int64_t n, Device d) {
    const Tensor &t = tensor(o, what);
    const ew_index type = index_of(t, what);
    return {type, vector(t, what, n, t.scalar_type(), d)};
}

// An output: the given tensor or a new one, and the Python object to return.
struct Output {
    PyObject *o = nullptr;
    Output() = default;
    Output(const Output &) = delete;
    Output &operator=(const Output &) = delete;
    ~Output() { Py_XDECREF(o); }
    void give(PyObject *given) {
        Py_INCREF(given);
        o = given;
    }
    void *make(at::IntArrayRef sizes, at::ScalarType type, Device d) {
        Tensor t = d.empty(sizes, type);
        void *p = t.data_ptr();
        o = THPVariable_Wrap(std::move(t));
        if (o == nullptr) throw Raised{};
        return p;
    }
    // rows x cols: the given one, or a new one of these sizes
    Matrix matrix(PyObject *given, const char *what, at::IntArrayRef sizes, int64_t rows, int64_t cols, at::ScalarType type,
                  Device d) {
        if (given != Py_None) {
            give(given);
            return matrix_like(tensor(given, what), what, rows, cols, type, d);
        }
        return {make(sizes, type, d), rows, cols, cols};
    }
    float *floats(PyObject *given, const char *what, int64_t n, Device d) {
        if (given != Py_None) {
            give(given);
            return static_cast<float *>(vector(tensor(given, what), what, n, at::kFloat, d));
        }
        return static_cast<float *>(make({n}, at::kFloat, d));
    }
    PyObject *take() {
        PyObject *r = o;
        o = nullptr;
        return r;
    }
};
template <typename... O> PyObject *tuple_of(O &...outs) {
    PyObject *t = PyTuple_New(sizeof...(O));
    if (t == nullptr) throw Raised{};
    Py_ssize_t i = 0;
    ((PyTuple_SET_ITEM(t, i++, outs.take())), ...);
    return t;
}

// A workspace: lives to the end of the call, on the call's stream.
struct Workspace {
    Tensor t;
    int64_t bytes;
    Workspace(int64_t need, const char *what, Device d) : bytes(need) {
        if (need < 0) REFUSE(PyExc_ValueError, "%s: sizes out of range", what);
        if (need > 0) t = d.empty({need}, at::kByte);
    }
    void *p() const { return t.defined() ? t.data_ptr() : nullptr; }
};

// ---------------------------------------------------------------- embedding

PyObject *embed(PyObject *const *a) {  // table, tokens, out, scale
    const Tensor &table = tensor(a[0], "table"), &tokens = tensor(a[1], "tokens");
    const Device d = device_of(table, "table");
    const ew_dtype code = code_of(table, "table");
    const Matrix m = matrix(table, "table", d);
    const int64_t rows = tokens.numel();
    const Ids ids = ids_of(a[1], "tokens", rows, d);
    const float scale = static_cast<float>(number(a[3]));
    c10::SmallVector<int64_t, 4> sizes(tokens.sizes().begin(), tokens.sizes().end());
    sizes.push_back(m.cols);
    Output out;
    const Matrix o = out.matrix(a[2], "out", sizes, rows, m.cols, table.scalar_type(), d);
    check_status(ew_embed(code, ids.type, m.p, m.rows, m.stride, ids.p, scale, o.p, o.stride, rows, m.cols, d.stream()),
                 "ew_embed");
    return out.take();
}

PyObject *embed_grad(PyObject *const *a) {  // dout, tokens, table_rows, dtable, scale, accumulate
    const Tensor &dout = tensor(a[0], "dout");
    const Device d = device_of(dout, "dout");
    const ew_dtype code = code_of(dout, "dout");
    const Matrix m = matrix(dout, "dout", d);
    const Ids ids = ids_of(a[1], "tokens", m.rows, d);
    const int64_t table_rows = integer(a[2]);
    const float scale = static_cast<float>(number(a[4]));
    const int accumulate = PyObject_IsTrue(a[5]);
    if (accumulate < 0) throw Raised{};
    at::ScalarType type = dout.scalar_type();
    if (a[3] != Py_None) {
        const at::ScalarType given = tensor(a[3], "dtable").scalar_type();
        if (given != type && given != at::kFloat)
            REFUSE(PyExc_TypeError, "dtable: %s or float32, got %s", c10::toString(type), c10::toString(given));
        type = given;
    } else if (accumulate) {
        REFUSE(PyExc_ValueError, "accumulate needs a dtable to add to");
    }
    const Workspace work(ew_embed_grad_workspace(table_rows, m.rows, m.cols), "ew_embed_grad", d);
    Output out;
    const Matrix o = out.matrix(a[3], "dtable", {table_rows, m.cols}, table_rows, m.cols, type, d);
    check_status(ew_embed_grad(code, ids.type, m.p, m.stride, ids.p, scale, type == at::kFloat ? EW_F32 : code, o.p,
                               table_rows, o.stride, m.rows, m.cols, accumulate, work.p(), work.bytes, d.stream()),
                 "ew_embed_grad");
    return out.take();
}

// ---------------------------------------------------------------- norm

struct Weight {
    ew_dtype type;
    const void *p;
};
Weight weight_of(PyObject *o, int64_t cols, ew_dtype code, at::ScalarType type, Device d, const char *what = "weight") {
    if (o == Py_None) return {code, nullptr};
    const Tensor &w = tensor(o, what);
    if (w.scalar_type() != type && w.scalar_type() != at::kFloat)
        REFUSE(PyExc_TypeError, "%s: %s or float32, got %s", what, c10::toString(type), c10::toString(w.scalar_type()));
    return {w.scalar_type() == type ? code : EW_F32, vector(w, what, cols, w.scalar_type(), d)};
}

// What the norm calls take (x, weight, residual, eps), and their outputs h and rstd.
struct NormCall {
    const Tensor &x;
    Device d;
    ew_dtype code;
    at::ScalarType type;
    Matrix m, residual{nullptr, 0, 0, 0}, hm{nullptr, 0, 0, 0};
    Weight w;
    float eps;
    float *rstd_p;
    Output h, rstd;
    // `y_given`: an output that may be x
    NormCall(PyObject *const *a, PyObject *y_given, PyObject *h_given, PyObject *rstd_given)
        : x(tensor(a[0], "x")), d(device_of(x, "x")), code(code_of(x, "x")), type(x.scalar_type()), m(matrix(x, "x", d)),
          w(weight_of(a[1], m.cols, code, type, d)), eps(static_cast<float>(number(a[3]))) {
        if (a[2] != Py_None) residual = matrix_like(tensor(a[2], "residual"), "residual", m.rows, m.cols, type, d);
        // without a residual h is x: nothing to write, unless y takes its place
        const bool over = y_given != Py_None && m.p != nullptr && tensor(y_given, "y").data_ptr() == m.p;
        if (a[2] == Py_None && h_given == Py_None && !over) h.give(a[0]);
        else hm = h.matrix(h_given, "h", x.sizes(), m.rows, m.cols, type, d);
        rstd_p = rstd.floats(rstd_given, "rstd", m.rows, d);
    }
};

PyObject *rmsnorm(PyObject *const *a) {  // x, weight, residual, eps, y, h, rstd
    NormCall c(a, a[4], a[5], a[6]);
    Output y;
    const Matrix o = y.matrix(a[4], "y", c.x.sizes(), c.m.rows, c.m.cols, c.type, c.d);
    check_status(ew_rmsnorm(c.code, c.m.p, c.m.stride, c.residual.p, c.residual.stride, c.w.type, c.w.p, c.eps, o.p, o.stride,
                            c.hm.p, c.hm.stride, c.rstd_p, c.m.rows, c.m.cols, c.d.stream()),
                 "ew_rmsnorm");
    return tuple_of(y, c.h, c.rstd);
}

PyObject *rmsnorm_quant(PyObject *const *a) {  // x, weight, residual, eps, group, q, scales, h, rstd, int8
    NormCall c(a, Py_None, a[7], a[8]);
    const int64_t group = integer(a[4]);
    const bool i8 = a[9] == Py_True;
    // a group that the library refuses gets any size here
    const int64_t groups = group > 0 ? (c.m.cols + group - 1) / group : 1;
    Output q, scales;
    const Matrix o = q.matrix(a[5], "q", c.x.sizes(), c.m.rows, c.m.cols, i8 ? at::kChar : at::kFloat8_e4m3fn, c.d);
    const Matrix s = scales.matrix(a[6], "scales", {c.m.rows, groups}, c.m.rows, groups, at::kFloat, c.d);
    check_status(ew_rmsnorm_quant(c.code, c.m.p, c.m.stride, c.residual.p, c.residual.stride, c.w.type, c.w.p, c.eps,
                                  i8 ? EW_Q_I8 : EW_Q_E4M3, group, o.p, o.stride, static_cast<float *>(s.p), s.stride,
                                  c.hm.p, c.hm.stride, c.rstd_p, c.m.rows, c.m.cols, c.d.stream()),
                 "ew_rmsnorm_quant");
    return tuple_of(q, scales, c.h, c.rstd);
}

PyObject *rmsnorm_grad(PyObject *const *a) {  // dy, h, weight, rstd, dh, dx, dweight
    const Tensor &dy = tensor(a[0], "dy");
    const Device d = device_of(dy, "dy");
    const ew_dtype code = code_of(dy, "dy");
    const at::ScalarType type = dy.scalar_type();
    const Matrix m = matrix(dy, "dy", d), h = matrix_like(tensor(a[1], "h"), "h", m.rows, m.cols, type, d);
    const Weight w = weight_of(a[2], m.cols, code, type, d);
    const float *rstd = floats(a[3], "rstd", m.rows, d);
    Matrix dh{nullptr, 0, 0, 0};
    if (a[4] != Py_None) dh = matrix_like(tensor(a[4], "dh"), "dh", m.rows, m.cols, type, d);
    const Workspace work(ew_rmsnorm_grad_workspace(m.rows, m.cols), "ew_rmsnorm_grad", d);
    Output dx, dweight;
    const Matrix o = dx.matrix(a[5], "dx", dy.sizes(), m.rows, m.cols, type, d);
    float *dw = dweight.floats(a[6], "dweight", m.cols, d);
    check_status(ew_rmsnorm_grad(code, m.p, m.stride, h.p, h.stride, w.type, w.p, rstd, dh.p, dh.stride, o.p, o.stride, dw,
                                 m.rows, m.cols, work.p(), work.bytes, d.stream()),
                 "ew_rmsnorm_grad");
    return tuple_of(dx, dweight);
}

PyObject *layernorm(PyObject *const *a) {  // x, weight, residual, eps, bias, y, h, mean, rstd
    NormCall c(a, a[5], a[6], a[8]);
    const Weight b = weight_of(a[4], c.m.cols, c.code, c.type, c.d, "bias");
    if (c.w.p != nullptr && b.p != nullptr && c.w.type != b.type) REFUSE(PyExc_TypeError, "weight and bias: one dtype");
    Output y, mean;
    const Matrix o = y.matrix(a[5], "y", c.x.sizes(), c.m.rows, c.m.cols, c.type, c.d);
    float *mean_p = mean.floats(a[7], "mean", c.m.rows, c.d);
    check_status(ew_layernorm(c.code, c.m.p, c.m.stride, c.residual.p, c.residual.stride, c.w.p != nullptr ? c.w.type : b.type,
                              c.w.p, b.p, c.eps, o.p, o.stride, c.hm.p, c.hm.stride, mean_p, c.rstd_p, c.m.rows, c.m.cols,
                              c.d.stream()),
                 "ew_layernorm");
    return tuple_of(y, c.h, mean, c.rstd);
}

PyObject *layernorm_grad(PyObject *const *a) {  // dy, h, weight, mean, rstd, dh, dx, dweight, dbias
    const Tensor &dy = tensor(a[0], "dy");
    const Device d = device_of(dy, "dy");
    const ew_dtype code = code_of(dy, "dy");
    const at::ScalarType type = dy.scalar_type();
    const Matrix m = matrix(dy, "dy", d), h = matrix_like(tensor(a[1], "h"), "h", m.rows, m.cols, type, d);
    const Weight w = weight_of(a[2], m.cols, code, type, d);
    const float *mean = floats(a[3], "mean", m.rows, d), *rstd = floats(a[4], "rstd", m.rows, d);
    Matrix dh{nullptr, 0, 0, 0};
    if (a[5] != Py_None) dh = matrix_like(tensor(a[5], "dh"), "dh", m.rows, m.cols, type, d);
    const Workspace work(ew_layernorm_grad_workspace(m.rows, m.cols), "ew_layernorm_grad", d);
    Output dx, dweight, dbias;
    const Matrix o = dx.matrix(a[6], "dx", dy.sizes(), m.rows, m.cols, type, d);
    float *dw = dweight.floats(a[7], "dweight", m.cols, d), *db = dbias.floats(a[8], "dbias", m.cols, d);
    check_status(ew_layernorm_grad(code, m.p, m.stride, h.p, h.stride, w.type, w.p, mean, rstd, dh.p, dh.stride, o.p, o.stride,
                                   dw, db, m.rows, m.cols, work.p(), work.bytes, d.stream()),
                 "ew_layernorm_grad");
    return tuple_of(dx, dweight, dbias);
}

// ---------------------------------------------------------------- experts

PyObject *expert_sort(PyObject *const *a) {  // experts, n_experts, align
    const Tensor &experts = tensor(a[0], "experts");
    const Device d = device_of(experts, "experts");
    const ew_index type = index_of(experts, "experts");
    const Matrix m = matrix(experts, "experts", d);
    const int64_t n_experts = integer(a[1]), align = integer(a[2]);
    const int64_t capacity = ew_expert_capacity(m.rows, m.cols, n_experts, align);
    const int64_t need = ew_expert_sort_workspace(m.rows, m.cols, n_experts);
    if (capacity < 0 || need < 0) check_status(EW_ERR_INVALID_VALUE, "ew_expert_sort");
    const Workspace work(need, "ew_expert_sort", d);
    Output positions, offsets, counts, slots;
    auto make = [&](Output &o, at::IntArrayRef sizes) { return static_cast<int32_t *>(o.make(sizes, at::kInt, d)); };
    int32_t *p = make(positions, {m.rows, m.cols}), *o = make(offsets, {n_experts + 1}), *c = make(counts, {n_experts});
    int32_t *s = make(slots, {capacity});
    check_status(ew_expert_sort(type, m.p, m.stride, n_experts, align, p, o, c, s, capacity, m.rows, m.cols, work.p(),
                                work.bytes, d.stream()),
                 "ew_expert_sort");
    return tuple_of(positions, offsets, counts, slots);
}

// What the calls take of a sort: positions (rows x k) and slots.
struct Plan {
    const int32_t *positions, *slots;
    int64_t rows, k, capacity;
    Plan(PyObject *o, Device d) {
        if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) REFUSE(PyExc_TypeError, "plan: what ew_expert_sort returns");
        const Tensor &p = tensor(PyTuple_GET_ITEM(o, 0), "positions"), &s = tensor(PyTuple_GET_ITEM(o, 3), "slots");
        if (p.dim() != 2) REFUSE(PyExc_ValueError, "positions: expected tokens x experts");
        rows = p.size(0);
        k = p.size(1);
        capacity = s.numel();
        positions = static_cast<const int32_t *>(vector(p, "positions", rows * k, at::kInt, d));
        slots = static_cast<const int32_t *>(vector(s, "slots", capacity, at::kInt, d));
    }
};
// A number for each slot: in the tokens' order, as tokens x k or flat.  Of as many
// elements in other shapes, such as k x tokens, the order would be another.
void check_slots(PyObject *o, const char *what, const Plan &plan) {
    if (o == Py_None || plan.k == 1) return;
    int64_t dims = 0, last = 1;  // of those above 1
    for (int64_t size : tensor(o, what).sizes())
        if (size != 1) ++dims, last = size;
    if (dims > 1 && last != plan.k)
        REFUSE(PyExc_ValueError, "%s: expected %lld x %lld", what, static_cast<long long>(plan.rows), static_cast<long long>(plan.k));
}
Weight weights_of(PyObject *o, const Plan &plan, ew_dtype code, at::ScalarType type, Device d) {
    check_slots(o, "weights", plan);
    return weight_of(o, plan.rows * plan.k, code, type, d, "weights");
}

PyObject *expert_dispatch(PyObject *const *a) {  // x, plan, out
    const Tensor &x = tensor(a[0], "x");
    const Device d = device_of(x, "x");
    const ew_dtype code = code_of(x, "x");
    const Matrix m = matrix(x, "x", d);
    const Plan plan(a[1], d);
    if (m.rows != plan.rows)
        REFUSE(PyExc_ValueError, "x: expected %lld rows, got %lld", static_cast<long long>(plan.rows), static_cast<long long>(m.rows));
    Output out;
    const Matrix o = out.matrix(a[2], "out", {plan.capacity, m.cols}, plan.capacity, m.cols, x.scalar_type(), d);
    check_status(ew_expert_dispatch(code, m.p, m.stride, plan.positions, plan.slots, o.p, o.stride, plan.capacity, plan.rows,
                                    plan.k, m.cols, d.stream()),
                 "ew_expert_dispatch");
    return out.take();
}

PyObject *expert_combine(PyObject *const *a) {  // y, plan, weights, residual, out
    const Tensor &y = tensor(a[0], "y");
    const Device d = device_of(y, "y");
    const ew_dtype code = code_of(y, "y");
    const at::ScalarType type = y.scalar_type();
    const Plan plan(a[1], d);
    const Matrix m = matrix(y, "y", d);
    if (m.rows != plan.capacity)
        REFUSE(PyExc_ValueError, "y: expected %lld rows, got %lld", static_cast<long long>(plan.capacity), static_cast<long long>(m.rows));
    const Weight w = weights_of(a[2], plan, code, type, d);
    Matrix residual{nullptr, 0, 0, 0};
    if (a[3] != Py_None) residual = matrix_like(tensor(a[3], "residual"), "residual", plan.rows, m.cols, type, d);
    Output out;
    const Matrix o = out.matrix(a[4], "out", {plan.rows, m.cols}, plan.rows, m.cols, type, d);
    check_status(ew_expert_combine(code, m.p, m.stride, plan.capacity, plan.positions, w.type, w.p, residual.p, residual.stride,
                                   o.p, o.stride, plan.rows, plan.k, m.cols, d.stream()),
                 "ew_expert_combine");
    return out.take();
}

PyObject *expert_combine_grad(PyObject *const *a) {  // dout, y, plan, weights, dy, dweights
    const Tensor &dout = tensor(a[0], "dout");
    const Device d = device_of(dout, "dout");
    const ew_dtype code = code_of(dout, "dout");
    const at::ScalarType type = dout.scalar_type();
    const Plan plan(a[2], d);
    const Matrix m = matrix(dout, "dout", d);
    if (m.rows != plan.rows)
        REFUSE(PyExc_ValueError, "dout: expected %lld rows, got %lld", static_cast<long long>(plan.rows), static_cast<long long>(m.rows));
    const Matrix y = matrix_like(tensor(a[1], "y"), "y", plan.capacity, m.cols, type, d);
    const Weight w = weights_of(a[3], plan, code, type, d);
    Output dy, dweights;
    const Matrix o = dy.matrix(a[4], "dy", {plan.capacity, m.cols}, plan.capacity, m.cols, type, d);
    float *dw;
    if (a[5] != Py_None) {
        check_slots(a[5], "dweights", plan);
        dw = dweights.floats(a[5], "dweights", plan.rows * plan.k, d);
    } else {
        dw = static_cast<float *>(dweights.make({plan.rows, plan.k}, at::kFloat, d));
    }
    check_status(ew_expert_combine_grad(code, m.p, m.stride, y.p, y.stride, plan.capacity, plan.positions, plan.slots, w.type,
                                        w.p, o.p, o.stride, dw, plan.rows, plan.k, m.cols, d.stream()),
                 "ew_expert_combine_grad");
    return tuple_of(dy, dweights);
}

// ---------------------------------------------------------------- logits

PyObject *logprob(PyObject *const *a) {  // logits, tokens, top, scale
    const Tensor &logits = tensor(a[0], "logits");
    const Device d = device_of(logits, "logits");
    const ew_dtype code = code_of(logits, "logits");
    const Matrix m = matrix(logits, "logits", d);
    const int64_t top = integer(a[2]);
    const float scale = static_cast<float>(number(a[3]));
    if (top < 0 || top > 64) check_status(EW_ERR_INVALID_VALUE, "ew_logprob");  // before sizes are made of it
    Ids ids{EW_INDEX_I32, nullptr};
    Output logp, entropy, lse, top_logp, top_ids;
    float *logp_p = nullptr;
    if (a[1] != Py_None) {
        ids = ids_of(a[1], "tokens", m.rows, d);
        logp_p = logp.floats(Py_None, "logp", m.rows, d);
    } else {
        logp.give(Py_None);
    }
    float *entropy_p = entropy.floats(Py_None, "entropy", m.rows, d), *lse_p = lse.floats(Py_None, "lse", m.rows, d);
    float *top_logp_p = static_cast<float *>(top_logp.make({m.rows, top}, at::kFloat, d));
    int32_t *top_ids_p = static_cast<int32_t *>(top_ids.make({m.rows, top}, at::kInt, d));
    check_status(ew_logprob(code, ids.type, m.p, m.stride, ids.p, scale, top, logp_p, entropy_p, lse_p, top_logp_p, top_ids_p,
                            m.rows, m.cols, d.stream()),
                 "ew_logprob");
    return tuple_of(logp, entropy, lse, top_logp, top_ids);
}

PyObject *logprob_grad(PyObject *const *a) {  // logits, tokens, lse, entropy, dlogp, dentropy, scale, dlogits
    const Tensor &logits = tensor(a[0], "logits");
    const Device d = device_of(logits, "logits");
    const ew_dtype code = code_of(logits, "logits");
    const Matrix m = matrix(logits, "logits", d);
    const float scale = static_cast<float>(number(a[6]));
    Ids ids{EW_INDEX_I32, nullptr};
    const float *dlogp = nullptr, *entropy = nullptr, *dentropy = nullptr;
    if (a[4] != Py_None) {
        ids = ids_of(a[1], "tokens", m.rows, d);
        dlogp = floats(a[4], "dlogp", m.rows, d);
    }
    const float *lse = floats(a[2], "lse", m.rows, d);
    if (a[5] != Py_None) {
        entropy = floats(a[3], "entropy", m.rows, d);
        dentropy = floats(a[5], "dentropy", m.rows, d);
    }
    Output out;
    const Matrix o = out.matrix(a[7], "dlogits", logits.sizes(), m.rows, m.cols, logits.scalar_type(), d);
    check_status(ew_logprob_grad(code, ids.type, m.p, m.stride, ids.p, lse, entropy, dlogp, dentropy, scale, o.p, o.stride,
                                 m.rows, m.cols, d.stream()),
                 "ew_logprob_grad");
    return out.take();
}

// What the three distillation calls take: logits, ids, teacher.
struct DistillCall {
    const Tensor &logits, &id_tensor, &teacher;
    Device d;
    ew_dtype code, teacher_code;
    ew_index index;
    Matrix m, ids, t;
    explicit DistillCall(PyObject *const *a)
        : logits(tensor(a[0], "logits")), id_tensor(tensor(a[1], "ids")), teacher(tensor(a[2], "teacher")),
          d(device_of(logits, "logits")), code(code_of(logits, "logits")), index(index_of(id_tensor, "ids")) {
        if (teacher.scalar_type() != logits.scalar_type() && teacher.scalar_type() != at::kFloat)
            REFUSE(PyExc_TypeError, "teacher: %s or float32, got %s", c10::toString(logits.scalar_type()),
                   c10::toString(teacher.scalar_type()));
        teacher_code = teacher.scalar_type() == logits.scalar_type() ? code : EW_F32;
        m = matrix(logits, "logits", d);
        ids = matrix(id_tensor, "ids", d);
        if (ids.rows != m.rows)
            REFUSE(PyExc_ValueError, "ids: expected %lld rows, got %lld", static_cast<long long>(m.rows),
                   static_cast<long long>(ids.rows));
        t = matrix_like(teacher, "teacher", m.rows, ids.cols, teacher.scalar_type(), d);
    }
};

PyObject *distill(PyObject *const *a) {  // logits, ids, teacher, scale
    const DistillCall c(a);
    const float scale = static_cast<float>(number(a[3]));
    Output loss, lse;
    float *loss_p = loss.floats(Py_None, "loss", c.m.rows, c.d), *lse_p = lse.floats(Py_None, "lse", c.m.rows, c.d);
    check_status(ew_distill(c.code, c.index, c.m.p, c.m.stride, c.ids.p, c.ids.stride, c.teacher_code, c.t.p, c.t.stride,
                            c.ids.cols, scale, loss_p, lse_p, c.m.rows, c.m.cols, c.d.stream()),
                 "ew_distill");
    return tuple_of(loss, lse);
}

PyObject *distill_grad(PyObject *const *a) {  // logits, ids, teacher, lse, dloss, scale, dlogits
    const DistillCall c(a);
    const float *lse = floats(a[3], "lse", c.m.rows, c.d), *dloss = floats(a[4], "dloss", c.m.rows, c.d);
    const float scale = static_cast<float>(number(a[5]));
    Output out;
    const Matrix o = out.matrix(a[6], "dlogits", c.logits.sizes(), c.m.rows, c.m.cols, c.logits.scalar_type(), c.d);
    check_status(ew_distill_grad(c.code, c.index, c.m.p, c.m.stride, c.ids.p, c.ids.stride, c.teacher_code, c.t.p,
                                 c.t.stride, c.ids.cols, scale, lse, dloss, o.p, o.stride, c.m.rows, c.m.cols, c.d.stream()),
                 "ew_distill_grad");
    return out.take();
}

PyObject *distill_step(PyObject *const *a) {  // logits, ids, teacher, dloss, scale, dlogits
    const DistillCall c(a);
    const float *dloss = floats(a[3], "dloss", c.m.rows, c.d);
    const float scale = static_cast<float>(number(a[4]));
    Output loss, lse, out;
    const Matrix o = out.matrix(a[5], "dlogits", c.logits.sizes(), c.m.rows, c.m.cols, c.logits.scalar_type(), c.d);
    float *loss_p = loss.floats(Py_None, "loss", c.m.rows, c.d), *lse_p = lse.floats(Py_None, "lse", c.m.rows, c.d);
    check_status(ew_distill_step(c.code, c.index, c.m.p, c.m.stride, c.ids.p, c.ids.stride, c.teacher_code, c.t.p,
                                 c.t.stride, c.ids.cols, scale, dloss, loss_p, lse_p, o.p, o.stride, c.m.rows, c.m.cols,
                                 c.d.stream()),
                 "ew_distill_step");
    return tuple_of(loss, lse, out);
}

// What the three calls of the policy loss take: logits, tokens, advantage, old_logp, ref_logp, clip_low, clip_high, kl, scale.
struct PolicyCall {
    const Tensor &logits;
    Device d;
    ew_dtype code;
    Matrix m;
    Ids tokens;
    const float *advantage, *old_logp = nullptr, *ref_logp = nullptr;
    float clip_low, clip_high, kl, scale;
    explicit PolicyCall(PyObject *const *a)
        : logits(tensor(a[0], "logits")), d(device_of(logits, "logits")), code(code_of(logits, "logits")),
          m(matrix(logits, "logits", d)), tokens(ids_of(a[1], "tokens", m.rows, d)),
          advantage(floats(a[2], "advantage", m.rows, d)), clip_low(static_cast<float>(number(a[5]))),
          clip_high(static_cast<float>(number(a[6]))), kl(static_cast<float>(number(a[7]))),
          scale(static_cast<float>(number(a[8]))) {
        if (a[3] != Py_None) old_logp = floats(a[3], "old_logp", m.rows, d);
        if (a[4] != Py_None) ref_logp = floats(a[4], "ref_logp", m.rows, d);
    }
};

// loss, logp and lse, new ones
std::array<float *, 3> policy_rows(Output &loss, Output &logp, Output &lse, const PolicyCall &c) {
    auto make = [&](Output &o, const char *what) { return o.floats(Py_None, what, c.m.rows, c.d); };
    float *loss_p = make(loss, "loss"), *logp_p = make(logp, "logp");
    return {loss_p, logp_p, make(lse, "lse")};
}

PyObject *policy(PyObject *const *a) {  // what PolicyCall takes
    const PolicyCall c(a);
    Output loss, logp, lse;
    const auto [loss_p, logp_p, lse_p] = policy_rows(loss, logp, lse, c);
    check_status(ew_policy(c.code, c.tokens.type, c.m.p, c.m.stride, c.tokens.p, c.advantage, c.old_logp, c.ref_logp, c.clip_low,
                           c.clip_high, c.kl, c.scale, loss_p, logp_p, lse_p, c.m.rows, c.m.cols, c.d.stream()),
                 "ew_policy");
    return tuple_of(loss, logp, lse);
}

PyObject *policy_grad(PyObject *const *a) {  // what PolicyCall takes, logp, lse, dloss, dlogits
    const PolicyCall c(a);
    const float *logp = floats(a[9], "logp", c.m.rows, c.d), *lse = floats(a[10], "lse", c.m.rows, c.d);
    const float *dloss = floats(a[11], "dloss", c.m.rows, c.d);
    Output out;
    const Matrix o = out.matrix(a[12], "dlogits", c.logits.sizes(), c.m.rows, c.m.cols, c.logits.scalar_type(), c.d);
    check_status(ew_policy_grad(c.code, c.tokens.type, c.m.p, c.m.stride, c.tokens.p, c.advantage, c.old_logp, c.ref_logp,
                                c.clip_low, c.clip_high, c.kl, c.scale, logp, lse, dloss, o.p, o.stride, c.m.rows, c.m.cols,
                                c.d.stream()),
                 "ew_policy_grad");
    return out.take();
}

PyObject *policy_step(PyObject *const *a) {  // what PolicyCall takes, dloss, dlogits
    const PolicyCall c(a);
    const float *dloss = floats(a[9], "dloss", c.m.rows, c.d);
    Output loss, logp, lse, out;
    const Matrix o = out.matrix(a[10], "dlogits", c.logits.sizes(), c.m.rows, c.m.cols, c.logits.scalar_type(), c.d);
    const auto [loss_p, logp_p, lse_p] = policy_rows(loss, logp, lse, c);
    check_status(ew_policy_step(c.code, c.tokens.type, c.m.p, c.m.stride, c.tokens.p, c.advantage, c.old_logp, c.ref_logp,
                                c.clip_low, c.clip_high, c.kl, c.scale, dloss, loss_p, logp_p, lse_p, o.p, o.stride, c.m.rows,
                                c.m.cols, c.d.stream()),
                 "ew_policy_step");
    return tuple_of(loss, logp, lse, out);
}

// ---------------------------------------------------------------- module

// A function of N positional arguments; C++ exceptions become Python's.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *set_check(PyObject *, PyObject *fn) {
    Py_INCREF(fn);
    Py_XDECREF(g_check);
    g_check = fn;
    Py_RETURN_NONE;
}

#define ENTRY(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<name, n>)), METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {
    ENTRY(embed, 4), ENTRY(embed_grad, 6), ENTRY(rmsnorm, 7), ENTRY(rmsnorm_quant, 10), ENTRY(rmsnorm_grad, 7),
    ENTRY(layernorm, 9), ENTRY(layernorm_grad, 9), ENTRY(expert_sort, 3), ENTRY(expert_dispatch, 3),
    ENTRY(expert_combine, 5), ENTRY(expert_combine_grad, 6), ENTRY(logprob, 4), ENTRY(logprob_grad, 8), ENTRY(distill, 4),
    ENTRY(distill_grad, 7), ENTRY(distill_step, 6),
    ENTRY(policy, 9), ENTRY(policy_grad, 13), ENTRY(policy_step, 11),
    {"set_check", set_check, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ew_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__ew_torch(void) { return PyModule_Create(&g_module); }
