// binding.cpp -- the Python module _ops: libgsort's language-model operators on
// torch tensors.  A call checks its arguments, allocates its outputs with torch
// and launches on the current stream of the tensors' device.  A single token's
// call costs little more than its launch that way (routing 8 tokens: 6 us of
// host time, 14 with the checks in Python and the call through ctypes).
//
// Functions take positional arguments only (the signatures that users see are in
// model_ops.py).  They raise TypeError for a wrong type and ValueError for a
// wrong shape, device or value, and return a gsort status (an int) where the
// library refuses or fails.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <optional>
#include <string>

#include "gsort.h"

namespace {

using at::Tensor;

struct Refused {};   // a Python error is set

template <typename... A> [[noreturn]] void refuse(PyObject *type, const char *format, A... args) {
    PyErr_Format(type, format, args...);
    throw Refused{};
}

std::string text(const Tensor &t) {
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "] of " + std::string(at::toString(t.scalar_type())) + " on " + t.device().str();
}

// While no Python object is touched, other threads run: an allocation may wait.
class WithoutGil {
  public:
    WithoutGil() : state_(PyEval_SaveThread()) {}
    ~WithoutGil() { PyEval_RestoreThread(state_); }

  private:
    PyThreadState *state_;
};

// ---------------------------------------------------------------- arguments
const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

std::optional<Tensor> optional_tensor(PyObject *o, const char *name) {
    if (o == Py_None) return std::nullopt;
    return tensor(o, name);
}

int integer(PyObject *o, const char *name) {
    PyObject *i = PyNumber_Index(o);
    if (i == nullptr) throw Refused{};
    int overflow = 0;
    const long v = PyLong_AsLongAndOverflow(i, &overflow);
    Py_DECREF(i);
    if (overflow != 0 || v < INT_MIN || v > INT_MAX) refuse(PyExc_ValueError, "%s is out of range", name);
    return static_cast<int>(v);
}

float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return static_cast<float>(v);
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v != 0;
}

// 0 for `first`, 1 for `second`.
int choice(PyObject *o, const char *name, const char *first, const char *second) {
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, first) == 0) return 0;
        if (PyUnicode_CompareWithASCIIString(o, second) == 0) return 1;
    }
    refuse(PyExc_ValueError, "%s must be '%s' or '%s', got %R", name, first, second, o);
}

int float_code(const Tensor &t, const char *name) {
    switch (t.scalar_type()) {
        case at::kFloat: return GSORT_F32;
        case at::kBFloat16: return GSORT_BF16;
        case at::kHalf: return GSORT_F16;
        default: refuse(PyExc_TypeError, "%s must be float32, bfloat16 or float16, got %s", name, text(t).c_str());
    }
}

// A 2-D float CUDA tensor whose row elements are consecutive.
struct Matrix {
    void *p;
    int code;
    int64_t rows, width, stride;
    at::Device device;
};

Matrix matrix(const Tensor &t, const char *name) {
    const int code = float_code(t, name);
    if (!t.is_cuda() || t.dim() != 2)
        refuse(PyExc_ValueError, "%s must be a CUDA tensor of two dimensions, got %s", name, text(t).c_str());
    const int64_t rows = t.size(0), width = t.size(1);
    if (width > 1 && t.stride(1) != 1) refuse(PyExc_ValueError, "the elements of a row of %s must be consecutive", name);
    // the stride of a tensor with one row (or none) means nothing
    return {t.data_ptr(), code, rows, width, rows > 1 ? t.stride(0) : width, t.device()};
}

// A contiguous tensor of the given type and shape on the device.
template <typename P = void>
P *flat(const Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, at::Device device) {
    if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s, got %s", name, at::toString(type), text(t).c_str());
    if (t.sizes() != shape) {
        std::string want = "[";
        for (size_t i = 0; i < shape.size(); ++i) want += (i ? ", " : "") + std::to_string(shape[i]);
        refuse(PyExc_ValueError, "%s must have shape %s], got %s", name, want.c_str(), text(t).c_str());
    }
    if (t.device() != device || !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be contiguous and on %s, got %s", name, device.str().c_str(), text(t).c_str());
    return static_cast<P *>(t.data_ptr());
}

template <typename P = void>
P *flat(const std::optional<Tensor> &t, const char *name, at::ScalarType type, at::IntArrayRef shape, at::Device device) {
    return t.has_value() ? flat<P>(*t, name, type, shape, device) : nullptr;
}

struct Targets {
    void *p;
    int bytes;
};

Targets targets_of(const std::optional<Tensor> &t, int64_t rows, at::Device device) {
    if (!t.has_value()) return {nullptr, 0};
    if (t->scalar_type() != at::kInt && t->scalar_type() != at::kLong)
        refuse(PyExc_TypeError, "targets must be int32 or int64, got %s", text(*t).c_str());
    return {flat(*t, "targets", t->scalar_type(), {rows}, device), static_cast<int>(t->element_size())};
}

// ------------------------------------------------------------------ results
Tensor make(at::IntArrayRef shape, at::ScalarType type, at::Device device) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(device));
}

float *floats(const Tensor &t) { return static_cast<float *>(t.data_ptr()); }
int32_t *ints(const Tensor &t) { return static_cast<int32_t *>(t.data_ptr()); }

cudaStream_t stream_of(at::Device device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

PyObject *wrap(const Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

PyObject *result(int status, const Tensor &t) { return status == GSORT_OK ? wrap(t) : PyLong_FromLong(status); }

template <size_t N> PyObject *result(int status, const Tensor (&t)[N]) {
    if (status != GSORT_OK) return PyLong_FromLong(status);
    PyObject *tuple = PyTuple_New(N);
    if (tuple == nullptr) return nullptr;
    for (size_t i = 0; i < N; ++i) {
        PyObject *o = wrap(t[i]);
        if (o == nullptr) {
            Py_DECREF(tuple);
            return nullptr;
        }
        PyTuple_SET_ITEM(tuple, static_cast<Py_ssize_t>(i), o);
    }
    return tuple;
}

// Runs f(args) for `want` arguments; C++ errors become Python's.
template <typename F> PyObject *entry(const char *name, Py_ssize_t given, Py_ssize_t want, F &&f) {
    HANDLE_TH_ERRORS
    if (given != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, given);
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ routing
PyObject *route_experts(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("route_experts", n, 9, [&] {
        const Matrix x = matrix(tensor(a[0], "logits"), "logits");
        const int k = integer(a[1], "k");
        const auto bias = optional_tensor(a[2], "bias");
        const int score = choice(a[3], "score", "softmax", "sigmoid"), groups = integer(a[4], "groups");
        const int kept = a[5] == Py_None ? groups : integer(a[5], "groups_kept");
        const int group_score = choice(a[6], "group_score", "max", "top2");
        const int renormalise = truth(a[7]);
        const float scale = real(a[8]);
        const float *b = flat<float>(bias, "bias", at::kFloat, {x.width}, x.device);
        if (k < 1) refuse(PyExc_ValueError, "k must be at least 1");
        Tensor out[2];
        // nothing is allocated for what the library refuses
        int rc = k > x.width ? GSORT_EINVAL : k > GSORT_ROUTE_MAX_CHOSEN ? GSORT_ETOOBIG : GSORT_OK;
        if (rc != GSORT_OK) return result(rc, out);
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(x.device);
            out[0] = make({x.rows, k}, at::kFloat, x.device);
            out[1] = make({x.rows, k}, at::kInt, x.device);
            const int experts = x.width > INT_MAX ? INT_MAX : static_cast<int>(x.width);
            rc = gsort_route_experts(x.p, x.code, x.rows, experts, x.stride, b, score, groups, kept, group_score, k, renormalise,
                                     scale, floats(out[0]), ints(out[1]), stream_of(x.device));
        }
        return result(rc, out);
    });
}

PyObject *route_experts_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("route_experts_backward", n, 6, [&] {
        const Tensor &d = tensor(a[0], "d_weights"), &logits = tensor(a[1], "logits"), &experts = tensor(a[2], "experts");
        const Matrix x = matrix(logits, "logits");
        const int score = choice(a[3], "score", "softmax", "sigmoid");
        const int renormalise = truth(a[4]);
        const float scale = real(a[5]);
        if (experts.dim() != 2) refuse(PyExc_ValueError, "experts must have two dimensions, got %s", text(experts).c_str());
        const int64_t k = experts.size(1);
        const int32_t *e = flat<int32_t>(experts, "experts", at::kInt, {x.rows, k}, x.device);
        const float *g = flat<float>(d, "d_weights", at::kFloat, {x.rows, k}, x.device);
        Tensor out;
        int rc;
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(x.device);
            out = make({x.rows, x.width}, logits.scalar_type(), x.device);
            const int number = x.width > INT_MAX ? INT_MAX : static_cast<int>(x.width);
            rc = gsort_route_experts_backward(g, x.p, x.code, x.rows, number, x.stride, e, k > INT_MAX ? INT_MAX : static_cast<int>(k),
                                              score, renormalise, scale, out.data_ptr(), stream_of(x.device));
        }
        return result(rc, out);
    });
}

// ----------------------------------------------------- grouping and row moves
PyObject *group_by_expert(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("group_by_expert", n, 4, [&] {
        const Tensor &experts = tensor(a[0], "experts");
        const int number = integer(a[1], "num_experts"), align = integer(a[2], "align");
        const auto given = optional_tensor(a[3], "workspace");
        if (!experts.is_cuda() || experts.dim() != 2)
            refuse(PyExc_ValueError, "experts must be a CUDA tensor of two dimensions, got %s", text(experts).c_str());
        const at::Device device = experts.device();
        const int32_t *e = flat<int32_t>(experts, "experts", at::kInt, experts.sizes(), device);
        if (given.has_value() && (given->device() != device || !given->is_contiguous()))
            refuse(PyExc_ValueError, "workspace must be contiguous and on %s", device.str().c_str());
        Tensor out[4];
        int rc;
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(device);
            const int64_t pairs = experts.numel(), capacity = gsort_group_capacity(pairs, number, align);
            const int64_t bytes = static_cast<int64_t>(gsort_group_workspace_bytes(pairs, number));
            Tensor ws = given.value_or(Tensor());
            if (!ws.defined() && bytes > 0) ws = make({bytes}, at::kByte, device);
            const int64_t held = number > 0 && number <= GSORT_ROUTE_MAX_EXPERTS ? number : 0;
            out[0] = make({held + 1}, at::kInt, device);
            out[1] = make({held}, at::kInt, device);
            out[2] = make({capacity}, at::kInt, device);
            out[3] = make(experts.sizes(), at::kInt, device);
            rc = gsort_group_by_expert(e, pairs, number, align, ints(out[0]), ints(out[1]), ints(out[2]), capacity, ints(out[3]),
                                       ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, stream_of(device));
        }
        return result(rc, out);
    });
}

// positions [tokens, slots] and rows [capacity] of the grouped layout.
struct Layout {
    const int32_t *positions, *rows;
    int64_t tokens, slots, capacity;
    int k() const { return slots > INT_MAX ? INT_MAX : static_cast<int>(slots); }
};

Layout layout(PyObject *positions, PyObject *rows, at::Device device) {
    const Tensor &p = tensor(positions, "groups.positions"), &r = tensor(rows, "groups.rows");
    if (p.dim() != 2) refuse(PyExc_ValueError, "groups.positions must have two dimensions, got %s", text(p).c_str());
    return {flat<int32_t>(p, "groups.positions", at::kInt, p.sizes(), device),
            flat<int32_t>(r, "groups.rows", at::kInt, {r.numel()}, device), p.size(0), p.size(1), r.numel()};
}

PyObject *dispatch_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("dispatch_rows", n, 3, [&] {
        const Tensor &t = tensor(a[0], "x");
        const Matrix x = matrix(t, "x");
        const Layout l = layout(a[1], a[2], x.device);
        if (x.rows != l.tokens) refuse(PyExc_ValueError, "x must have %lld rows, got %s", static_cast<long long>(l.tokens), text(t).c_str());
        Tensor out;
        int rc;
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(x.device);
            out = make({l.capacity, x.width}, t.scalar_type(), x.device);
            rc = gsort_dispatch_rows(x.p, x.code, l.tokens, x.width, x.stride, l.positions, l.k(), l.rows, l.capacity, out.data_ptr(),
                                     stream_of(x.device));
        }
        return result(rc, out);
    });
}

PyObject *combine_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("combine_rows", n, 4, [&] {
        const Tensor &t = tensor(a[0], "y");
        const Matrix y = matrix(t, "y");
        const Layout l = layout(a[1], a[2], y.device);
        const auto weights = optional_tensor(a[3], "weights");
        if (y.rows != l.capacity) refuse(PyExc_ValueError, "y must have %lld rows, got %s", static_cast<long long>(l.capacity), text(t).c_str());
        const float *w = flat<float>(weights, "weights", at::kFloat, {l.tokens, l.slots}, y.device);
        Tensor out;
        int rc;
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(y.device);
            out = make({l.tokens, y.width}, t.scalar_type(), y.device);
            rc = gsort_combine_rows(y.p, y.code, l.capacity, y.width, y.stride, w, l.positions, l.tokens, l.k(), out.data_ptr(),
                                    stream_of(y.device));
        }
        return result(rc, out);
    });
}

PyObject *combine_rows_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("combine_rows_backward", n, 5, [&] {
        const Tensor &dt = tensor(a[0], "d_out"), &yt = tensor(a[1], "y"), &wt = tensor(a[4], "weights");
        const Matrix d = matrix(dt, "d_out"), y = matrix(yt, "y");
        if (d.code != y.code) refuse(PyExc_TypeError, "d_out and y must have one dtype");
        const Layout l = layout(a[2], a[3], d.device);
        if (d.rows != l.tokens || y.rows != l.capacity || d.width != y.width || y.device != d.device)
            refuse(PyExc_ValueError, "d_out must be [tokens, width] and y [capacity, width] on one device, got %s and %s", text(dt).c_str(),
                   text(yt).c_str());
        const float *w = flat<float>(wt, "weights", at::kFloat, {l.tokens, l.slots}, d.device);
        Tensor out[2];
        int rc;
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(d.device);
            out[0] = make({l.capacity, y.width}, yt.scalar_type(), d.device);
            out[1] = make({l.tokens, l.slots}, at::kFloat, d.device);
            rc = gsort_combine_rows_backward(d.p, d.code, l.tokens, d.width, d.stride, y.p, l.capacity, y.stride, w, l.positions, l.k(),
                                             l.rows, out[0].data_ptr(), floats(out[1]), stream_of(d.device));
        }
        return result(rc, out);
    });
}

// -------------------------------------------------------- log probabilities
PyObject *token_logprobs(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("token_logprobs", n, 3, [&] {
        const Matrix x = matrix(tensor(a[0], "logits"), "logits");
        const auto targets = optional_tensor(a[1], "targets");
        const int top = integer(a[2], "top");
        const Targets t = targets_of(targets, x.rows, x.device);
        if (top < 0) refuse(PyExc_ValueError, "top must not be negative");
        Tensor out[5];     // logprobs, entropy, top_logprobs, top_ids, stats
        int rc = top > GSORT_LOGPROBS_MAX_TOP ? GSORT_ETOOBIG : GSORT_OK;   // nothing is allocated for it
        if (rc != GSORT_OK) return result(rc, out);
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(x.device);
            if (targets.has_value()) out[0] = make({x.rows}, at::kFloat, x.device);
            out[1] = make({x.rows}, at::kFloat, x.device);
            if (top > 0) {
                out[2] = make({x.rows, top}, at::kFloat, x.device);
                out[3] = make({x.rows, top}, at::kInt, x.device);
            }
            out[4] = make({x.rows, 2}, at::kFloat, x.device);
            rc = gsort_token_logprobs(x.p, x.code, x.rows, x.width, x.stride, t.p, t.bytes, top, out[0].defined() ? floats(out[0]) : nullptr,
                                      floats(out[1]), floats(out[4]), top > 0 ? floats(out[2]) : nullptr, top > 0 ? ints(out[3]) : nullptr,
                                      stream_of(x.device));
        }
        return result(rc, out);
    });
}

PyObject *token_logprobs_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("token_logprobs_backward", n, 7, [&] {
        const auto dl = optional_tensor(a[0], "d_logprobs"), dh = optional_tensor(a[1], "d_entropy");
        const Tensor &logits = tensor(a[2], "logits"), &entropy = tensor(a[4], "result.entropy"), &stats = tensor(a[5], "result.stats");
        const auto targets = optional_tensor(a[3], "targets");
        const auto given = optional_tensor(a[6], "out");
        const Matrix x = matrix(logits, "logits");
        const Targets t = targets_of(targets, x.rows, x.device);
        if (dl.has_value() && !targets.has_value()) refuse(PyExc_ValueError, "d_logprobs needs targets");
        const float *l = flat<float>(dl, "d_logprobs", at::kFloat, {x.rows}, x.device);
        const float *h = flat<float>(dh, "d_entropy", at::kFloat, {x.rows}, x.device);
        const float *ent = flat<float>(entropy, "result.entropy", at::kFloat, {x.rows}, x.device);
        const float *st = flat<float>(stats, "result.stats", at::kFloat, {x.rows, 2}, x.device);
        Tensor out;
        int64_t stride;
        if (given.has_value()) {
            const Matrix o = matrix(*given, "out");
            if (o.code != x.code || o.rows != x.rows || o.width != x.width || o.device != x.device)
                refuse(PyExc_ValueError, "out must have the logits' dtype, shape and device, got %s", text(*given).c_str());
            out = *given;
            stride = o.stride;
        } else {
            // rows as far from a 16-byte boundary as the logits' move in whole vectors
            const int64_t vector = 16 / logits.element_size(), between = (x.stride - x.width) % vector;
            stride = x.width + (between < 0 ? 0 : between);
        }
        int rc;
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(x.device);
            if (!out.defined()) {
                out = make({x.rows, stride}, logits.scalar_type(), x.device);
                if (stride != x.width) out = out.narrow(1, 0, x.width);
            }
            rc = gsort_token_logprobs_backward(l, h, x.p, x.code, x.rows, x.width, x.stride, t.p, t.bytes, ent, st, out.data_ptr(), stride,
                                               stream_of(x.device));
        }
        return result(rc, out);
    });
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(route_experts),   METHOD(route_experts_backward), METHOD(group_by_expert),
                         METHOD(dispatch_rows),   METHOD(combine_rows),           METHOD(combine_rows_backward),
                         METHOD(token_logprobs),  METHOD(token_logprobs_backward), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops() { return PyModule_Create(&module); }
