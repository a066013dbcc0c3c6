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
#include <ATen/ops/empty_like.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <optional>
#include <string>
#include <vector>

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
    if (!THPVariable_CheckExact(o) && !THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
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

// ---------------------------------------------------------------- embedding
// Token ids of any shape, one behind another.
Targets tokens_of(const Tensor &t, at::Device device) {
    if (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong)
        refuse(PyExc_TypeError, "tokens must be int32 or int64, got %s", text(t).c_str());
    return {flat(t, "tokens", t.scalar_type(), t.sizes(), device), static_cast<int>(t.element_size())};
}

PyObject *embed_tokens(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("embed_tokens", n, 3, [&] {
        const Tensor &table = tensor(a[0], "table"), &tokens = tensor(a[1], "tokens");
        const Matrix x = matrix(table, "table");
        const Targets t = tokens_of(tokens, x.device);
        const float scale = real(a[2]);
        Tensor out;
        int rc;
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(x.device);
            std::vector<int64_t> shape(tokens.sizes().begin(), tokens.sizes().end());
            shape.push_back(x.width);
            out = make(shape, table.scalar_type(), x.device);
            rc = gsort_embed_tokens(x.p, x.code, x.rows, x.width, x.stride, t.p, t.bytes, tokens.numel(), scale, out.data_ptr(),
                                    stream_of(x.device));
        }
        return result(rc, out);
    });
}

PyObject *embed_tokens_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("embed_tokens_backward", n, 7, [&] {
        const Tensor &d = tensor(a[0], "d_out"), &tokens = tensor(a[1], "tokens");
        const int vocab = integer(a[2], "vocab");
        const float scale = real(a[3]);
        const auto given = optional_tensor(a[4], "out"), space = optional_tensor(a[6], "workspace");
        const bool accumulate = truth(a[5]);
        const int code = float_code(d, "d_out");
        if (!d.is_cuda() || d.dim() != tokens.dim() + 1 || d.sizes().slice(0, tokens.dim()) != tokens.sizes())
            refuse(PyExc_ValueError, "d_out must be a CUDA tensor with a row for each token, got %s for tokens %s", text(d).c_str(), text(tokens).c_str());
        const at::Device device = d.device();
        const Targets t = tokens_of(tokens, device);
        const int64_t width = d.size(-1), rows = tokens.numel();
        int64_t stride = width;
        if (d.dim() == 2) stride = matrix(d, "d_out").stride;
        else if (!d.is_contiguous()) refuse(PyExc_ValueError, "d_out must be contiguous, or have two dimensions, got %s", text(d).c_str());
        if (vocab < 1) refuse(PyExc_ValueError, "vocab must be at least 1");
        if (accumulate && !given.has_value()) refuse(PyExc_ValueError, "accumulate needs out");
        if (space.has_value() && (space->device() != device || !space->is_contiguous()))
            refuse(PyExc_ValueError, "workspace must be contiguous and on %s", device.str().c_str());
        int64_t table_stride = width;
        if (given.has_value()) {
            const Matrix o = matrix(*given, "out");
            if (o.code != code || o.rows != vocab || o.width != width || o.device != device)
                refuse(PyExc_ValueError, "out must have d_out's dtype and device and shape [%d, %lld], got %s", vocab,
                       static_cast<long long>(width), text(*given).c_str());
            table_stride = o.stride;
        }
        Tensor out;
        int rc;
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(device);
            const int64_t bytes = static_cast<int64_t>(gsort_embed_tokens_backward_workspace_bytes(rows, vocab, width, code));
            Tensor ws = space.value_or(Tensor());
            if (!ws.defined() && bytes > 0) ws = make({bytes}, at::kByte, device);
            out = given.has_value() ? *given : make({vocab, width}, d.scalar_type(), device);
            rc = gsort_embed_tokens_backward(d.data_ptr(), code, rows, width, stride, t.p, t.bytes, vocab, scale, accumulate, out.data_ptr(),
                                             table_stride, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0,
                                             stream_of(device));
        }
        return result(rc, out);
    });
}

// ---------------------------------------------------------- adjusted logits
// [rows, any] on the device, the elements of a row consecutive; the rows may be one (expanded).
struct Lists {
    void *p;
    int64_t length, stride;
    int bytes;
};

Lists lists(const std::optional<Tensor> &t, const char *name, int64_t rows, at::Device device, std::initializer_list<at::ScalarType> types) {
    if (!t.has_value()) return {nullptr, 0, 0, 0};
    bool fits = false;
    std::string names;
    for (const at::ScalarType type : types) {
        fits = fits || t->scalar_type() == type;
        names += (names.empty() ? "" : " or ") + std::string(at::toString(type));
    }
    if (!fits) refuse(PyExc_TypeError, "%s must be %s, got %s", name, names.c_str(), text(*t).c_str());
    if (t->device() != device || t->dim() != 2 || t->size(0) != rows)
        refuse(PyExc_ValueError, "%s must have %lld rows on %s, got %s", name, static_cast<long long>(rows), device.str().c_str(), text(*t).c_str());
    if (t->size(1) > 1 && t->stride(1) != 1) refuse(PyExc_ValueError, "the elements of a row of %s must be consecutive", name);
    return {t->data_ptr(), t->size(1), rows > 1 ? t->stride(0) : t->size(1), static_cast<int>(t->element_size())};
}

// The fields of the adjustments, in the order of the arguments from a[0] on.
gsort_adjustments adjustments(const std::optional<Tensor> (&t)[8], const Matrix &x) {
    gsort_adjustments h = {};
    const Lists history = lists(t[0], "history", x.rows, x.device, {at::kInt, at::kLong});
    const Lists tokens = lists(t[5], "bias_tokens", x.rows, x.device, {at::kInt, at::kLong});
    const Lists bias = lists(t[6], "bias", x.rows, x.device, {at::kFloat});
    const Lists allowed = lists(t[7], "allowed", x.rows, x.device, {at::kInt});
    h.d_prompt = flat<int32_t>(t[1], "prompt", at::kInt, {x.rows}, x.device);
    h.d_repetition = flat<float>(t[2], "repetition", at::kFloat, {x.rows}, x.device);
    h.d_presence = flat<float>(t[3], "presence", at::kFloat, {x.rows}, x.device);
    h.d_frequency = flat<float>(t[4], "frequency", at::kFloat, {x.rows}, x.device);
    if (!t[0].has_value() && (t[1].has_value() || t[2].has_value() || t[3].has_value() || t[4].has_value()))
        refuse(PyExc_ValueError, "penalties need a history");
    if (t[5].has_value() != t[6].has_value()) refuse(PyExc_ValueError, "bias_tokens and bias come together");
    if (tokens.length != bias.length || (tokens.length > 0 && tokens.stride != bias.stride))
        refuse(PyExc_ValueError, "bias_tokens and bias must have one shape and one distance between rows");
    const int64_t words = (x.width + 31) / 32;
    if (t[7].has_value() && allowed.length != words)
        refuse(PyExc_ValueError, "allowed must have %lld words to a row, got %s", static_cast<long long>(words), text(*t[7]).c_str());
    // an empty history has no address, but its penalties are no mistake
    if (history.length > 0) {
        h.d_history = history.p;
        h.length = history.length;
        h.history_stride = history.stride;
        h.history_bytes = history.bytes;
    } else {
        h.d_prompt = nullptr;
        h.d_repetition = h.d_presence = h.d_frequency = nullptr;
    }
    h.d_bias_tokens = tokens.p;
    h.d_bias = static_cast<float *>(bias.p);
    h.biases = tokens.length;
    h.bias_stride = tokens.stride;
    h.bias_bytes = tokens.bytes;
    h.d_allowed = static_cast<uint32_t *>(allowed.p);
    h.allowed_stride = allowed.stride;
    return h;
}

// The output's row stride: of the tensor given, or one with which rows lie to 16
// bytes as the input's do, so that both move in whole vectors.
int64_t adjusted_stride(const std::optional<Tensor> &given, const Matrix &x, int64_t element) {
    if (!given.has_value()) {
        const int64_t vector = 16 / element, between = (x.stride - x.width) % vector;
        return x.width + (between < 0 ? 0 : between);
    }
    const Matrix o = matrix(*given, "out");
    if (o.code != x.code || o.rows != x.rows || o.width != x.width || o.device != x.device)
        refuse(PyExc_ValueError, "out must have the input's dtype, shape and device, got %s", text(*given).c_str());
    return o.stride;
}

Tensor adjusted_out(const std::optional<Tensor> &given, const Matrix &x, at::ScalarType type, int64_t stride) {
    if (given.has_value()) return *given;
    const Tensor whole = make({x.rows, stride}, type, x.device);
    return stride == x.width ? whole : whole.narrow(1, 0, x.width);
}

PyObject *adjust_logits(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("adjust_logits", n, 10, [&] {
        const Tensor &logits = tensor(a[0], "logits");
        const Matrix x = matrix(logits, "logits");
        const std::optional<Tensor> given = optional_tensor(a[9], "out");
        const std::optional<Tensor> how[8] = {optional_tensor(a[1], "history"),     optional_tensor(a[2], "prompt"),
                                              optional_tensor(a[3], "repetition"),  optional_tensor(a[4], "presence"),
                                              optional_tensor(a[5], "frequency"),   optional_tensor(a[6], "bias_tokens"),
                                              optional_tensor(a[7], "bias"),        optional_tensor(a[8], "allowed")};
        const gsort_adjustments h = adjustments(how, x);
        const int64_t stride = adjusted_stride(given, x, logits.element_size());
        Tensor out;
        int rc;
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(x.device);
            out = adjusted_out(given, x, logits.scalar_type(), stride);
            rc = gsort_adjust_logits(x.p, x.code, x.rows, x.width, x.stride, &h, out.data_ptr(), stride, stream_of(x.device));
        }
        return result(rc, out);
    });
}

PyObject *adjust_logits_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("adjust_logits_backward", n, 6, [&] {
        const Tensor &dt = tensor(a[0], "d_out");
        const Matrix d = matrix(dt, "d_out");
        const auto logits = optional_tensor(a[1], "logits"), given = optional_tensor(a[5], "out");
        const std::optional<Tensor> how[8] = {optional_tensor(a[2], "history"), std::nullopt, optional_tensor(a[3], "repetition"), std::nullopt,
                                              std::nullopt, std::nullopt, std::nullopt, optional_tensor(a[4], "allowed")};
        const gsort_adjustments h = adjustments(how, d);
        void *lp = nullptr;
        int64_t logits_stride = 0;
        if (logits.has_value()) {
            const Matrix x = matrix(*logits, "logits");
            if (x.code != d.code || x.rows != d.rows || x.width != d.width || x.device != d.device)
                refuse(PyExc_ValueError, "logits must have d_out's dtype, shape and device, got %s and %s", text(*logits).c_str(), text(dt).c_str());
            lp = x.p;
            logits_stride = x.stride;
        } else if (h.d_repetition != nullptr) {
            refuse(PyExc_ValueError, "repetition needs the logits");
        }
        const int64_t stride = adjusted_stride(given, d, dt.element_size());
        Tensor out;
        int rc;
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(d.device);
            out = adjusted_out(given, d, dt.scalar_type(), stride);
            rc = gsort_adjust_logits_backward(d.p, d.code, d.rows, d.width, d.stride, lp, logits_stride, &h, out.data_ptr(), stride,
                                              stream_of(d.device));
        }
        return result(rc, out);
    });
}

// ------------------------------------------------------------ gradient norm
// The tensors of a list: dense, on one device.
struct TensorList {
    PyObject *items = nullptr;      // a tuple of the call's own: another thread may change the list meanwhile
    std::vector<const void *> data;
    std::vector<int64_t> sizes;
    std::vector<int> codes;
    std::optional<at::Device> device;

    ~TensorList() { Py_XDECREF(items); }
    int64_t count() const { return static_cast<int64_t>(sizes.size()); }
    const Tensor &at(int64_t i) const { return THPVariable_Unpack(PyTuple_GET_ITEM(items, i)); }

    void read(PyObject *o, const char *name, const char *what) {
        PyObject *fast = PySequence_Fast(o, what);
        if (fast == nullptr) throw Refused{};
        items = PySequence_Tuple(fast);
        Py_DECREF(fast);
        if (items == nullptr) throw Refused{};
        const Py_ssize_t n = PyTuple_GET_SIZE(items);
        data.reserve(n);
        sizes.reserve(n);
        codes.reserve(n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            const Tensor &t = tensor(PyTuple_GET_ITEM(items, i), name);
            codes.push_back(float_code(t, name));
            if (t.layout() != at::kStrided || !t.is_cuda() || (device.has_value() && t.device() != *device))
                refuse(PyExc_ValueError, "%s must be strided CUDA tensors of one device, got %s", name, text(t).c_str());
            if (!t.is_non_overlapping_and_dense()) refuse(PyExc_ValueError, "%s must be dense, got %s with gaps or overlaps", name, text(t).c_str());
            if (t.requires_grad() && c10::GradMode::is_enabled())
                refuse(PyExc_RuntimeError, "norm and clipping have no gradient: call them under torch.no_grad() or on detached tensors");
            device = t.device();
            data.push_back(t.data_ptr());
            sizes.push_back(t.numel());
        }
    }
};

at::Device norm_device(const TensorList &list) {
    if (!list.device.has_value()) refuse(PyExc_ValueError, "there are no gradients");
    return *list.device;
}

Tensor norm_workspace(const TensorList &list, at::Device device) {
    return make({static_cast<int64_t>(gsort_gradient_norm_workspace_bytes(list.count()))}, at::kByte, device);
}

PyObject *gradient_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("gradient_norm", n, 1, [&] {
        TensorList g;
        g.read(a[0], "gradients", "gradients must be a list of tensors");
        const at::Device device = norm_device(g);
        Tensor out;
        int rc;
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(device);
            const Tensor ws = norm_workspace(g, device);
            out = make({}, at::kFloat, device);
            rc = gsort_gradient_norm(g.data.data(), g.sizes.data(), g.codes.data(), g.count(), floats(out), ws.data_ptr(), ws.nbytes(),
                                     stream_of(device));
        }
        return result(rc, out);
    });
}

// (list of the clipped tensors, norm)
PyObject *clip_gradients(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry("clip_gradients", n, 4, [&]() -> PyObject * {
        TensorList g, o;
        g.read(a[0], "gradients", "gradients must be a list of tensors");
        const float max_norm = real(a[1]), scale = real(a[2]);
        const at::Device device = norm_device(g);
        std::vector<Tensor> made;
        std::vector<void *> out;
        out.reserve(g.count());
        if (a[3] != Py_None) {
            o.read(a[3], "out", "out must be a list of tensors");
            if (o.count() > 0 && *o.device != device) refuse(PyExc_ValueError, "out must be on %s", device.str().c_str());
            if (o.count() != g.count()) refuse(PyExc_ValueError, "out must have as many tensors as the gradients");
            for (int64_t i = 0; i < g.count(); ++i) {
                const Tensor &x = g.at(i), &y = o.at(i);
                bool same = g.codes[i] == o.codes[i] && x.sizes() == y.sizes();
                if (same && x.strides() != y.strides())
                    for (int64_t k = 0; same && k < x.dim(); ++k) same = x.size(k) < 2 || x.stride(k) == y.stride(k);
                if (!same) refuse(PyExc_ValueError, "out[%lld] must have its gradient's dtype, shape and strides, got %s and %s",
                                  static_cast<long long>(i), text(y).c_str(), text(x).c_str());
                out.push_back(const_cast<void *>(o.data[i]));
            }
        }
        Tensor norm;
        int rc;
        {
            WithoutGil released;
            const c10::cuda::CUDAGuard guard(device);
            if (out.empty()) {
                made.reserve(g.count());
                for (int64_t i = 0; i < g.count(); ++i) {
                    made.push_back(at::empty_like(g.at(i)));
                    out.push_back(made.back().data_ptr());
                }
            }
            const Tensor ws = norm_workspace(g, device);
            norm = make({}, at::kFloat, device);
            rc = gsort_clip_gradients(g.data.data(), out.data(), g.sizes.data(), g.codes.data(), g.count(), max_norm, scale, floats(norm),
                                      ws.data_ptr(), ws.nbytes(), stream_of(device));
        }
        if (rc != GSORT_OK) return PyLong_FromLong(rc);
        PyObject *list;
        if (o.items != nullptr) {
            // autograd refuses what it had saved of them
            for (int64_t i = 0; i < g.count(); ++i)
                if (!o.at(i).is_inference()) o.at(i).unsafeGetTensorImpl()->bump_version();
            list = PySequence_List(o.items);
        } else {
            list = PyList_New(static_cast<Py_ssize_t>(g.count()));
            for (int64_t i = 0; list != nullptr && i < g.count(); ++i) {
                PyObject *item = wrap(made[i]);
                if (item == nullptr) Py_CLEAR(list);
                else PyList_SET_ITEM(list, i, item);
            }
        }
        if (list == nullptr) return nullptr;
        PyObject *last = wrap(norm);
        PyObject *both = last ? PyTuple_Pack(2, list, last) : nullptr;
        Py_XDECREF(last);
        Py_DECREF(list);
        return both;
    });
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(route_experts),   METHOD(route_experts_backward), METHOD(group_by_expert),
                         METHOD(dispatch_rows),   METHOD(combine_rows),           METHOD(combine_rows_backward),
                         METHOD(token_logprobs),  METHOD(token_logprobs_backward), METHOD(embed_tokens),
                         METHOD(embed_tokens_backward), METHOD(adjust_logits),     METHOD(adjust_logits_backward),
                         METHOD(gradient_norm),   METHOD(clip_gradients),          {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops() { return PyModule_Create(&module); }
