// api_model.cu -- the extern "C" boundary of the language-model operators:
// argument checks before any CUDA call, then one launcher.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "model_ops.cuh"

namespace gsort {
namespace {

// A strided array of rows: its first byte and its extent.
struct Span {
    const void *p;
    size_t bytes;
};

Span rows_span(const void *p, int64_t rows, int64_t width, int64_t stride, size_t size) {
    return {p, rows > 0 ? (static_cast<size_t>(rows - 1) * stride + width) * size : 0};
}

bool overlap(const Span &a, const Span &b) {
    return a.p != nullptr && b.p != nullptr && ranges_overlap(a.p, a.bytes, b.p, b.bytes);
}

// Whether an output overlaps an input or another output.
template <size_t I, size_t O> bool clash(const Span (&in)[I], const Span (&out)[O]) {
    for (size_t o = 0; o < O; ++o) {
        for (size_t i = 0; i < I; ++i)
            if (overlap(out[o], in[i])) return true;
        for (size_t q = 0; q < o; ++q)
            if (overlap(out[o], out[q])) return true;
    }
    return false;
}

// Rows of a strided array; the extent has to fit 63 bits.
int rows_args(int64_t rows, int64_t width, int64_t stride) {
    if (rows < 0 || width < 1 || stride < 0) return GSORT_EINVAL;
    if (rows > GSORT_MAX_N || width > GSORT_MAX_N) return GSORT_ETOOBIG;
    if (rows > 1 && stride < width) return GSORT_EINVAL;
    if (stride > (static_cast<int64_t>(1) << 62) / 8 / std::max<int64_t>(rows, 1)) return GSORT_ETOOBIG;
    return GSORT_OK;
}

int route_args(int dtype, int64_t tokens, int experts, int64_t row_stride, int score, int chosen, float scale) {
    if (float_bytes(dtype) == 0 || experts < 1) return GSORT_EINVAL;
    if (experts > GSORT_ROUTE_MAX_EXPERTS) return GSORT_ETOOBIG;
    const int rc = rows_args(tokens, experts, row_stride);
    if (rc != GSORT_OK) return rc;
    if (score != GSORT_SCORE_SOFTMAX && score != GSORT_SCORE_SIGMOID) return GSORT_EINVAL;
    if (chosen < 1 || chosen > experts) return GSORT_EINVAL;
    if (chosen > GSORT_ROUTE_MAX_CHOSEN) return GSORT_ETOOBIG;
    return std::isfinite(scale) ? GSORT_OK : GSORT_EINVAL;
}

// Shape of the grouped layout and the positions into it.
int layout_args(int dtype, int64_t tokens, int64_t width, int chosen, int64_t capacity) {
    if (float_bytes(dtype) == 0 || tokens < 0 || width < 1 || chosen < 1 || capacity < 0) return GSORT_EINVAL;
    if (tokens > GSORT_MAX_N || width > GSORT_MAX_N || capacity > GSORT_MAX_N) return GSORT_ETOOBIG;
    if (tokens * chosen > GSORT_MAX_N) return GSORT_ETOOBIG;
    return GSORT_OK;
}

int embed_args(int dtype, int64_t vocab, int64_t width, int64_t tokens, int token_bytes, float scale) {
    if (float_bytes(dtype) == 0 || vocab < 1 || width < 1 || tokens < 0) return GSORT_EINVAL;
    if (token_bytes != 4 && token_bytes != 8) return GSORT_EINVAL;
    if (tokens > GSORT_MAX_N || vocab > GSORT_MAX_N || width > GSORT_MAX_N) return GSORT_ETOOBIG;
    return std::isfinite(scale) ? GSORT_OK : GSORT_EINVAL;
}

// Rows that are only read may all be one (stride 0).
int list_args(int64_t rows, int64_t width, int64_t stride) {
    return stride == 0 ? rows_args(1, width, width) : rows_args(rows, width, stride);
}

// The options of an extended call: limits of its waits.
int waits_of(const gsort_options *o, Waits *w) {
    if (o == nullptr) return GSORT_OK;
    if (o->variant != 0 || o->num_events < 0 || (o->num_events > 0 && o->events == nullptr)) return GSORT_EINVAL;
    if (o->spin_limit != 0) w->polls = o->spin_limit;
    if (o->stall_tile >= 0 && o->stall_tile < 0xFFFFFFFFll) w->stall = static_cast<uint32_t>(o->stall_tile);
    return GSORT_OK;
}

// The logits' adjustment (in: the logits) or its gradient (in: the gradient by the adjusted logits).
int adjust(bool backward, const void *logits, int64_t logits_stride, const void *in, int64_t in_stride, int dtype, int64_t rows,
           int64_t vocab, const gsort_adjustments *how, void *out, int64_t out_stride, cudaStream_t stream, const gsort_options *options) {
    if (float_bytes(dtype) == 0 || how == nullptr) return GSORT_EINVAL;
    const gsort_adjustments &h = *how;
    AdjustLaunch L;
    int rc = waits_of(options, &L.waits);
    if (rc == GSORT_OK) rc = rows_args(rows, vocab, in_stride);
    if (rc == GSORT_OK) rc = rows_args(rows, vocab, out_stride);
    const bool history = h.d_history != nullptr && h.length > 0 && (!backward || h.d_repetition != nullptr);
    if (rc == GSORT_OK && backward && history) rc = rows_args(rows, vocab, logits_stride);
    if (rc != GSORT_OK) return rc;
    if (h.length < 0 || h.biases < 0) return GSORT_EINVAL;
    const int64_t words = (vocab + 31) / 32;
    if (h.d_history != nullptr && h.history_bytes != 4 && h.history_bytes != 8) return GSORT_EINVAL;
    if (h.d_history == nullptr && (h.length > 0 || h.d_prompt || h.d_repetition || h.d_presence || h.d_frequency)) return GSORT_EINVAL;
    if (h.biases > 0 && (h.d_bias_tokens == nullptr || h.d_bias == nullptr)) return GSORT_EINVAL;
    if (h.biases > 0 && h.bias_bytes != 4 && h.bias_bytes != 8) return GSORT_EINVAL;
    if (history) rc = list_args(rows, h.length, h.history_stride);
    if (rc == GSORT_OK && h.biases > 0) rc = list_args(rows, h.biases, h.bias_stride);
    if (rc == GSORT_OK && h.d_allowed != nullptr) rc = list_args(rows, words, h.allowed_stride);
    if (rc != GSORT_OK || rows == 0) return rc;
    if (in == nullptr || out == nullptr || (backward && history && logits == nullptr)) return GSORT_EINVAL;
    const size_t size = float_bytes(dtype), n = static_cast<size_t>(rows);
    if (!aligned(in, size) || !aligned(out, size) || !aligned(logits, size) || !aligned(h.d_prompt, 4) || !aligned(h.d_repetition, 4) ||
        !aligned(h.d_presence, 4) || !aligned(h.d_frequency, 4) || !aligned(h.d_bias, 4) || !aligned(h.d_allowed, 4) ||
        (history && !aligned(h.d_history, h.history_bytes)) || (h.biases > 0 && !aligned(h.d_bias_tokens, h.bias_bytes)))
        return GSORT_EALIGN;
    const bool in_place = in == out && (in_stride == out_stride || rows == 1);
    const Span ins[] = {in_place ? Span{nullptr, 0} : rows_span(in, rows, vocab, in_stride, size),
                        backward && history ? rows_span(logits, rows, vocab, logits_stride, size) : Span{nullptr, 0},
                        history ? rows_span(h.d_history, rows, h.length, h.history_stride, h.history_bytes) : Span{nullptr, 0},
                        {h.d_prompt, n * 4}, {h.d_repetition, n * 4}, {h.d_presence, n * 4}, {h.d_frequency, n * 4},
                        h.biases > 0 ? rows_span(h.d_bias_tokens, rows, h.biases, h.bias_stride, h.bias_bytes) : Span{nullptr, 0},
                        h.biases > 0 ? rows_span(h.d_bias, rows, h.biases, h.bias_stride, 4) : Span{nullptr, 0},
                        h.d_allowed ? rows_span(h.d_allowed, rows, words, h.allowed_stride, 4) : Span{nullptr, 0}};
    const Span outs[] = {rows_span(out, rows, vocab, out_stride, size)};
    if (clash(ins, outs)) return GSORT_EINVAL;
    L.backward = backward;
    L.logits = logits;
    L.in = in;
    L.out = out;
    L.dtype = dtype;
    L.rows = rows;
    L.vocab = vocab;
    L.logits_stride = logits_stride;
    L.in_stride = in_stride;
    L.out_stride = out_stride;
    L.history = history ? h.d_history : nullptr;
    L.history_stride = h.history_stride;
    L.length = h.length;
    L.history_bytes = h.history_bytes;
    L.prompt = h.d_prompt;
    L.repetition = h.d_repetition;
    L.presence = h.d_presence;
    L.frequency = h.d_frequency;
    L.bias_tokens = h.d_bias_tokens;
    L.bias = h.d_bias;
    L.bias_stride = h.bias_stride;
    L.biases = h.biases;
    L.bias_bytes = h.bias_bytes;
    L.allowed = h.d_allowed;
    L.allowed_stride = h.allowed_stride;
    L.stream = stream;
    return launch_adjust(L);
}

// Whether the outputs lie one behind another, upwards or downwards, on one side of the inputs
// that are not outputs too, and nothing overlaps the norm and the workspace.  One look at lists as
// they mostly are (1500 tensors: 10 us, 50 with the lists below).
bool tensors_apart(const void *const *in, void *const *out, const int64_t *elements, const int *dtypes, int64_t tensors, const Span &norm,
                   const Span &ws) {
    bool up = true, down = true;
    uintptr_t last = 0, last_end = 0, low = UINTPTR_MAX, high = 0, read_low = UINTPTR_MAX, read_high = 0;
    auto outside = [&](uintptr_t a, uintptr_t n) {
        return !ranges_overlap(norm.p, norm.bytes, reinterpret_cast<const void *>(a), n) &&
               !(ws.bytes > 0 && ranges_overlap(ws.p, ws.bytes, reinterpret_cast<const void *>(a), n));
    };
    bool clear = ws.bytes == 0 || !ranges_overlap(norm.p, norm.bytes, ws.p, ws.bytes);
    for (int64_t i = 0; i < tensors; ++i) {
        const uintptr_t n = static_cast<uintptr_t>(elements[i]) * float_bytes(dtypes[i]);
        if (n == 0) continue;
        const uintptr_t a = reinterpret_cast<uintptr_t>(in[i]), o = out != nullptr ? reinterpret_cast<uintptr_t>(out[i]) : a;
        clear &= outside(a, n);
        if (out == nullptr) continue;
        if (o != a) {
            clear &= outside(o, n);
            read_low = std::min(read_low, a);
            read_high = std::max(read_high, a + n);
        }
        if (high > 0) {
            up &= o >= last_end;
            down &= o + n <= last;
        }
        last = o;
        last_end = o + n;
        low = std::min(low, o);
        high = std::max(high, o + n);
    }
    return clear && (up || down) && (read_high <= low || high <= read_low || read_high == 0);
}

struct Range {
    uintptr_t begin, end;
    bool written;
};

// By address.  An allocator gives tensors in runs that go up or down: those are merged.
void sort_runs(std::vector<Range> &v) {
    auto before = [](const Range &x, const Range &y) { return x.begin < y.begin; };
    std::vector<size_t> ends{0};         // of the runs
    for (size_t i = 0, k; i < v.size(); i = k) {
        k = i + 1;
        if (k < v.size() && before(v[k], v[i])) {
            while (k < v.size() && before(v[k], v[k - 1])) ++k;
            std::reverse(v.begin() + i, v.begin() + k);
        } else {
            while (k < v.size() && !before(v[k], v[k - 1])) ++k;
        }
        ends.push_back(k);
        if (ends.size() > v.size() / 8 + 8) return std::sort(v.begin(), v.end(), before);
    }
    while (ends.size() > 2) {
        size_t kept = 1;
        for (size_t i = 1; i < ends.size(); i += 2) {
            const size_t last = std::min(i + 1, ends.size() - 1);
            if (last > i) std::inplace_merge(v.begin() + ends[i - 1], v.begin() + ends[i], v.begin() + ends[last], before);
            ends[kept++] = ends[last];
        }
        ends.resize(kept);
    }
}

// Whether an output overlaps another output, the workspace, the norm or another tensor than the one
// it is the clipped form of (or that one in part).
bool tensors_clash(const void *const *in, void *const *out, const int64_t *elements, const int *dtypes, int64_t tensors, const Span &norm,
                   const Span &ws) {
    if (tensors_apart(in, out, elements, dtypes, tensors, norm, ws)) return false;
    std::vector<Range> lists[2];             // read (and written over, where the output is the input), written
    lists[0].reserve(tensors);
    lists[1].reserve(out != nullptr ? tensors + 2 : 2);
    auto add = [&](int l, const void *p, uintptr_t n, bool written) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p);
        if (n > 0) lists[l].push_back({a, a + n, written});
    };
    for (int64_t i = 0; i < tensors; ++i) {
        const uintptr_t n = static_cast<uintptr_t>(elements[i]) * float_bytes(dtypes[i]);
        const bool same = out != nullptr && in[i] == out[i];
        add(0, in[i], n, same);
        if (out != nullptr && !same) add(1, out[i], n, true);
    }
    add(1, norm.p, norm.bytes, true);
    add(1, ws.p, ws.bytes, true);
    for (std::vector<Range> &list : lists) sort_runs(list);
    uintptr_t end = 0, written = 0;      // the furthest end of any range so far, and of a written one
    for (size_t i = 0, k = 0; i < lists[0].size() || k < lists[1].size();) {
        const bool first = k == lists[1].size() || (i < lists[0].size() && lists[0][i].begin < lists[1][k].begin);
        const Range &r = first ? lists[0][i++] : lists[1][k++];
        if (r.begin < written || (r.written && r.begin < end)) return true;
        end = std::max(end, r.end);
        if (r.written) written = std::max(written, r.end);
    }
    return false;
}

int norm(const void *const *in, void *const *out, const int64_t *elements, const int *dtypes, int64_t tensors, float max_norm,
         float scale, float *d_norm, void *ws, size_t ws_bytes, cudaStream_t stream, const gsort_options *options) {
    NormLaunch L;
    const int rc = waits_of(options, &L.waits);
    if (rc != GSORT_OK) return rc;
    if (tensors < 0 || !std::isfinite(scale) || !(max_norm >= 0.0f)) return GSORT_EINVAL;
    if (tensors > GSORT_MAX_N) return GSORT_ETOOBIG;
    if (d_norm == nullptr || (tensors > 0 && (in == nullptr || elements == nullptr || dtypes == nullptr))) return GSORT_EINVAL;
    if (!aligned(d_norm, 4)) return GSORT_EALIGN;
    for (int64_t i = 0; i < tensors; ++i) {
        const int size = float_bytes(dtypes[i]);
        if (size == 0 || elements[i] < 0) return GSORT_EINVAL;
        if (elements[i] > static_cast<int64_t>(1) << 44) return GSORT_ETOOBIG;
        if (elements[i] > 0 && (in[i] == nullptr || (out != nullptr && out[i] == nullptr))) return GSORT_EINVAL;
        if (!aligned(in[i], size) || (out != nullptr && !aligned(out[i], size))) return GSORT_EALIGN;
    }
    const size_t need = norm_workspace_bytes(tensors);
    if (need > 0) {
        if (ws == nullptr || ws_bytes < need) return GSORT_EWORKSPACE;
        if (!aligned(ws, kWsAlign)) return GSORT_EALIGN;
    }
    try {
        if (tensors_clash(in, out, elements, dtypes, tensors, {d_norm, 4}, {ws, need})) return GSORT_EINVAL;
    } catch (const std::bad_alloc &) {
        return GSORT_ETOOBIG;
    }
    L.in = in;
    L.out = out;
    L.sizes = elements;
    L.dtypes = dtypes;
    L.tensors = tensors;
    L.scale = scale;
    L.max_norm = max_norm;
    L.norm = d_norm;
    L.ws = static_cast<unsigned char *>(ws);
    L.stream = stream;
    return launch_norm(L);
}

}  // namespace
}  // namespace gsort

using namespace gsort;

extern "C" {

int gsort_route_experts(const void *d_logits, int dtype, int64_t tokens, int experts,
                        int64_t row_stride, const float *d_bias, int score, int groups,
                        int groups_kept, int group_score, int chosen, int renormalise, float scale,
                        float *d_weights, int32_t *d_experts, cudaStream_t stream) {
    const int rc = route_args(dtype, tokens, experts, row_stride, score, chosen, scale);
    if (rc != GSORT_OK) return rc;
    if (groups < 1 || groups > 32 || experts % groups != 0) return GSORT_EINVAL;
    if (groups_kept < 1 || groups_kept > groups) return GSORT_EINVAL;
    if (group_score != GSORT_GROUP_MAX && group_score != GSORT_GROUP_TOP2) return GSORT_EINVAL;
    if (tokens == 0) return GSORT_OK;
    if (d_logits == nullptr || d_weights == nullptr || d_experts == nullptr) return GSORT_EINVAL;
    const size_t size = float_bytes(dtype), pairs = static_cast<size_t>(tokens) * chosen;
    if (!aligned(d_logits, size) || !aligned(d_weights, 4) || !aligned(d_experts, 4) || !aligned(d_bias, 4))
        return GSORT_EALIGN;
    const Span in[] = {rows_span(d_logits, tokens, experts, row_stride, size), {d_bias, experts * sizeof(float)}};
    const Span out[] = {{d_weights, pairs * 4}, {d_experts, pairs * 4}};
    if (clash(in, out)) return GSORT_EINVAL;
    RouteLaunch L;
    L.logits = d_logits;
    L.dtype = dtype;
    L.tokens = tokens;
    L.row_stride = row_stride;
    L.experts = experts;
    L.bias = d_bias;
    L.score = score;
    L.groups = groups_kept == groups ? 1 : groups;   // every group kept: no groups
    L.groups_kept = groups_kept == groups ? 1 : groups_kept;
    L.group_score = group_score;
    L.chosen = chosen;
    L.renormalise = renormalise != 0;
    L.scale = scale;
    L.weights = d_weights;
    L.experts_out = d_experts;
    L.stream = stream;
    return launch_route(L);
}

int gsort_route_experts_backward(const float *d_grad_weights, const void *d_logits, int dtype,
                                 int64_t tokens, int experts, int64_t row_stride,
                                 const int32_t *d_experts, int chosen, int score, int renormalise,
                                 float scale, void *d_grad_logits, cudaStream_t stream) {
    const int rc = route_args(dtype, tokens, experts, row_stride, score, chosen, scale);
    if (rc != GSORT_OK || tokens == 0) return rc;
    if (d_grad_weights == nullptr || d_logits == nullptr || d_experts == nullptr || d_grad_logits == nullptr)
        return GSORT_EINVAL;
    const size_t size = float_bytes(dtype), pairs = static_cast<size_t>(tokens) * chosen;
    if (!aligned(d_logits, size) || !aligned(d_grad_logits, size) || !aligned(d_grad_weights, 4) || !aligned(d_experts, 4))
        return GSORT_EALIGN;
    const Span in[] = {rows_span(d_logits, tokens, experts, row_stride, size), {d_grad_weights, pairs * 4}, {d_experts, pairs * 4}};
    const Span out[] = {rows_span(d_grad_logits, tokens, experts, experts, size)};
    if (clash(in, out)) return GSORT_EINVAL;
    RouteBackwardLaunch L;
    L.grad_weights = d_grad_weights;
    L.logits = d_logits;
    L.dtype = dtype;
    L.tokens = tokens;
    L.row_stride = row_stride;
    L.experts = experts;
    L.experts_in = d_experts;
    L.chosen = chosen;
    L.score = score;
    L.renormalise = renormalise != 0;
    L.scale = scale;
    L.grad_logits = d_grad_logits;
    L.stream = stream;
    return launch_route_backward(L);
}

int64_t gsort_group_capacity(int64_t pairs, int experts, int align) {
    if (pairs < 0 || pairs > GSORT_MAX_N || experts < 1 || experts > GSORT_ROUTE_MAX_EXPERTS || align < 1) return 0;
    const int64_t most = pairs + std::min<int64_t>(experts, pairs) * (align - 1);
    const int64_t capacity = most / align * align;
    return capacity <= GSORT_MAX_N ? capacity : 0;
}

size_t gsort_group_workspace_bytes(int64_t pairs, int experts) {
    if (pairs < 0 || pairs > GSORT_MAX_N || experts < 1 || experts > GSORT_ROUTE_MAX_EXPERTS) return 0;
    return group_workspace_bytes(static_cast<uint32_t>(pairs), experts);
}

int gsort_group_by_expert(const int32_t *d_experts, int64_t pairs, int experts, int align,
                          int32_t *d_offsets, int32_t *d_counts, int32_t *d_rows, int64_t capacity,
                          int32_t *d_positions, void *d_ws, size_t ws_bytes, cudaStream_t stream) {
    if (pairs < 0 || experts < 1 || align < 1 || capacity < 0) return GSORT_EINVAL;
    if (pairs > GSORT_MAX_N || experts > GSORT_ROUTE_MAX_EXPERTS) return GSORT_ETOOBIG;
    const int64_t need = gsort_group_capacity(pairs, experts, align);
    if (pairs > 0 && need == 0) return GSORT_ETOOBIG;
    if (capacity < need) return GSORT_EINVAL;
    if (capacity > GSORT_MAX_N) return GSORT_ETOOBIG;
    if (d_offsets == nullptr || d_counts == nullptr || (capacity > 0 && d_rows == nullptr)) return GSORT_EINVAL;
    if (pairs > 0 && (d_experts == nullptr || d_positions == nullptr)) return GSORT_EINVAL;
    if (!aligned(d_experts, 4) || !aligned(d_offsets, 4) || !aligned(d_counts, 4) || !aligned(d_rows, 4) || !aligned(d_positions, 4))
        return GSORT_EALIGN;
    const size_t ws = group_workspace_bytes(static_cast<uint32_t>(pairs), experts);
    if (ws > 0) {
        if (d_ws == nullptr || ws_bytes < ws) return GSORT_EWORKSPACE;
        if (!aligned(d_ws, kWsAlign)) return GSORT_EALIGN;
    }
    const Span in[] = {{d_experts, static_cast<size_t>(pairs) * 4}};
    const Span out[] = {{d_offsets, (static_cast<size_t>(experts) + 1) * 4},
                        {d_counts, static_cast<size_t>(experts) * 4},
                        {d_rows, static_cast<size_t>(capacity) * 4},
                        {d_positions, static_cast<size_t>(pairs) * 4},
                        {ws > 0 ? d_ws : nullptr, ws}};
    if (clash(in, out)) return GSORT_EINVAL;
    GroupLaunch L;
    L.experts_in = d_experts;
    L.pairs = static_cast<uint32_t>(pairs);
    L.experts = experts;
    L.align = static_cast<uint32_t>(align);
    L.offsets = d_offsets;
    L.counts = d_counts;
    L.rows = d_rows;
    L.positions = d_positions;
    L.capacity = static_cast<uint32_t>(capacity);
    L.ws = static_cast<uint32_t *>(d_ws);
    L.stream = stream;
    return launch_group(L);
}

int gsort_dispatch_rows(const void *d_x, int dtype, int64_t tokens, int64_t width, int64_t row_stride,
                        const int32_t *d_positions, int chosen, const int32_t *d_rows,
                        int64_t capacity, void *d_out, cudaStream_t stream) {
    int rc = layout_args(dtype, tokens, width, chosen, capacity);
    if (rc == GSORT_OK) rc = rows_args(tokens, width, row_stride);
    if (rc != GSORT_OK || capacity == 0) return rc;
    if (d_rows == nullptr || d_out == nullptr || (tokens > 0 && (d_x == nullptr || d_positions == nullptr))) return GSORT_EINVAL;
    const size_t size = float_bytes(dtype), pairs = static_cast<size_t>(tokens) * chosen;
    if (!aligned(d_x, size) || !aligned(d_out, size) || !aligned(d_positions, 4) || !aligned(d_rows, 4)) return GSORT_EALIGN;
    const Span in[] = {rows_span(d_x, tokens, width, row_stride, size), {d_positions, pairs * 4}, {d_rows, static_cast<size_t>(capacity) * 4}};
    const Span out[] = {rows_span(d_out, capacity, width, width, size)};
    if (clash(in, out)) return GSORT_EINVAL;
    RowsLaunch L{};
    L.dtype = dtype;
    L.tokens = tokens;
    L.width = width;
    L.chosen = chosen;
    L.capacity = capacity;
    L.positions = d_positions;
    L.rows = d_rows;
    L.by_token = d_x;
    L.token_stride = row_stride;
    L.out = d_out;
    L.stream = stream;
    return launch_dispatch(L);
}

int gsort_combine_rows(const void *d_y, int dtype, int64_t capacity, int64_t width, int64_t row_stride,
                       const float *d_weights, const int32_t *d_positions, int64_t tokens, int chosen,
                       void *d_out, cudaStream_t stream) {
    int rc = layout_args(dtype, tokens, width, chosen, capacity);
    if (rc == GSORT_OK) rc = rows_args(capacity, width, row_stride);
    if (rc != GSORT_OK || tokens == 0) return rc;
    if (d_positions == nullptr || d_out == nullptr || (capacity > 0 && d_y == nullptr)) return GSORT_EINVAL;
    const size_t size = float_bytes(dtype), pairs = static_cast<size_t>(tokens) * chosen;
    if (!aligned(d_y, size) || !aligned(d_out, size) || !aligned(d_positions, 4) || !aligned(d_weights, 4)) return GSORT_EALIGN;
    const Span in[] = {rows_span(d_y, capacity, width, row_stride, size), {d_positions, pairs * 4}, {d_weights, pairs * 4}};
    const Span out[] = {rows_span(d_out, tokens, width, width, size)};
    if (clash(in, out)) return GSORT_EINVAL;
    RowsLaunch L{};
    L.dtype = dtype;
    L.tokens = tokens;
    L.width = width;
    L.chosen = chosen;
    L.capacity = capacity;
    L.positions = d_positions;
    L.weights = d_weights;
    L.by_row = d_y;
    L.row_stride = row_stride;
    L.out = d_out;
    L.stream = stream;
    return launch_combine(L);
}

int gsort_combine_rows_backward(const void *d_grad_out, int dtype, int64_t tokens, int64_t width,
                                int64_t grad_stride, const void *d_y, int64_t capacity,
                                int64_t row_stride, const float *d_weights,
                                const int32_t *d_positions, int chosen, const int32_t *d_rows,
                                void *d_grad_y, float *d_grad_weights, cudaStream_t stream) {
    int rc = layout_args(dtype, tokens, width, chosen, capacity);
    if (rc == GSORT_OK) rc = rows_args(tokens, width, grad_stride);
    if (rc == GSORT_OK) rc = rows_args(capacity, width, row_stride);
    if (rc != GSORT_OK || (tokens == 0 && capacity == 0)) return rc;
    if (tokens > 0 && (d_grad_out == nullptr || d_weights == nullptr || d_positions == nullptr || d_grad_weights == nullptr))
        return GSORT_EINVAL;
    if (capacity > 0 && (d_y == nullptr || d_rows == nullptr || d_grad_y == nullptr)) return GSORT_EINVAL;
    const size_t size = float_bytes(dtype), pairs = static_cast<size_t>(tokens) * chosen;
    if (!aligned(d_grad_out, size) || !aligned(d_y, size) || !aligned(d_grad_y, size) || !aligned(d_weights, 4) ||
        !aligned(d_positions, 4) || !aligned(d_rows, 4) || !aligned(d_grad_weights, 4))
        return GSORT_EALIGN;
    const Span in[] = {rows_span(d_grad_out, tokens, width, grad_stride, size), rows_span(d_y, capacity, width, row_stride, size),
                       {d_weights, pairs * 4}, {d_positions, pairs * 4}, {d_rows, static_cast<size_t>(capacity) * 4}};
    const Span out[] = {rows_span(d_grad_y, capacity, width, width, size), {d_grad_weights, pairs * 4}};
    if (clash(in, out)) return GSORT_EINVAL;
    DeviceInfo dev;
    if (device_info(&dev) != GSORT_OK) return GSORT_ECUDA;
    RowsLaunch L{};
    L.sm_count = dev.sm_count;
    L.dtype = dtype;
    L.tokens = tokens;
    L.width = width;
    L.chosen = chosen;
    L.capacity = capacity;
    L.positions = d_positions;
    L.rows = d_rows;
    L.weights = d_weights;
    L.by_token = d_grad_out;
    L.token_stride = grad_stride;
    L.by_row = d_y;
    L.row_stride = row_stride;
    L.out = d_grad_y;
    L.grad_weights = d_grad_weights;
    L.stream = stream;
    return launch_combine_backward(L);
}

int gsort_token_logprobs(const void *d_logits, int dtype, int64_t rows, int64_t vocab,
                         int64_t row_stride, const void *d_targets, int target_bytes, int top,
                         float *d_logprobs, float *d_entropy, float *d_stats, float *d_top_logprobs,
                         int32_t *d_top_ids, cudaStream_t stream) {
    if (float_bytes(dtype) == 0 || top < 0) return GSORT_EINVAL;
    if (top > GSORT_LOGPROBS_MAX_TOP) return GSORT_ETOOBIG;
    int rc = rows_args(rows, vocab, row_stride);
    if (rc != GSORT_OK) return rc;
    if ((d_targets == nullptr) != (d_logprobs == nullptr) && rows > 0) return GSORT_EINVAL;
    if (d_targets != nullptr && target_bytes != 4 && target_bytes != 8) return GSORT_EINVAL;
    if (rows > (1 << 28)) return GSORT_ETOOBIG;      // up to 8 CTAs to a row
    if (rows == 0) return GSORT_OK;
    if (d_logits == nullptr || d_stats == nullptr || (top > 0 && (d_top_logprobs == nullptr || d_top_ids == nullptr)))
        return GSORT_EINVAL;
    const size_t size = float_bytes(dtype), n = static_cast<size_t>(rows);
    if (!aligned(d_logits, size) || !aligned(d_logprobs, 4) || !aligned(d_entropy, 4) || !aligned(d_stats, 8) ||
        !aligned(d_top_logprobs, 4) || !aligned(d_top_ids, 4) || (d_targets != nullptr && !aligned(d_targets, target_bytes)))
        return GSORT_EALIGN;
    const Span in[] = {rows_span(d_logits, rows, vocab, row_stride, size), {d_targets, n * target_bytes}};
    const Span out[] = {{d_logprobs, n * 4}, {d_entropy, n * 4}, {d_stats, n * 8},
                        {top > 0 ? d_top_logprobs : nullptr, n * top * 4}, {top > 0 ? d_top_ids : nullptr, n * top * 4}};
    if (clash(in, out)) return GSORT_EINVAL;
    DeviceInfo dev;
    if (device_info(&dev) != GSORT_OK) return GSORT_ECUDA;
    LogprobsLaunch L;
    L.logits = d_logits;
    L.dtype = dtype;
    L.rows = rows;
    L.vocab = vocab;
    L.row_stride = row_stride;
    L.targets = d_targets;
    L.target_bytes = target_bytes;
    L.top = top;
    L.logprobs = d_logprobs;
    L.entropy = d_entropy;
    L.stats = d_stats;
    L.top_logprobs = d_top_logprobs;
    L.top_ids = d_top_ids;
    L.stream = stream;
    L.sm_count = dev.sm_count;
    return launch_logprobs(L);
}

int gsort_token_logprobs_backward(const float *d_grad_logprobs, const float *d_grad_entropy,
                                  const void *d_logits, int dtype, int64_t rows, int64_t vocab,
                                  int64_t row_stride, const void *d_targets, int target_bytes,
                                  const float *d_entropy, const float *d_stats, void *d_grad_logits,
                                  int64_t grad_stride, cudaStream_t stream) {
    if (float_bytes(dtype) == 0) return GSORT_EINVAL;
    int rc = rows_args(rows, vocab, row_stride);
    if (rc == GSORT_OK) rc = rows_args(rows, vocab, grad_stride);
    if (rc != GSORT_OK) return rc;
    if (d_targets != nullptr && target_bytes != 4 && target_bytes != 8) return GSORT_EINVAL;
    if (rows == 0) return GSORT_OK;
    if (d_logits == nullptr || d_entropy == nullptr || d_stats == nullptr || d_grad_logits == nullptr) return GSORT_EINVAL;
    if (d_grad_logprobs != nullptr && d_targets == nullptr) return GSORT_EINVAL;
    const size_t size = float_bytes(dtype), n = static_cast<size_t>(rows);
    if (!aligned(d_logits, size) || !aligned(d_grad_logits, size) || !aligned(d_grad_logprobs, 4) || !aligned(d_grad_entropy, 4) ||
        !aligned(d_entropy, 4) || !aligned(d_stats, 8) || (d_targets != nullptr && !aligned(d_targets, target_bytes)))
        return GSORT_EALIGN;
    const bool in_place = d_grad_logits == d_logits && grad_stride == row_stride;
    const Span in[] = {in_place ? Span{nullptr, 0} : rows_span(d_logits, rows, vocab, row_stride, size),
                       {d_targets, n * target_bytes}, {d_grad_logprobs, n * 4}, {d_grad_entropy, n * 4},
                       {d_entropy, n * 4}, {d_stats, n * 8}};
    const Span out[] = {rows_span(d_grad_logits, rows, vocab, grad_stride, size)};
    if (clash(in, out)) return GSORT_EINVAL;
    LogprobsBackwardLaunch L;
    L.grad_logprobs = d_grad_logprobs;
    L.grad_entropy = d_grad_entropy;
    L.logits = d_logits;
    L.dtype = dtype;
    L.rows = rows;
    L.vocab = vocab;
    L.row_stride = row_stride;
    L.targets = d_targets;
    L.target_bytes = target_bytes;
    L.entropy = d_entropy;
    L.stats = d_stats;
    L.grad_logits = d_grad_logits;
    L.grad_stride = grad_stride;
    L.stream = stream;
    return launch_logprobs_backward(L);
}

int gsort_embed_tokens(const void *d_table, int dtype, int64_t vocab, int64_t width,
                       int64_t row_stride, const void *d_tokens, int token_bytes, int64_t tokens,
                       float scale, void *d_out, cudaStream_t stream) {
    int rc = embed_args(dtype, vocab, width, tokens, token_bytes, scale);
    if (rc == GSORT_OK) rc = rows_args(vocab, width, row_stride);
    if (rc != GSORT_OK || tokens == 0) return rc;
    if (d_table == nullptr || d_tokens == nullptr || d_out == nullptr) return GSORT_EINVAL;
    const size_t size = float_bytes(dtype);
    if (!aligned(d_table, size) || !aligned(d_out, size) || !aligned(d_tokens, token_bytes)) return GSORT_EALIGN;
    const Span in[] = {rows_span(d_table, vocab, width, row_stride, size), {d_tokens, static_cast<size_t>(tokens) * token_bytes}};
    const Span out[] = {rows_span(d_out, tokens, width, width, size)};
    if (clash(in, out)) return GSORT_EINVAL;
    EmbedLaunch L;
    L.in = d_table;
    L.dtype = dtype;
    L.vocab = vocab;
    L.width = width;
    L.in_stride = row_stride;
    L.tokens = d_tokens;
    L.token_bytes = token_bytes;
    L.n = tokens;
    L.scale = scale;
    L.out = d_out;
    L.stream = stream;
    return launch_embed(L);
}

int gsort_embed_tokens_backward(const void *d_grad_out, int dtype, int64_t tokens, int64_t width,
                                int64_t grad_stride, const void *d_tokens, int token_bytes,
                                int64_t vocab, float scale, int accumulate, void *d_grad_table,
                                int64_t table_stride, void *d_ws, size_t ws_bytes,
                                cudaStream_t stream) {
    return gsort_embed_tokens_backward_ex(d_grad_out, dtype, tokens, width, grad_stride, d_tokens, token_bytes, vocab, scale, accumulate,
                                          d_grad_table, table_stride, d_ws, ws_bytes, stream, nullptr);
}

size_t gsort_embed_tokens_backward_workspace_bytes(int64_t tokens, int64_t vocab, int64_t width, int dtype) {
    if (tokens < 1 || embed_args(dtype, vocab, width, tokens, 4, 1.0f) != GSORT_OK) return 0;
    return embed_workspace_bytes(tokens, vocab, width, dtype);
}

int gsort_embed_tokens_backward_ex(const void *d_grad_out, int dtype, int64_t tokens, int64_t width,
                                   int64_t grad_stride, const void *d_tokens, int token_bytes,
                                   int64_t vocab, float scale, int accumulate, void *d_grad_table,
                                   int64_t table_stride, void *d_ws, size_t ws_bytes,
                                   cudaStream_t stream, const gsort_options *options) {
    EmbedBackwardLaunch L;
    int rc = waits_of(options, &L.waits);
    if (rc == GSORT_OK) rc = embed_args(dtype, vocab, width, tokens, token_bytes, scale);
    if (rc == GSORT_OK) rc = rows_args(tokens, width, grad_stride);
    if (rc == GSORT_OK) rc = rows_args(vocab, width, table_stride);
    if (rc != GSORT_OK) return rc;
    if (tokens == 0 && accumulate != 0) return GSORT_OK;
    if (d_grad_table == nullptr || (tokens > 0 && (d_grad_out == nullptr || d_tokens == nullptr))) return GSORT_EINVAL;
    const size_t size = float_bytes(dtype);
    if (!aligned(d_grad_out, size) || !aligned(d_grad_table, size) || !aligned(d_tokens, token_bytes)) return GSORT_EALIGN;
    const size_t ws = gsort_embed_tokens_backward_workspace_bytes(tokens, vocab, width, dtype);
    if (ws > 0) {
        if (d_ws == nullptr || ws_bytes < ws) return GSORT_EWORKSPACE;
        if (!aligned(d_ws, kWsAlign)) return GSORT_EALIGN;
    }
    const Span in[] = {rows_span(d_grad_out, tokens, width, grad_stride, size), {d_tokens, static_cast<size_t>(tokens) * token_bytes}};
    const Span out[] = {rows_span(d_grad_table, vocab, width, table_stride, size), {ws > 0 ? d_ws : nullptr, ws}};
    if (clash(in, out)) return GSORT_EINVAL;
    DeviceInfo dev;
    if (device_info(&dev) != GSORT_OK) return GSORT_ECUDA;
    L.d_out = d_grad_out;
    L.dtype = dtype;
    L.n = tokens;
    L.width = width;
    L.d_stride = grad_stride;
    L.tokens = d_tokens;
    L.token_bytes = token_bytes;
    L.vocab = vocab;
    L.scale = scale;
    L.accumulate = accumulate != 0;
    L.d_table = d_grad_table;
    L.table_stride = table_stride;
    L.ws = static_cast<unsigned char *>(d_ws);
    L.stream = stream;
    L.sm_count = dev.sm_count;
    return launch_embed_backward(L);
}

int gsort_adjust_logits(const void *d_logits, int dtype, int64_t rows, int64_t vocab,
                        int64_t row_stride, const gsort_adjustments *how, void *d_out,
                        int64_t out_stride, cudaStream_t stream) {
    return adjust(false, nullptr, 0, d_logits, row_stride, dtype, rows, vocab, how, d_out, out_stride, stream, nullptr);
}

int gsort_adjust_logits_ex(const void *d_logits, int dtype, int64_t rows, int64_t vocab,
                           int64_t row_stride, const gsort_adjustments *how, void *d_out,
                           int64_t out_stride, cudaStream_t stream, const gsort_options *options) {
    return adjust(false, nullptr, 0, d_logits, row_stride, dtype, rows, vocab, how, d_out, out_stride, stream, options);
}

int gsort_adjust_logits_backward(const void *d_grad_out, int dtype, int64_t rows, int64_t vocab,
                                 int64_t grad_stride, const void *d_logits, int64_t row_stride,
                                 const gsort_adjustments *how, void *d_grad_logits,
                                 int64_t grad_logits_stride, cudaStream_t stream) {
    return adjust(true, d_logits, row_stride, d_grad_out, grad_stride, dtype, rows, vocab, how, d_grad_logits, grad_logits_stride, stream,
                  nullptr);
}

int gsort_adjust_logits_backward_ex(const void *d_grad_out, int dtype, int64_t rows, int64_t vocab,
                                    int64_t grad_stride, const void *d_logits, int64_t row_stride,
                                    const gsort_adjustments *how, void *d_grad_logits,
                                    int64_t grad_logits_stride, cudaStream_t stream,
                                    const gsort_options *options) {
    return adjust(true, d_logits, row_stride, d_grad_out, grad_stride, dtype, rows, vocab, how, d_grad_logits, grad_logits_stride, stream,
                  options);
}

size_t gsort_gradient_norm_workspace_bytes(int64_t tensors) {
    return tensors < 1 || tensors > GSORT_MAX_N ? 0 : norm_workspace_bytes(tensors);
}

int gsort_gradient_norm(const void *const *d_gradients, const int64_t *elements, const int *dtypes,
                        int64_t tensors, float *d_norm, void *d_ws, size_t ws_bytes,
                        cudaStream_t stream) {
    return norm(d_gradients, nullptr, elements, dtypes, tensors, INFINITY, 1.0f, d_norm, d_ws, ws_bytes, stream, nullptr);
}

int gsort_gradient_norm_ex(const void *const *d_gradients, const int64_t *elements, const int *dtypes,
                           int64_t tensors, float *d_norm, void *d_ws, size_t ws_bytes,
                           cudaStream_t stream, const gsort_options *options) {
    return norm(d_gradients, nullptr, elements, dtypes, tensors, INFINITY, 1.0f, d_norm, d_ws, ws_bytes, stream, options);
}

int gsort_clip_gradients(const void *const *d_gradients, void *const *d_out, const int64_t *elements,
                         const int *dtypes, int64_t tensors, float max_norm, float scale,
                         float *d_norm, void *d_ws, size_t ws_bytes, cudaStream_t stream) {
    if (tensors > 0 && d_out == nullptr) return GSORT_EINVAL;
    return norm(d_gradients, d_out, elements, dtypes, tensors, max_norm, scale, d_norm, d_ws, ws_bytes, stream, nullptr);
}

int gsort_clip_gradients_ex(const void *const *d_gradients, void *const *d_out, const int64_t *elements,
                            const int *dtypes, int64_t tensors, float max_norm, float scale,
                            float *d_norm, void *d_ws, size_t ws_bytes, cudaStream_t stream,
                            const gsort_options *options) {
    if (tensors > 0 && d_out == nullptr) return GSORT_EINVAL;
    return norm(d_gradients, d_out, elements, dtypes, tensors, max_norm, scale, d_norm, d_ws, ws_bytes, stream, options);
}

}  // extern "C"
