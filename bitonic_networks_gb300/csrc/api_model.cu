// api_model.cu -- the extern "C" boundary of the language-model operators:
// argument checks before any CUDA call, then one launcher.
#include <algorithm>
#include <cmath>

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

}  // extern "C"
