// route.cu -- routing of tokens to experts, and its gradient.
//
// Per token, over E experts with logits x (read once, 32-bit arithmetic):
//   candidate   x > -inf (so -inf and NaN take no part)
//   score s     softmax over the candidates, or 1 / (1 + e^-x)
//   choice c    x where there is no bias (s grows with x), else s + bias
//   groups      E / G consecutive experts each; a group's value is its largest
//               c, or the sum of its two largest s (+ bias); only experts of
//               the best groups stay candidates
//   chosen      the k largest c, ties to the lower index
//   weight      s * scale, or s / (sum of the chosen s) * scale
//
// One warp holds one token: lane l keeps experts [l * C, (l + 1) * C) in
// registers, so lower lanes hold lower indices and the tie rule is "lowest
// lane, then lowest slot".  A pick is one warp-wide integer maximum
// (redux.sync) of 32-bit order keys, one ballot and one shuffle.
#include <algorithm>

#include "model_ops.cuh"

namespace gsort {
namespace {

constexpr int kRouteWarps = 4;

// A warp's row of E values, C per lane, -inf beyond the row's end.
template <typename T, int C>
__device__ __forceinline__ void load_row(const T *row, int experts, bool wide, int lane, float (&x)[C]) {
    const int e0 = lane * C;
    constexpr int N = C * sizeof(T) <= 16 ? C : static_cast<int>(16 / sizeof(T));
    if (wide && e0 + C <= experts) {
#pragma unroll
        for (int b = 0; b < C; b += N) {
            const Vec<T, N> v = *reinterpret_cast<const Vec<T, N> *>(row + e0 + b);
#pragma unroll
            for (int i = 0; i < N; ++i) x[b + i] = to_f32(v.e[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) x[i] = e0 + i < experts ? to_f32(row[e0 + i]) : kNegInf;
    }
}

// Sum over the warp's row in one fixed order: neighbours first.
template <int C> __device__ __forceinline__ float row_sum(const float (&v)[C]) {
    float t[C];
#pragma unroll
    for (int i = 0; i < C; ++i) t[i] = v[i];
#pragma unroll
    for (int w = 1; w < C; w *= 2)
#pragma unroll
        for (int i = 0; i < C; i += 2 * w) t[i] += t[i + w];
    float s = t[0];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) s += __shfl_xor_sync(kFullMask, s, o);
    return s;
}

// Exponentials e^(x - m) of a row's candidates; x - m is exact enough because
// it is formed before the multiplication inside expf.
template <int C>
__device__ __forceinline__ void row_exp(const float (&x)[C], float m, float (&e)[C]) {
#pragma unroll
    for (int i = 0; i < C; ++i) e[i] = x[i] > kNegInf ? (x[i] == m ? 1.0f : expf(x[i] - m)) : 0.0f;
}

// Largest candidate of the row (NaN is none); -inf where there is no candidate.
template <int C> __device__ __forceinline__ float row_max(const float (&x)[C]) {
    float m = x[0] > kNegInf ? x[0] : kNegInf;
#pragma unroll
    for (int i = 1; i < C; ++i) m = x[i] > m ? x[i] : m;
    return warp_max(m);
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

struct RouteArgs {
    const void *logits;
    int64_t tokens, row_stride;
    const float *bias;
    float *weights;
    int32_t *experts_out;
    float scale;
    int experts, groups, groups_kept, group_size, chosen;
    uint32_t group_magic;    // ceil(2^21 / group_size): e / group_size = e * magic >> 21 for e < 1024
    bool softmax, top2, renormalise, wide;
};

template <typename T, int C>
__global__ void __launch_bounds__(kRouteWarps * 32) k_route(const RouteArgs a) {
    // group values are read by other lanes; one word of padding for 32
    __shared__ float s_value[kRouteWarps][C * 33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t token = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
    if (token >= a.tokens) return;   // whole warp: no block-wide barrier below
    const T *row = static_cast<const T *>(a.logits) + token * a.row_stride;
    const int e0 = lane * C;

    float x[C], c[C];
    load_row<T, C>(row, a.experts, a.wide, lane, x);

    const bool biased = a.bias != nullptr;
    const bool by_score = a.groups > 1 && a.top2;
    float m = kNegInf, sum = 0.0f;
    if (a.softmax && (biased || by_score || !a.renormalise)) {
        m = row_max<C>(x);
        float e[C];
        row_exp<C>(x, m, e);
        sum = row_sum<C>(e);
#pragma unroll
        for (int i = 0; i < C; ++i) c[i] = e[i] / sum;
    } else if (!a.softmax && (biased || by_score)) {
#pragma unroll
        for (int i = 0; i < C; ++i) c[i] = sigmoid(x[i]);
    }
    if (biased) {
#pragma unroll
        for (int i = 0; i < C; ++i) c[i] += e0 + i < a.experts ? a.bias[e0 + i] : 0.0f;
    }
    // order keys of the choice values; 0: no candidate
    uint32_t key[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const float v = biased ? c[i] : x[i];
        key[i] = x[i] > kNegInf && v > kNegInf ? order_key(v) : 0u;
    }

    if (a.groups > 1) {
        float *sv = s_value[warp];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int e = e0 + i;
            sv[e + (e >> 5)] = key[i] == 0u ? kNegInf : (biased || by_score) ? c[i] : x[i];
        }
        __syncwarp();
        // `per` lanes to a group, a power of two
        int per = 1;
        while (per * 2 * a.groups <= 32) per *= 2;
        const int g = lane / per, sub = lane % per;
        float first = kNegInf, second = kNegInf;
        if (g < a.groups) {
            for (int i = sub; i < a.group_size; i += per) {
                const int e = g * a.group_size + i;
                const float v = sv[e + (e >> 5)];
                second = fmaxf(second, fminf(first, v));
                first = fmaxf(first, v);
            }
        }
        for (int o = 1; o < per; o <<= 1) {
            const float f = __shfl_xor_sync(kFullMask, first, o), s = __shfl_xor_sync(kFullMask, second, o);
            second = fmaxf(fmaxf(second, s), fminf(first, f));
            first = fmaxf(first, f);
        }
        float value = first;
        if (a.top2 && second > kNegInf) value += second;
        uint32_t gkey = g < a.groups && sub == 0 && first > kNegInf ? order_key(value) : 0u;
        uint32_t kept = 0;
        for (int r = 0; r < a.groups_kept; ++r) {
            const uint32_t best = __reduce_max_sync(kFullMask, gkey);
            if (best == 0u) break;
            const int src = __ffs(__ballot_sync(kFullMask, gkey == best)) - 1;
            kept |= 1u << (src / per);
            if (lane == src) gkey = 0u;
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const uint32_t gi = (static_cast<uint32_t>(e0 + i) * a.group_magic) >> 21;
            if (gi >= 32u || !((kept >> gi) & 1u)) key[i] = 0u;
        }
    }

    // k picks: the lane's best candidate, then the warp's
    int mine = -1;           // the pick that this lane keeps: number `lane`
    uint32_t best = 0u;
    int slot = 0;
#pragma unroll
    for (int i = 0; i < C; ++i)
        if (key[i] > best) best = key[i], slot = i;
    for (int r = 0; r < a.chosen; ++r) {
        const uint32_t top = __reduce_max_sync(kFullMask, best);
        if (top == 0u) break;
        const int src = __ffs(__ballot_sync(kFullMask, best == top)) - 1;
        const int e = __shfl_sync(kFullMask, e0 + slot, src);
        if (lane == r) mine = e;
        if (lane == src) {
            const int old = slot;
            best = 0u;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (i == old) key[i] = 0u;
                if (key[i] > best) best = key[i], slot = i;
            }
        }
    }

    // the chosen experts' weights, pick r in lane r
    float w = 0.0f;
    const float xe = mine >= 0 ? to_f32(row[mine]) : kNegInf;
    if (a.softmax) {
        if (a.renormalise) {     // a softmax over the chosen alone
            const float mc = warp_max(xe);
            const float e = mine >= 0 ? (xe == mc ? 1.0f : expf(xe - mc)) : 0.0f;
            const float total = warp_sum(e);
            w = total > 0.0f ? e / total : 0.0f;
        } else if (mine >= 0) {
            w = (xe == m ? 1.0f : expf(xe - m)) / sum;
        }
    } else {
        w = mine >= 0 ? sigmoid(xe) : 0.0f;
        if (a.renormalise) {
            const float total = warp_sum(w);
            w = total > 0.0f ? w / total : 0.0f;
        }
    }
    if (lane < a.chosen) {
        a.weights[token * a.chosen + lane] = w * a.scale;
        a.experts_out[token * a.chosen + lane] = mine;
    }
}

struct RouteBackwardArgs {
    const float *grad_weights;
    const void *logits;
    int64_t tokens, row_stride;
    const int32_t *experts_in;
    void *grad_logits;
    float scale;
    int experts, chosen;
    bool softmax, renormalise, wide, wide_out;
};

// Gradient of the weights by the logits, pick j in lane j, with dw scaled:
//   softmax                 dx_e = p_e * (dw_e [chosen] - sum_j dw_j p_j)
//   softmax, renormalised   dx_j = q_j * (dw_j - sum_i dw_i q_i), chosen only
//   sigmoid                 dx_j = dw_j * s_j (1 - s_j), chosen only
//   sigmoid, renormalised   dx_j = (dw_j - sum_i dw_i q_i) / S * s_j (1 - s_j)
// The choice itself, the groups and the bias have no gradient.  The dense row
// is written first (zeros, or -p_e times the sum), then the chosen entries.
template <typename T, int C>
__global__ void __launch_bounds__(kRouteWarps * 32) k_route_backward(const RouteBackwardArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t token = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
    if (token >= a.tokens) return;
    const T *row = static_cast<const T *>(a.logits) + token * a.row_stride;
    T *out = static_cast<T *>(a.grad_logits) + token * a.experts;
    const int e0 = lane * C;

    int e = -1;
    float d = 0.0f, xe = kNegInf;
    if (lane < a.chosen) {
        e = a.experts_in[token * a.chosen + lane];
        if (e >= 0 && e < a.experts) {
            xe = to_f32(row[e]);
            d = a.grad_weights[token * a.chosen + lane] * a.scale;
        } else {
            e = -1;
        }
    }
    const bool there = e >= 0 && xe > kNegInf;
    if (!there) d = 0.0f;

    float g = 0.0f;          // gradient of the chosen entry
    float dense[C];
#pragma unroll
    for (int i = 0; i < C; ++i) dense[i] = 0.0f;
    if (!a.softmax) {
        const float s = there ? sigmoid(xe) : 0.0f;
        const float slope = there ? s * (1.0f / (1.0f + expf(xe))) : 0.0f;   // s (1 - s) without cancellation
        if (a.renormalise) {
            const float total = warp_sum(s);
            const float mean = warp_sum(total > 0.0f ? d * (s / total) : 0.0f);
            g = total > 0.0f ? (d - mean) / total * slope : 0.0f;
        } else {
            g = d * slope;
        }
    } else if (a.renormalise) {
        const float m = warp_max(there ? xe : kNegInf);
        const float q0 = there ? (xe == m ? 1.0f : expf(xe - m)) : 0.0f;
        const float total = warp_sum(q0);
        const float q = total > 0.0f ? q0 / total : 0.0f;
        const float mean = warp_sum(d * q);
        g = q * (d - mean);
    } else {
        float x[C], ex[C];
        load_row<T, C>(row, a.experts, a.wide, lane, x);
        const float m = row_max<C>(x);
        row_exp<C>(x, m, ex);
        const float sum = row_sum<C>(ex);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        const float p = there ? (xe == m ? 1.0f : expf(xe - m)) * inv : 0.0f;
        const float mean = warp_sum(d * p);
        g = p * (d - mean);
#pragma unroll
        for (int i = 0; i < C; ++i) dense[i] = -(ex[i] * inv) * mean;
    }

    constexpr int N = C * sizeof(T) <= 16 ? C : static_cast<int>(16 / sizeof(T));
    if (a.wide_out && e0 + C <= a.experts) {
#pragma unroll
        for (int b = 0; b < C; b += N) {
            Vec<T, N> v;
#pragma unroll
            for (int i = 0; i < N; ++i) v.e[i] = from_f32<T>(dense[b + i]);
            *reinterpret_cast<Vec<T, N> *>(out + e0 + b) = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (e0 + i < a.experts) out[e0 + i] = from_f32<T>(dense[i]);
    }
    __syncwarp();            // the row's stores come before the chosen entries'
    if (there) out[e] = from_f32<T>(g);
}

// Whether rows of `experts` T at `base`, `stride` apart, can move as the
// vectors of a lane with `per_lane` experts.
template <typename T> bool wide_rows(const void *base, int64_t stride, int per_lane) {
    const size_t bytes = std::min<size_t>(16, per_lane * sizeof(T));
    return aligned(base, bytes) && (static_cast<size_t>(stride) * sizeof(T)) % bytes == 0;
}

// Calls f with the smallest power of two C for which 32 * C >= experts.
template <typename F> int with_slots(int experts, F &&f) {
    if (experts <= 32) return f(std::integral_constant<int, 1>{});
    if (experts <= 64) return f(std::integral_constant<int, 2>{});
    if (experts <= 128) return f(std::integral_constant<int, 4>{});
    if (experts <= 256) return f(std::integral_constant<int, 8>{});
    if (experts <= 512) return f(std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{});
}

}  // namespace

int launch_route(const RouteLaunch &L) {
    RouteArgs a{};
    a.logits = L.logits;
    a.tokens = L.tokens;
    a.row_stride = L.row_stride;
    a.bias = L.bias;
    a.weights = L.weights;
    a.experts_out = L.experts_out;
    a.scale = L.scale;
    a.experts = L.experts;
    a.groups = L.groups;
    a.groups_kept = L.groups_kept;
    a.group_size = L.experts / L.groups;
    a.group_magic = ((1u << 21) + a.group_size - 1) / a.group_size;
    a.chosen = L.chosen;
    a.softmax = L.score == GSORT_SCORE_SOFTMAX;
    a.top2 = L.group_score == GSORT_GROUP_TOP2;
    a.renormalise = L.renormalise;
    const uint32_t grid = static_cast<uint32_t>((L.tokens + kRouteWarps - 1) / kRouteWarps);
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        return with_slots(L.experts, [&](auto slots) {
            constexpr int C = decltype(slots)::value;
            a.wide = wide_rows<T>(L.logits, L.row_stride, C);
            k_route<T, C><<<grid, kRouteWarps * 32, 0, L.stream>>>(a);
            return cudaGetLastError() == cudaSuccess ? GSORT_OK : GSORT_ECUDA;
        });
    });
}

int launch_route_backward(const RouteBackwardLaunch &L) {
    RouteBackwardArgs a{};
    a.grad_weights = L.grad_weights;
    a.logits = L.logits;
    a.tokens = L.tokens;
    a.row_stride = L.row_stride;
    a.experts_in = L.experts_in;
    a.grad_logits = L.grad_logits;
    a.scale = L.scale;
    a.experts = L.experts;
    a.chosen = L.chosen;
    a.softmax = L.score == GSORT_SCORE_SOFTMAX;
    a.renormalise = L.renormalise;
    const uint32_t grid = static_cast<uint32_t>((L.tokens + kRouteWarps - 1) / kRouteWarps);
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        return with_slots(L.experts, [&](auto slots) {
            constexpr int C = decltype(slots)::value;
            a.wide = wide_rows<T>(L.logits, L.row_stride, C);
            a.wide_out = wide_rows<T>(L.grad_logits, L.experts, C);
            k_route_backward<T, C><<<grid, kRouteWarps * 32, 0, L.stream>>>(a);
            return cudaGetLastError() == cudaSuccess ? GSORT_OK : GSORT_ECUDA;
        });
    });
}

}  // namespace gsort
