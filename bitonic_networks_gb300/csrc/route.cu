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
// L lanes (a power of two, at least k) hold one token, C experts each: lane l
// keeps experts [l * C, (l + 1) * C) in registers, so lower lanes hold lower
// indices and the tie rule is "lowest lane, then lowest slot".  64 experts take 4
// lanes, and a warp works on 8 tokens at once.  Each lane sorts its candidates;
// a pick is then a maximum over the lanes' best (redux.sync for a whole warp),
// one vote and the winner's next candidate.
//
// Bound by instructions, about 680 a token at 256 experts in groups with k = 8,
// not by its bytes: 16384 x 256 32-bit logits with bias and groups take 15.5 us, where
// reading them takes 2.5.
#include <algorithm>

#include "model_ops.cuh"

namespace gsort {
namespace {

constexpr int kRouteThreads = 128;

// A lane's C values of a row, -inf beyond the row's end.  `access` (1..16
// bytes): what the rows' alignment allows at once.
template <typename T, int C, int N>
__device__ __forceinline__ void load_values(const T *row, int experts, int e0, float (&x)[C]) {
#pragma unroll
    for (int b = 0; b < C; b += N) {
        if (e0 + b + N <= experts) {
            const Vec<T, N> v = *reinterpret_cast<const Vec<T, N> *>(row + e0 + b);
#pragma unroll
            for (int i = 0; i < N; ++i) x[b + i] = to_f32(v.e[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) x[b + i] = N > 1 && e0 + b + i < experts ? to_f32(row[e0 + b + i]) : kNegInf;
        }
    }
}

template <typename T, int C>
__device__ __forceinline__ void load_row(const T *row, int experts, int access, int e0, float (&x)[C]) {
    constexpr int kMost = 16 / sizeof(T) < C ? 16 / sizeof(T) : C;
    if (access >= 16) load_values<T, C, kMost>(row, experts, e0, x);
    else if (access >= 8) load_values<T, C, 8 / sizeof(T)>(row, experts, e0, x);
    else if (access >= 4) load_values<T, C, 4 / sizeof(T)>(row, experts, e0, x);
    else load_values<T, C, 1>(row, experts, e0, x);
}

template <typename T, int C, int N>
__device__ __forceinline__ void store_values(T *row, int experts, int e0, const float (&x)[C]) {
#pragma unroll
    for (int b = 0; b < C; b += N) {
        if (e0 + b + N <= experts) {
            Vec<T, N> v;
#pragma unroll
            for (int i = 0; i < N; ++i) v.e[i] = from_f32<T>(x[b + i]);
            *reinterpret_cast<Vec<T, N> *>(row + e0 + b) = v;
        } else if (N > 1) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (e0 + b + i < experts) row[e0 + b + i] = from_f32<T>(x[b + i]);
        }
    }
}

template <typename T, int C>
__device__ __forceinline__ void store_row(T *row, int experts, int access, int e0, const float (&x)[C]) {
    constexpr int kMost = 16 / sizeof(T) < C ? 16 / sizeof(T) : C;
    if (access >= 16) store_values<T, C, kMost>(row, experts, e0, x);
    else if (access >= 8) store_values<T, C, 8 / sizeof(T)>(row, experts, e0, x);
    else if (access >= 4) store_values<T, C, 4 / sizeof(T)>(row, experts, e0, x);
    else store_values<T, C, 1>(row, experts, e0, x);
}

// Reductions over a token's L lanes.
template <int L> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

template <int L> __device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}

template <int L> __device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if (L == 32) return __reduce_max_sync(kFullMask, v);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v = max(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}

// The lanes below this one that hold the same token.
template <int L> __device__ __forceinline__ uint32_t lanes_before(int lane) {
    return lanemask_lt() & ~((1u << (lane & ~(L - 1))) - 1u);
}

// Whether this is the token's first lane for which `p` holds.  The vote is the
// whole warp's: it is taken before `p` is looked at.
__device__ __forceinline__ bool is_first(bool p, uint32_t before) {
    const uint32_t votes = __ballot_sync(kFullMask, p);
    return p && (votes & before) == 0u;
}

// Sum over a token's row in one fixed order: neighbours first.
template <int C, int L> __device__ __forceinline__ float row_sum(const float (&v)[C]) {
    float t[C];
#pragma unroll
    for (int i = 0; i < C; ++i) t[i] = v[i];
#pragma unroll
    for (int w = 1; w < C; w *= 2)
#pragma unroll
        for (int i = 0; i < C; i += 2 * w) t[i] += t[i + w];
    return lanes_sum<L>(t[0]);
}

// e^(x - m) of a candidate: the difference is formed before expf multiplies it.
// The largest candidate has 1 even at +inf.
__device__ __forceinline__ float exp_from(float x, float m) { return x == m ? 1.0f : expf(x - m); }

// A softmax's score, each operation rounded to nearest: the product is not fused
// with what is added to it.
__device__ __forceinline__ float softmax_score(float x, float m, float inv) { return __fmul_rn(exp_from(x, m), inv); }

// e^(x - m) for a whole row, where only sums and a gradient's dense part are
// formed from it: 2 ulp and (m - x) 2^-23, and a third of the instructions.  What
// a sum gets of that is (m - x) e^(x - m) 2^-23 at most, below its own rounding;
// a dense part in 16 bits rounds to 2^-9 or 2^-12.  EXACT: a dense part in 32 bits.
template <bool EXACT, int C>
__device__ __forceinline__ void row_exp(const float (&x)[C], float m, float (&e)[C]) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const float d = x[i] == m ? 0.0f : x[i] - m;      // +inf - +inf
        e[i] = x[i] > kNegInf ? (EXACT ? exp_exact(d) : exp2_approx(d * kLog2e)) : 0.0f;
    }
}

// Largest candidate of the row (NaN is none); -inf where there is no candidate.
template <int C, int L> __device__ __forceinline__ float row_max(const float (&x)[C]) {
    float m = x[0] > kNegInf ? x[0] : kNegInf;
#pragma unroll
    for (int i = 1; i < C; ++i) m = x[i] > m ? x[i] : m;
    return lanes_max<L>(m);
}

// 1 / (1 + e^-x), each operation rounded to nearest: a choice among biased
// scores does not depend on how the quotient is formed.
__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(1.0f + expf(-x)); }

// e^-low * sigmoid(x) for low = min(0, the chosen experts' largest logit): scores
// to be renormalised, which do not underflow together.  A score below e^-745, the
// least number above 0 in 64 bits, is 0 all the same: a token whose experts are all
// masked by their type's lowest value has no weights, as with sigmoids formed in 64
// bits, and not equal ones.
__device__ __forceinline__ float raised_sigmoid(float x, float low) {
    return x > 0.0f ? sigmoid(x) : x < -745.0f ? 0.0f : expf(x - low) * __frcp_rn(1.0f + expf(x));
}

// 1 - sigmoid(x) without cancellation.
__device__ __forceinline__ float sigmoid_rest(float x) { return __frcp_rn(1.0f + expf(x)); }

struct RouteArgs {
    const void *logits;
    int64_t tokens, row_stride;
    const float *bias;
    float *weights;
    int32_t *experts_out;
    float scale;
    int experts, groups, groups_kept, group_size, chosen;
    int group_lanes;         // lanes to a group where each lane's experts are of one group, else 0
    uint32_t group_magic;    // ceil(2^21 / group_size): e / group_size = e * magic >> 21 for e < 1024
    int access, bias_access;
    bool softmax, top2, renormalise;
};

// Batcher's odd-even merge sort of C words in registers, largest first.  The
// recursion is over constants, so that every index is one.
template <int A, int B, int C> __device__ __forceinline__ void exchange(uint32_t (&v)[C]) {
    const uint32_t a = v[A], b = v[B];
    v[A] = max(a, b);
    v[B] = min(a, b);
}

template <int LO, int N, int STEP, int C, int I = LO + STEP> __device__ __forceinline__ void exchange_odd(uint32_t (&v)[C]) {
    if constexpr (I + STEP < LO + N) {
        exchange<I, I + STEP>(v);
        exchange_odd<LO, N, STEP, C, I + 2 * STEP>(v);
    }
}

// Merges the sorted halves of every STEP-th word of [LO, LO + N).
template <int LO, int N, int STEP, int C> __device__ __forceinline__ void merge_halves(uint32_t (&v)[C]) {
    if constexpr (2 * STEP < N) {
        merge_halves<LO, N, 2 * STEP>(v);
        merge_halves<LO + STEP, N, 2 * STEP>(v);
        exchange_odd<LO, N, STEP>(v);
    } else {
        exchange<LO, LO + STEP>(v);
    }
}

template <int LO, int N, int C> __device__ __forceinline__ void sort_desc(uint32_t (&v)[C]) {
    if constexpr (N > 1) {
        sort_desc<LO, N / 2>(v);
        sort_desc<LO + N / 2, N / 2>(v);
        merge_halves<LO, N, 1>(v);
    }
}

// The k best candidates by their full keys, each lane looking through all of
// its own for every pick; pick r's expert is left in picks[r], -1 beyond the
// candidates.  Rarely needed, but a whole launch may wait for one warp that
// does: without a branch in the loop over the slots it takes about a
// microsecond, with some it took eight.
template <int C, int L>
__device__ __forceinline__ void pick_exactly(uint32_t (&key)[C], int chosen, int lane, int32_t *picks) {
    const int e0 = (lane & (L - 1)) * C;
    const uint32_t before = lanes_before<L>(lane);
#pragma unroll 1
    for (int r = 0; r < chosen; ++r) {
        uint32_t best = 0u;
        int slot = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            slot = key[i] > best ? i : slot;
            best = max(best, key[i]);
        }
        const uint32_t top = lanes_max<L>(best);
        const bool won = is_first(best == top, before);
        if (won) picks[r] = top != 0u ? e0 + slot : -1;
        slot = won ? slot : -1;
#pragma unroll
        for (int i = 0; i < C; ++i) key[i] = i == slot ? 0u : key[i];
    }
}

// The same with one word for a candidate: its key with the last bits given to
// the slot, lower slots first.  Each lane sorts its words beforehand and keeps
// them in shared memory, so that a pick is a maximum, a vote, and the winner's
// next word.  Returns whether keys that differ in the bits given up met: two
// picks one after the other, or the last and what is left, are then equal in
// the others.
template <int C, int L>
__device__ __forceinline__ bool pick_sorted(const uint32_t (&key)[C], int chosen, int lane, uint32_t *words, int32_t *picks) {
    constexpr uint32_t kSlot = C - 1;
    const int e0 = (lane & (L - 1)) * C;
    const uint32_t before = lanes_before<L>(lane);
    uint32_t v[C];
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = (key[i] & ~kSlot) | (kSlot - i);    // up to kSlot: no candidate
    sort_desc<0, C>(v);
    uint32_t *mine = words + lane * (C + 1);
#pragma unroll
    for (int i = 0; i < C; ++i) mine[i] = v[i];
    mine[C] = 0u;
    uint32_t head = v[0], last = ~0u;
    int next = 1;
    bool met = false;
#pragma unroll 1
    for (int r = 0; r < chosen; ++r) {
        const uint32_t top = lanes_max<L>(head);
        met |= (top ^ last) <= kSlot;
        last = top > kSlot ? top : ~0u;
        if (is_first((head ^ top) <= kSlot, before)) {
            picks[r] = head > kSlot ? e0 + static_cast<int>(kSlot - (head & kSlot)) : -1;
            head = mine[min(next++, C)];
        }
    }
    return met | ((lanes_max<L>(head) ^ last) <= kSlot);
}

template <typename T, int C, int L>
__global__ void __launch_bounds__(kRouteThreads) k_route(const RouteArgs a) {
    __shared__ uint32_t s_words[kRouteThreads / 32][32 * (C + 1)];
    __shared__ int32_t s_picks[kRouteThreads];       // a token's picks, one for each of its lanes
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & (L - 1);
    const int64_t token = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / L) + threadIdx.x / L;
    const bool live = token < a.tokens;      // every lane goes through the warp's votes
    const T *row = static_cast<const T *>(a.logits) + (live ? token : 0) * a.row_stride;
    const int e0 = sub * C;

    float x[C];
    load_row<T, C>(row, a.experts, a.access, e0, x);

    const bool biased = a.bias != nullptr;
    float m = kNegInf, inv = 0.0f;       // softmax: the row's largest logit and 1 / sum
    float c[C];
    if (a.softmax && (biased || !a.renormalise || (a.groups > 1 && a.top2))) {
        m = row_max<C, L>(x);
        row_exp<false, C>(x, m, c);
        const float sum = row_sum<C, L>(c);
        inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    }

    // order keys of the choice values; 0: no candidate
    uint32_t key[C];
    if (biased) {
        // the scores that the weights are made of, to the last bit: near ties are theirs to decide
        if (a.softmax) {
#pragma unroll
            for (int i = 0; i < C; ++i) c[i] = x[i] > kNegInf ? softmax_score(x[i], m, inv) : 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i) c[i] = sigmoid(x[i]);
        }
        float b[C];
        load_row<float, C>(a.bias, a.experts, a.bias_access, e0, b);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float v = c[i] + b[i];
            key[i] = x[i] > kNegInf && v > kNegInf ? order_key(v) : 0u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) key[i] = x[i] > kNegInf ? order_key(x[i]) : 0u;
    }

    if (a.groups > 1) {
        // the two largest keys of a group; scores grow with their keys
        const int per = a.group_lanes > 0 ? a.group_lanes : 1, g = sub / per;
        uint32_t first = 0u, second = 0u;
        if (a.group_lanes > 0) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                second = max(second, min(first, key[i]));
                first = max(first, key[i]);
            }
            for (int o = 1; o < per; o <<= 1) {
                const uint32_t f = __shfl_xor_sync(kFullMask, first, o), s = __shfl_xor_sync(kFullMask, second, o);
                second = max(max(second, s), min(first, f));
                first = max(first, f);
            }
        } else {
            // groups that end inside a lane: lane g reads group g's keys (there are as many lanes)
            uint32_t *sk = s_words[warp];
#pragma unroll
            for (int i = 0; i < C; ++i) sk[lane * (C + 1) + i] = key[i];
            __syncwarp();
            if (g < a.groups)
                for (int i = 0; i < a.group_size; ++i) {
                    const int e = (lane & ~(L - 1)) * C + g * a.group_size + i;
                    const uint32_t v = sk[e / C * (C + 1) + e % C];
                    second = max(second, min(first, v));
                    first = max(first, v);
                }
            __syncwarp();
        }
        uint32_t gkey = 0u;
        if (g < a.groups && first != 0u && sub % per == 0) {
            if (!a.top2) {
                gkey = first;
            } else {
                float value = order_key_value(first), other = order_key_value(second);
                if (!biased && a.softmax) value = softmax_score(value, m, inv), other = softmax_score(other, m, inv);
                if (!biased && !a.softmax) value = sigmoid(value), other = sigmoid(other);
                gkey = order_key(second != 0u ? value + other : value);
            }
        }
        bool keep = false;       // in a group's first lane: it is one of the best
        const uint32_t before = lanes_before<L>(lane);
        for (int r = 0; r < a.groups_kept; ++r) {
            const uint32_t top = lanes_max<L>(gkey);
            if (is_first(gkey == top, before) && top != 0u) {
                keep = true;
                gkey = 0u;
            }
        }
        if (a.group_lanes > 0) {
            keep = __shfl_sync(kFullMask, keep, lane & ~(per - 1));
#pragma unroll
            for (int i = 0; i < C; ++i) key[i] = keep ? key[i] : 0u;
        } else {
            const uint32_t kept = __ballot_sync(kFullMask, keep) >> (lane & ~(L - 1));
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const uint32_t gi = (static_cast<uint32_t>(e0 + i) * a.group_magic) >> 21;
                if (gi >= static_cast<uint32_t>(L) || !((kept >> gi) & 1u)) key[i] = 0u;
            }
        }
    }

    int32_t *picks = s_picks + (threadIdx.x & ~(L - 1));
    const bool met = pick_sorted<C, L>(key, a.chosen, lane, s_words[warp], picks);
    // 16-bit logits have no bits there: equal words are equal logits
    __syncwarp();
    if ((sizeof(T) == 4 || biased) && __any_sync(kFullMask, met)) {
        pick_exactly<C, L>(key, a.chosen, lane, picks);
        __syncwarp();
    }
    const int mine = sub < a.chosen ? picks[sub] : -1;

    // the chosen experts' weights
    float w = 0.0f;
    const bool there = mine >= 0;
    const float xe = there ? to_f32(row[mine]) : kNegInf;
    if (a.softmax) {
        if (a.renormalise) {     // a softmax over the chosen alone
            const float mc = lanes_max<L>(xe);
            w = there ? exp_from(xe, mc) : 0.0f;
        } else if (there) {
            w = softmax_score(xe, m, inv);
        }
    } else {
        const float low = a.renormalise ? fminf(lanes_max<L>(xe), 0.0f) : 0.0f;
        w = !there ? 0.0f : a.renormalise ? raised_sigmoid(xe, low) : sigmoid(xe);
    }
    if (a.renormalise) {
        const float total = lanes_sum<L>(w);
        // a quotient, not a product with 1 / total: one expert alone has exactly 1
        if (there) w = total > 0.0f ? w / total : 0.0f;
    }
    if (live && sub < a.chosen) {
        a.weights[token * a.chosen + sub] = w * a.scale;
        a.experts_out[token * a.chosen + sub] = mine;
    }
}

struct RouteBackwardArgs {
    const float *grad_weights;
    const void *logits;
    int64_t tokens, row_stride;
    const int32_t *experts_in;
    void *grad_logits;
    float scale;
    int experts, chosen, access, access_out;
    bool softmax, renormalise;
};

// Gradient of the weights by the logits, pick j in the token's lane j, with dw
// scaled:
//   softmax                 dx_e = p_e * (dw_e [chosen] - sum_j dw_j p_j)
//   softmax, renormalised   dx_j = q_j * (dw_j - sum_i dw_i q_i), chosen only
//   sigmoid                 dx_j = dw_j * s_j (1 - s_j), chosen only
//   sigmoid, renormalised   dx_j = (dw_j - sum_i dw_i q_i) * q_j (1 - s_j)
// The choice itself, the groups and the bias have no gradient.  The dense row
// is written first (zeros, or -p_e times the sum), then the chosen entries.
template <typename T, int C, int L>
__global__ void __launch_bounds__(kRouteThreads) k_route_backward(const RouteBackwardArgs a) {
    const int sub = threadIdx.x & (L - 1);
    const int64_t token = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / L) + threadIdx.x / L;
    const bool live = token < a.tokens;
    const T *row = static_cast<const T *>(a.logits) + (live ? token : 0) * a.row_stride;
    T *out = static_cast<T *>(a.grad_logits) + (live ? token : 0) * a.experts;
    const int e0 = sub * C;

    int e = -1;
    float d = 0.0f, xe = kNegInf;
    if (live && sub < a.chosen) {
        e = a.experts_in[token * a.chosen + sub];
        if (e >= 0 && e < a.experts) {
            xe = to_f32(row[e]);
            d = a.grad_weights[token * a.chosen + sub] * a.scale;
        }
    }
    const bool there = xe > kNegInf;
    if (!there) d = 0.0f;

    float g = 0.0f;          // gradient of the chosen entry
    float dense[C];
#pragma unroll
    for (int i = 0; i < C; ++i) dense[i] = 0.0f;
    if (!a.softmax) {
        if (a.renormalise) {
            const float low = fminf(lanes_max<L>(xe), 0.0f), t = there ? raised_sigmoid(xe, low) : 0.0f;
            const float total = lanes_sum<L>(t);
            float q = 0.0f;          // a quotient: of one expert alone it is 1 and the gradient 0
            if (there && total > 0.0f) q = t / total;
            g = (d - lanes_sum<L>(d * q)) * q * sigmoid_rest(xe);
        } else {
            g = there ? d * sigmoid(xe) * sigmoid_rest(xe) : 0.0f;
        }
    } else if (a.renormalise) {
        const float m = lanes_max<L>(there ? xe : kNegInf);
        const float q0 = there ? exp_from(xe, m) : 0.0f;
        const float total = lanes_sum<L>(q0);
        float q = 0.0f;
        if (there) q = q0 / total;       // the largest adds 1 to the total
        const float mean = lanes_sum<L>(d * q);
        g = q * (d - mean);
    } else {
        float x[C];
        load_row<T, C>(row, a.experts, a.access, e0, x);
        const float m = row_max<C, L>(x);
        row_exp<sizeof(T) == 4, C>(x, m, dense);
        const float sum = row_sum<C, L>(dense);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        const float p = there ? exp_from(xe, m) * inv : 0.0f;
        const float mean = lanes_sum<L>(d * p);
        g = p * (d - mean);
#pragma unroll
        for (int i = 0; i < C; ++i) dense[i] = -(dense[i] * inv) * mean;
    }
    if (live) store_row<T, C>(out, a.experts, a.access_out, e0, dense);
    __syncwarp();            // the rows' stores come before the chosen entries'
    if (there) out[e] = from_f32<T>(g);
}

// Bytes, up to 16, that rows of T at `base`, `stride` apart, can move at once.
template <typename T> int access_of(const void *base, int64_t stride) {
    int bytes = 16;
    while (bytes > static_cast<int>(sizeof(T)) && !(aligned(base, bytes) && static_cast<size_t>(stride) * sizeof(T) % bytes == 0)) bytes /= 2;
    return bytes;
}

// Calls f with (C, L), at least `lanes` lanes to a token.  Measured, routing of
// bf16 logits with k = 8 in us:
//   up to 1024 tokens every one gets a warp, with redux.sync instead of shuffles
//   (256 experts, a warp / 16 lanes to a token: 8 tokens 2.3 / 3.0, 1024 2.7 / 3.2, 4096 4.4 /
//   4.6, 8192 6.8 / 6.4; 60 experts: 1024 2.8 / 3.3, 2048 3.3 / 3.3, 4096 4.6 / 3.6);
//   16 experts to a lane from 33 experts on (65536 x 128: 15 against 23 with 8,
//   x 256: 31 against 40), 8 up to 32 experts (x 16, k = 2: 5.2 against 7.3),
//   32 only where they must be.
template <typename F> int with_shape(int64_t tokens, int experts, int lanes, F &&f) {
    using std::integral_constant;
    if (tokens <= 1024 && experts <= 256) return f(integral_constant<int, 8>{}, integral_constant<int, 32>{});
    if (experts <= 32 && lanes <= 4) return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
    if (experts <= 32 && lanes <= 8) return f(integral_constant<int, 8>{}, integral_constant<int, 8>{});
    const int need = std::max((experts + 15) / 16, lanes);
    if (need <= 4) return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    if (need <= 8) return f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
    if (need <= 16) return f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    if (need <= 32) return f(integral_constant<int, 16>{}, integral_constant<int, 32>{});
    return f(integral_constant<int, 32>{}, integral_constant<int, 32>{});
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
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        // without whole lanes to a group, a lane reads each group: as many lanes as groups
        return with_shape(L.tokens, L.experts, std::max(L.chosen, L.groups), [&](auto slots, auto lanes) {
            constexpr int C = decltype(slots)::value, W = decltype(lanes)::value;
            a.access = access_of<T>(L.logits, L.row_stride);
            a.bias_access = access_of<float>(L.bias, 0);
            const int per = a.group_size / C;
            a.group_lanes = a.group_size % C == 0 && (per & (per - 1)) == 0 ? per : 0;
            const uint32_t grid = static_cast<uint32_t>((L.tokens + kRouteThreads / W - 1) / (kRouteThreads / W));
            k_route<T, C, W><<<grid, kRouteThreads, 0, L.stream>>>(a);
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
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        return with_shape(L.tokens, L.experts, L.chosen, [&](auto slots, auto lanes) {
            constexpr int C = decltype(slots)::value, W = decltype(lanes)::value;
            a.access = access_of<T>(L.logits, L.row_stride);
            a.access_out = access_of<T>(L.grad_logits, L.experts);
            const uint32_t grid = static_cast<uint32_t>((L.tokens + kRouteThreads / W - 1) / (kRouteThreads / W));
            k_route_backward<T, C, W><<<grid, kRouteThreads, 0, L.stream>>>(a);
            return cudaGetLastError() == cudaSuccess ? GSORT_OK : GSORT_ECUDA;
        });
    });
}

}  // namespace gsort
