// logprobs.cu -- log probabilities of given tokens, the distribution's entropy
// and its most likely tokens, from one read of the logits; and the gradient.
//
// Per row x of V logits (-inf: masked), with m = max x, d_i = x_i - m:
//   S = sum e^d_i,  U = sum e^d_i d_i
//   log p_i = d_i - ln S,   H = ln S - U / S
//   gradient of g log p_t + h H:  g [i = t] - p_i (g + h (log p_i + H))
// A row without a logit above -inf has S = 0: log p = -inf, H = 0, no gradient.
// NaN and +inf in a row make its results NaN.
//
// The forward pass keeps a running maximum per thread and rescales its sums
// when the maximum grows, so a row is read once.  The largest logits are found
// in the same pass: the first 16,384 16-bit (8,192 32-bit) logits give a
// threshold that at least `top` of them reach, and only logits above it are
// written to a shared buffer, which is sorted by warps (bitonic networks of 32)
// when the row ends or the buffer fills.  Few rows are split over a cluster of
// CTAs, joined through distributed shared memory.
#include <algorithm>

#include "model_ops.cuh"

namespace gsort {
namespace {

#ifndef LP_THREADS
#define LP_THREADS 256
#define LP_VECTORS 4
#define LP_CTAS 4
#endif
constexpr int kLpThreads = LP_THREADS;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpVectors = LP_VECTORS;     // 16-byte vectors per thread and step
constexpr int kLpCtas = LP_CTAS;           // CTAs per SM that the registers allow
constexpr uint32_t kLpStep = kLpThreads * kLpVectors;
constexpr int kGroupLanes = kLpThreads / 32;   // 32 groups of lanes give the first threshold
constexpr uint32_t kCandidates = 2048;     // shared buffer of candidates
constexpr int kMaxCluster = 8;
constexpr float kLowLogit = -1e37f;        // x - max above it: the exponent does not overflow
constexpr float kTinyExponent = -256.0f;   // 2^-256 is 0 in 32 bits: masked logits add e^d * d = 0 * -256

// A candidate: order key of the logit, then the lower index first.
__device__ __forceinline__ uint64_t candidate(float x, uint32_t index) {
    return (static_cast<uint64_t>(order_key(x)) << 32) | (0xFFFFFFFFu - index);
}

__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// Merges a bitonic sequence, one element per lane, into descending order.
__device__ __forceinline__ uint64_t bitonic_merge_desc(uint64_t v, int lane) {
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) {
        const uint64_t o = __shfl_xor_sync(kFullMask, v, j);
        const bool upper = (lane & j) != 0;
        v = (v > o) != upper ? v : o;
    }
    return v;
}

__device__ __forceinline__ uint64_t bitonic_sort_desc(uint64_t v, int lane) {
#pragma unroll
    for (int k = 2; k < 32; k <<= 1) {
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const uint64_t o = __shfl_xor_sync(kFullMask, v, j);
            const bool upper = ((lane & j) != 0) != ((lane & k) != 0);
            v = (v > o) != upper ? v : o;
        }
    }
    return bitonic_merge_desc(v, lane);
}

// The 32 largest of two descending lists, descending.
__device__ __forceinline__ uint64_t merge_lists(uint64_t a, uint64_t b, int lane) {
    return bitonic_merge_desc(max64(a, __shfl_sync(kFullMask, b, 31 - lane)), lane);
}

// Sums over a part of a row with running maximum `max`, in powers of two:
// S = sum 2^y, U = sum 2^y y, y = (x - max) log2(e).
struct RowSums {
    float max, sum, dot;
};

// Moves sums taken at maximum s.max to maximum `to` (to >= s.max).
__device__ __forceinline__ void rescale(RowSums &s, float to) {
    if (s.sum != 0.0f && s.max != to) {    // a NaN sum goes on
        const float shift = (s.max - to) * kLog2e;
        const float f = exp2_approx(shift);
        // sum 2^y' y' = f * (dot + sum * shift); f = 0 where the shift overflows
        s.dot = f > 0.0f ? f * fmaf(s.sum, shift, s.dot) : 0.0f * s.sum;
        s.sum *= f;
    }
    s.max = to;
}

// Sums over the lanes of a warp: all to the largest maximum, then added.
__device__ __forceinline__ RowSums warp_join(RowSums s) {
    rescale(s, order_key_value(__reduce_max_sync(kFullMask, order_key(s.max))));
    return {s.max, warp_sum(s.sum), warp_sum(s.dot)};
}

// Two 32-bit numbers that move through one packed instruction.
union Pair {
    uint64_t u;
    float2 f;
};

__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair c;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(c.u) : "l"(a.u), "l"(b.u));
    return c;
}

__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair c;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(c.u) : "l"(a.u), "l"(b.u));
    return c;
}

__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.u) : "l"(a.u), "l"(b.u), "l"(c.u));
    return d;
}

__device__ __forceinline__ Pair pair(float x, float y) {
    Pair p;
    p.f = make_float2(x, y);
    return p;
}

// A thread's running sums, even and odd logits apart.
struct ThreadSums {
    float max;
    Pair minus, sum, dot;    // minus: -max twice; 0 before the first logit above -inf, so that -inf - 0 stays -inf

    __device__ ThreadSums() : max(kNegInf), minus(pair(0.0f, 0.0f)), sum(pair(0.0f, 0.0f)), dot(pair(0.0f, 0.0f)) {}

    __device__ __forceinline__ void raise(float to) {
        RowSums a{max, sum.f.x, dot.f.x}, b{max, sum.f.y, dot.f.y};
        rescale(a, to);
        rescale(b, to);
        max = to;
        minus = pair(-to, -to);
        sum = pair(a.sum, b.sum);
        dot = pair(a.dot, b.dot);
    }

    // low: some logit is so low that its exponent needs the bound
    template <int N> __device__ __forceinline__ void add(const float (&x)[N], bool low) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            Pair y = mul2(add2(pair(x[i], x[i + 1]), minus), pair(kLog2e, kLog2e));
            if (low) y = pair(max_nan(y.f.x, kTinyExponent), max_nan(y.f.y, kTinyExponent));
            const Pair e = pair(exp2_approx(y.f.x), exp2_approx(y.f.y));
            sum = add2(sum, e);
            dot = fma2(e, y, dot);
        }
    }

    __device__ __forceinline__ RowSums total() const { return {max, sum.f.x + sum.f.y, dot.f.x + dot.f.y}; }
};

struct LogprobsArgs {
    const void *logits;
    int64_t row_stride;
    uint32_t vocab;
    const void *targets;
    bool wide_targets;
    int top;
    uint32_t split;          // CTAs (of one cluster) per row
    float *logprobs, *entropy, *stats, *top_logprobs;
    int32_t *top_ids;
};

__device__ __forceinline__ int64_t target_of(const void *targets, bool wide, int64_t row) {
    return wide ? static_cast<const int64_t *>(targets)[row] : static_cast<const int32_t *>(targets)[row];
}

// The row in 16-byte vectors from the last boundary at or before its start.
template <typename T> struct RowView {
    const T *row;
    uint32_t shift, end, full_begin, full_end, vectors;   // elements: the row is [shift, end)

    __device__ RowView(const T *r, uint32_t vocab) : row(r) {
        constexpr uint32_t N = Wide<T>::kCount;
        shift = static_cast<uint32_t>((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(T));
        end = shift + vocab;
        full_begin = shift ? 1 : 0;
        full_end = end / N;
        vectors = (end + N - 1) / N;
    }

    __device__ __forceinline__ typename Wide<T>::type load_full(uint32_t v) const {
        const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(row - shift) + v);
        return *reinterpret_cast<const typename Wide<T>::type *>(&q);
    }

    // Vector v, -inf where it is not of the row or not below `last`.
    __device__ __forceinline__ typename Wide<T>::type load(uint32_t v, uint32_t last) const {
        using V = typename Wide<T>::type;
        constexpr int N = Wide<T>::kCount;
        V x;
        const T *base = row - shift;
        if (v < last && v >= full_begin && v < full_end) {
            const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(base) + v);
            x = *reinterpret_cast<const V *>(&q);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t e = v * N + i;
                x.e[i] = v < last && e >= shift && e < end ? base[e] : neg_inf<T>();
            }
        }
        return x;
    }
};

// Largest and smallest of a vector's logits, NaN left out.
template <typename T> __device__ __forceinline__ float2 vector_range(const typename Wide<T>::type &v) {
    float lo = to_f32(v.e[0]), hi = lo;
#pragma unroll
    for (int i = 1; i < Wide<T>::kCount; ++i) {
        const float x = to_f32(v.e[i]);
        lo = fminf(lo, x);
        hi = fmaxf(hi, x);
    }
    return make_float2(lo, hi);
}

// 16-bit types: two at a time, before they are widened.
template <> __device__ __forceinline__ float2 vector_range<__nv_bfloat16>(const Wide<__nv_bfloat16>::type &v) {
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&v);
    const __nv_bfloat162 lo = __hmin2(__hmin2(p[0], p[1]), __hmin2(p[2], p[3]));
    const __nv_bfloat162 hi = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
    return make_float2(fminf(to_f32(lo.x), to_f32(lo.y)), fmaxf(to_f32(hi.x), to_f32(hi.y)));
}

template <> __device__ __forceinline__ float2 vector_range<__half>(const Wide<__half>::type &v) {
    const __half2 *p = reinterpret_cast<const __half2 *>(&v);
    const __half2 lo = __hmin2(__hmin2(p[0], p[1]), __hmin2(p[2], p[3]));
    const __half2 hi = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
    return make_float2(fminf(to_f32(lo.x), to_f32(lo.y)), fmaxf(to_f32(hi.x), to_f32(hi.y)));
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kLpThreads, kLpCtas) k_logprobs(const LogprobsArgs a) {
    constexpr int N = Wide<T>::kCount;
    using V = typename Wide<T>::type;
    __shared__ RowSums s_sums[kLpWarps], s_cluster[kMaxCluster];
    __shared__ uint32_t s_group[32];                           // the groups' largest keys
    __shared__ uint64_t s_list[TOP ? kLpWarps : 1][32];        // the warps' lists
    __shared__ uint64_t s_remote[TOP ? kMaxCluster : 1][32];   // the cluster's lists
    __shared__ uint64_t s_buffer[TOP ? kCandidates : 1];
    __shared__ uint32_t s_count;
    __shared__ float s_threshold;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / a.split;
    const uint32_t part = blockIdx.x % a.split;
    if (a.split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

    const RowView<T> view(static_cast<const T *>(a.logits) + row * a.row_stride, a.vocab);
    const uint32_t full = view.full_end > view.full_begin ? view.full_end - view.full_begin : 0;
    const uint32_t per = (full + a.split - 1) / a.split;
    const uint32_t first = view.full_begin + min(full, part * per), last = view.full_begin + min(full, (part + 1) * per);

    float given = kNegInf;
    int64_t target = -1;
    if (a.targets != nullptr && part == 0 && tid == 0) {
        target = target_of(a.targets, a.wide_targets, row);
        if (target >= 0 && target < a.vocab) given = to_f32(view.row[target]);
    }

    ThreadSums mine;
    float threshold = kNegInf;
    uint64_t kept = 0;           // warp 0: the running list of the row's part, descending
    if (TOP) {
        if (tid == 0) s_count = 0;
        __syncthreads();
    }

    // sorts the buffer (and, where it overflowed, the candidates still held in
    // registers, given by `more`) into warp 0's list
    auto compress = [&](auto &&more) {
        const uint32_t have = min(s_count, kCandidates);
        uint64_t list = warp == 0 ? kept : 0;
        for (uint32_t b = warp * 32; b < have; b += kLpThreads) {
            const uint64_t c = b + lane < have ? s_buffer[b + lane] : 0;
            list = merge_lists(list, bitonic_sort_desc(c, lane), lane);
        }
        more(list);
        s_list[warp][lane] = list;
        __syncthreads();
        for (int w = kLpWarps / 2; w > 0; w >>= 1) {
            if (warp < w) {
                list = merge_lists(list, s_list[warp + w][lane], lane);
                s_list[warp][lane] = list;
            }
            __syncthreads();
        }
        if (warp == 0) kept = list;
        if (tid == 0) {
            const uint64_t c = s_list[0][a.top - 1];
            s_threshold = c ? order_key_value(static_cast<uint32_t>(c >> 32)) : kNegInf;
            s_count = 0;
        }
        __syncthreads();
        threshold = s_threshold;
    };

    for (uint32_t base = first; base < last; base += kLpStep) {
        V now[kLpVectors];
        const uint32_t v0 = base + tid;
#pragma unroll
        for (int u = 0; u < kLpVectors; ++u) {
            if (v0 + u * kLpThreads < last) {
                now[u] = view.load_full(v0 + u * kLpThreads);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) now[u].e[i] = neg_inf<T>();
            }
        }
        float bound = threshold;     // candidates are above it
        if (TOP && base == first) {
            // the largest logit of each of 32 groups of threads: `top` logits reach their top-th
            float hi = kNegInf;
#pragma unroll
            for (int u = 0; u < kLpVectors; ++u) hi = fmaxf(hi, vector_range<T>(now[u]).y);
#pragma unroll
            for (int o = kGroupLanes / 2; o > 0; o >>= 1) hi = fmaxf(hi, __shfl_xor_sync(kFullMask, hi, o));
            if (tid % kGroupLanes == 0) s_group[tid / kGroupLanes] = hi > kNegInf ? order_key(hi) : 0u;
            __syncthreads();
            const uint32_t key = s_group[lane];
            uint32_t rank = 0;       // groups before this one
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const uint32_t o = __shfl_sync(kFullMask, key, i);
                rank += (o > key || (o == key && i < lane)) ? 1u : 0u;
            }
            const uint32_t cut = __reduce_max_sync(kFullMask, rank == static_cast<uint32_t>(a.top - 1) ? key : 0u);
            // logits of this step that equal it may belong to the best; later ones have
            // higher indices: only a greater logit displaces one of this step
            threshold = cut ? order_key_value(cut) : kNegInf;
            bound = cut ? order_key_value(cut - (cut == 0x80000000u ? 2u : 1u)) : kNegInf;   // the key below zero's is unused
        }
        uint32_t held = 0;       // candidates of this step that found a place in the buffer
        bool full_buffer = false;
#pragma unroll
        for (int u = 0; u < kLpVectors; ++u) {
            const float2 range = vector_range<T>(now[u]);
            if (range.y > mine.max) mine.raise(range.y);
            float x[N];
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = to_f32(now[u].e[i]);
            if (range.x - mine.max > kLowLogit) mine.template add<N>(x, false);
            else mine.template add<N>(x, true);
            if (TOP && range.y > bound) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if (x[i] > bound) {
                        const uint32_t at = atomicAdd(&s_count, 1u);
                        if (at < kCandidates) {
                            s_buffer[at] = candidate(x[i], (v0 + u * kLpThreads) * N + i - view.shift);
                            held |= 1u << (u * N + i);
                        }
                        full_buffer |= at >= kCandidates / 2;
                    }
                }
            }
        }
        if (TOP && __syncthreads_or(full_buffer)) {
            const bool over = s_count > kCandidates;
            compress([&](uint64_t &list) {
                if (!over) return;
#pragma unroll 1
                for (int b = 0; b < kLpVectors * N; ++b) {
                    float x = kNegInf;
#pragma unroll
                    for (int u = 0; u < kLpVectors; ++u)
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            if (u * N + i == b) x = to_f32(now[u].e[i]);
                    uint64_t c = 0;
                    if (x > bound && !((held >> b) & 1u))
                        c = candidate(x, (v0 + (b / N) * kLpThreads) * N + b % N - view.shift);
                    if (__any_sync(kFullMask, c != 0)) list = merge_lists(list, bitonic_sort_desc(c, lane), lane);
                }
            });
        }
    }

    // the row's ends, up to N - 1 logits each that do not fill a vector
    if (part == 0 && warp == 0) {
        const uint32_t head = full ? view.full_begin * N : view.end;    // without a full vector: everything
        uint32_t e = view.shift + lane;
        if (e >= head) e = e - head + (full ? view.full_end * N : view.end);
        if (e < view.end) {
            const float x = to_f32((view.row - view.shift)[e]);
            if (x > mine.max) mine.raise(x);
            const float xs[2] = {x, kNegInf};
            mine.template add<2>(xs, true);
            if (TOP && x > kNegInf && x >= threshold) {    // less than half of the buffer is taken
                const uint32_t at = atomicAdd(&s_count, 1u);
                s_buffer[at] = candidate(x, e - view.shift);
            }
        }
    }

    RowSums s = warp_join(mine.total());
    if (lane == 0) s_sums[warp] = s;
    __syncthreads();
    if (TOP && s_count > 0) compress([](uint64_t &) {});
    if (warp == 0) s = warp_join(lane < kLpWarps ? s_sums[lane] : RowSums{kNegInf, 0.0f, 0.0f});

    if (a.split > 1) {
        // every CTA of the cluster runs; hand the part's results to CTA 0
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (warp == 0) {
            auto remote = [](const void *p) {
                uint32_t addr;
                asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(addr) : "r"(smem_addr(p)));
                return addr;
            };
            if (lane == 0) {
                const uint32_t to = remote(&s_cluster[part]);
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(s.max) : "memory");
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(s.sum) : "memory");
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(s.dot) : "memory");
            }
            if (TOP) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(&s_remote[part][lane])), "l"(kept) : "memory");
        }
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (part != 0) return;
        if (warp == 0) {
            s = warp_join(lane < static_cast<int>(a.split) ? s_cluster[lane] : RowSums{kNegInf, 0.0f, 0.0f});
            if (TOP)
                for (uint32_t p = 1; p < a.split; ++p) kept = merge_lists(kept, s_remote[p][lane], lane);
        }
    }
    if (warp != 0) return;

    const float log_sum = logf(s.sum);
    if (lane == 0) {
        if (a.logprobs != nullptr) {
            float lp = 0.0f;
            if (target >= static_cast<int64_t>(a.vocab)) lp = __int_as_float(0x7FC00000);   // no such token
            else if (target >= 0) lp = given == kNegInf && s.sum == s.sum ? kNegInf : (given - s.max) - log_sum;
            a.logprobs[row] = lp;
        }
        if (a.entropy != nullptr) a.entropy[row] = s.sum == 0.0f ? 0.0f : log_sum - s.dot / s.sum * kLn2;
        reinterpret_cast<float2 *>(a.stats)[row] = make_float2(s.max, s.sum);
    }
    if (TOP && lane < a.top) {
        float lp = kNegInf;
        int32_t id = -1;
        if (kept != 0) {
            id = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(kept));
            lp = (order_key_value(static_cast<uint32_t>(kept >> 32)) - s.max) - log_sum;
        }
        a.top_logprobs[row * a.top + lane] = lp;
        a.top_ids[row * a.top + lane] = id;
    }
}

// ------------------------------------------------------------------ gradient
constexpr int kGradThreads = 256;
constexpr int kGradVectors = 4;

struct LogprobsBackwardArgs {
    const float *grad_logprobs, *grad_entropy;
    const void *logits;
    int64_t row_stride, grad_stride;
    uint32_t vocab;
    const void *targets;
    bool wide_targets;
    const float *entropy, *stats;
    void *grad_logits;
    uint32_t blocks_per_row;
};

template <typename T>
__global__ void __launch_bounds__(kGradThreads) k_logprobs_backward(const LogprobsBackwardArgs a) {
    constexpr int N = Wide<T>::kCount;
    using V = typename Wide<T>::type;
    const int64_t row = blockIdx.x / a.blocks_per_row;
    const uint32_t block = blockIdx.x % a.blocks_per_row;
    const RowView<T> view(static_cast<const T *>(a.logits) + row * a.row_stride, a.vocab);
    T *out = static_cast<T *>(a.grad_logits) + row * a.grad_stride;
    // the gradient's rows move as vectors where they lie as the logits' do
    const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(view.row) & 15);
    out -= view.shift;

    V x[kGradVectors];
    const uint32_t v0 = block * (kGradThreads * kGradVectors) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kGradVectors; ++u) x[u] = view.load(v0 + u * kGradThreads, view.vectors);

    const float2 stats = reinterpret_cast<const float2 *>(a.stats)[row];
    const float m = stats.x, sum = stats.y;
    float g = a.grad_logprobs != nullptr ? a.grad_logprobs[row] : 0.0f;
    const float h = a.grad_entropy != nullptr ? a.grad_entropy[row] : 0.0f;
    int64_t t = -1;
    if (a.targets != nullptr) t = target_of(a.targets, a.wide_targets, row);
    if (t < 0) g = 0.0f;
    if (t >= static_cast<int64_t>(a.vocab)) g = __int_as_float(0x7FC00000);
    const bool empty = sum == 0.0f;
    const float inv = empty ? 0.0f : 1.0f / sum;
    const float cb = h * kLn2, ca = empty ? 0.0f : g + h * (a.entropy[row] - logf(sum));
    const uint32_t at = t >= 0 && t < static_cast<int64_t>(a.vocab) && !empty ? static_cast<uint32_t>(t) + view.shift : 0xFFFFFFFFu;

#pragma unroll
    for (int u = 0; u < kGradVectors; ++u) {
        const uint32_t v = v0 + u * kGradThreads;
        if (v >= view.vectors) break;
        V o;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float xi = to_f32(x[u].e[i]);
            // in a row that is masked whole x - m is NaN, and so masked apart
            const float y = empty ? kTinyExponent : max_nan((xi - m) * kLog2e, kTinyExponent);
            const float p = exp2_approx(y) * inv;
            float d = -p * fmaf(cb, y, ca);
            if (v * N + i == at) d += g;
            o.e[i] = from_f32<T>(d);
        }
        if (same && v >= view.full_begin && v < view.full_end) {
            __stcs(reinterpret_cast<uint4 *>(out) + v, *reinterpret_cast<const uint4 *>(&o));
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t e = v * N + i;
                if (e >= view.shift && e < view.end) out[e] = o.e[i];
            }
        }
    }
}

template <typename T, bool TOP> int start_logprobs(const LogprobsLaunch &L, const LogprobsArgs &a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<uint32_t>(L.rows) * a.split);
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {a.split, 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = a.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_logprobs<T, TOP>, a) == cudaSuccess ? GSORT_OK : GSORT_ECUDA;
}

}  // namespace

int launch_logprobs(const LogprobsLaunch &L) {
    LogprobsArgs a{};
    a.logits = L.logits;
    a.row_stride = L.row_stride;
    a.vocab = static_cast<uint32_t>(L.vocab);
    a.targets = L.targets;
    a.wide_targets = L.target_bytes == 8;
    a.top = L.top;
    a.logprobs = L.logprobs;
    a.entropy = L.entropy;
    a.stats = L.stats;
    a.top_logprobs = L.top_logprobs;
    a.top_ids = L.top_ids;
    // split a row while the device has idle SMs and a part still fills a CTA
    const int64_t vectors = L.vocab * float_bytes(L.dtype) / 16;
    a.split = 1;
    while (a.split < kMaxCluster && L.rows * a.split < 2 * L.sm_count && vectors / (2 * a.split) >= kLpThreads) a.split *= 2;
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        return L.top > 0 ? start_logprobs<T, true>(L, a) : start_logprobs<T, false>(L, a);
    });
}

int launch_logprobs_backward(const LogprobsBackwardLaunch &L) {
    LogprobsBackwardArgs a{};
    a.grad_logprobs = L.grad_logprobs;
    a.grad_entropy = L.grad_entropy;
    a.logits = L.logits;
    a.row_stride = L.row_stride;
    a.grad_stride = L.grad_stride;
    a.vocab = static_cast<uint32_t>(L.vocab);
    a.targets = L.targets;
    a.wide_targets = L.target_bytes == 8;
    a.entropy = L.entropy;
    a.stats = L.stats;
    a.grad_logits = L.grad_logits;
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int64_t per_block = static_cast<int64_t>(kGradThreads) * kGradVectors * Wide<T>::kCount;
        // a row can start inside a vector: up to kCount - 1 elements more
        a.blocks_per_row = static_cast<uint32_t>((L.vocab + Wide<T>::kCount - 1 + per_block - 1) / per_block);
        if (L.rows * a.blocks_per_row > 0x7FFFFFFF) return static_cast<int>(GSORT_ETOOBIG);
        k_logprobs_backward<T><<<static_cast<uint32_t>(L.rows * a.blocks_per_row), kGradThreads, 0, L.stream>>>(a);
        return cudaGetLastError() == cudaSuccess ? static_cast<int>(GSORT_OK) : static_cast<int>(GSORT_ECUDA);
    });
}

}  // namespace gsort
