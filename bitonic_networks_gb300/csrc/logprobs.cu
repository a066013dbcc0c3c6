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
// The forward pass keeps a running maximum per warp and rescales its sums when
// the maximum grows, so a row is read once: 8192 x 131072 bf16 take 300 us, the
// memory's rate.  The largest logits are found in the same pass: the first 8,192
// 16-bit (4,096 32-bit) logits give a threshold that at least `top` of them
// reach, and only logits above it are written to a shared buffer, which is sorted
// by warps (bitonic networks of 32) when the row ends; where the buffer is full,
// a warp sorts into a list of its own.  With alternatives the ends of rows are
// what is left above the memory's time: 4096 x 100003 bf16 take 134 us, reading
// them 123.  Few rows are split over a cluster of CTAs, joined through
// distributed shared memory; short rows take a warp each.
#include <algorithm>

#include "model_ops.cuh"

namespace gsort {
namespace {

// 256 threads with 4 vectors each in flight and 5 CTAs per SM keep the memory
// busy: 4096 x 100003 bf16 with one alternative takes 134 us (6.1 TB/s). In an
// earlier state: 158, with 4 CTAs 165, 2 vectors 182, CTAs of 512 threads 190.
constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;   // at most 8: join_lists
constexpr int kLpVectors = 4;               // 16-byte vectors per thread and step
constexpr int kLpCtas = 5;                  // CTAs per SM that the registers allow
constexpr uint32_t kCandidates = 2048;      // shared buffers of candidates, of a CTA
constexpr int kMaxCluster = 8;
// Up to so many alternatives 32 groups give a threshold that hardly more logits
// pass than have to; with more of them it would be far too low (4096 x 131072
// bf16 with 32 alternatives: 585 us, 259 with a group for every thread, 217 now).
constexpr int kFewTop = 8;
constexpr uint32_t kRefresh = 64;          // candidates of a warp's row that are sorted before its end
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

// The same networks for order keys alone.
__device__ __forceinline__ uint32_t merge_keys_desc(uint32_t v, int lane) {
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) {
        const uint32_t o = __shfl_xor_sync(kFullMask, v, j);
        v = (lane & j) ? min(v, o) : max(v, o);
    }
    return v;
}

__device__ __forceinline__ uint32_t sort_keys_desc(uint32_t v, int lane) {
#pragma unroll
    for (int k = 2; k < 32; k <<= 1) {
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const uint32_t o = __shfl_xor_sync(kFullMask, v, j);
            v = ((lane & j) != 0) != ((lane & k) != 0) ? min(v, o) : max(v, o);
        }
    }
    return merge_keys_desc(v, lane);
}

// The 32 largest keys of COUNT descending lists, joined by a tree.
template <int COUNT> __device__ __forceinline__ uint32_t join_keys(uint32_t (&v)[COUNT], int lane) {
#pragma unroll
    for (int w = COUNT / 2; w > 0; w >>= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) v[i] = merge_keys_desc(max(v[i], __shfl_sync(kFullMask, v[i + w], 31 - lane)), lane);
    return v[0];
}

// Joins `count` (1..8) lists of 32, one after another in shared memory, by a
// tree: the merges of a level do not wait on each other.
__device__ __forceinline__ uint64_t join_lists(const uint64_t (*lists)[32], int count, int lane) {
    uint64_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < count ? lists[i][lane] : 0;
#pragma unroll
    for (int w = 4; w > 0; w >>= 1) {
        if (count > w) {
#pragma unroll
            for (int i = 0; i < w; ++i) v[i] = merge_lists(v[i], v[i + w], lane);
        }
    }
    return v[0];
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

// A lane's running sums at its warp's running maximum, even and odd logits apart.
struct LaneSums {
    float max;
    Pair minus, sum, dot;    // minus: -max twice; 0 before the first logit above -inf, so that -inf - 0 stays -inf

    __device__ LaneSums() : max(kNegInf), minus(pair(0.0f, 0.0f)), sum(pair(0.0f, 0.0f)), dot(pair(0.0f, 0.0f)) {}

    // Raises the warp's maximum to the largest of the lanes' `hi`.  It grows
    // about ln(steps) times in a row, so this is rarely more than one vote.
    __device__ __forceinline__ void raise(float hi) {
        if (!__any_sync(kFullMask, hi > max)) return;
        const float to = order_key_value(__reduce_max_sync(kFullMask, order_key(hi > max ? hi : max)));
        RowSums a{max, sum.f.x, dot.f.x}, b{max, sum.f.y, dot.f.y};
        rescale(a, to);
        rescale(b, to);
        max = to;
        minus = pair(-to, -to);
        sum = pair(a.sum, b.sum);
        dot = pair(a.dot, b.dot);
    }

    // Adds COUNT pairs, summed on their own first: the sum is about 1 beside the
    // largest logit and rounds at each addition to it.  An exponential is off by up to
    // 2^-22 + (max - x) 2^-23 of itself (ex2.approx, and the product rounded); in a sum
    // that is (max - x) e^(x - max) 2^-23 a logit, and rows from 1000 to 131072
    // logits are as near to 64 bits as with expf (3e-8 to 5e-8 on normal logits).
    // low: some logit is so low that its exponent needs the bound.
    template <int COUNT> __device__ __forceinline__ void add(const Pair (&x)[COUNT], bool low) {
        Pair part;
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            Pair y = mul2(add2(x[i], minus), pair(kLog2e, kLog2e));
            if (low) y = pair(max_nan(y.f.x, kTinyExponent), max_nan(y.f.y, kTinyExponent));
            const Pair e = pair(exp2_approx(y.f.x), exp2_approx(y.f.y));
            part = i == 0 ? e : add2(part, e);
            dot = fma2(e, y, dot);
        }
        sum = add2(sum, part);
    }

    template <typename T> __device__ __forceinline__ void add_vector(const uint4 &q, bool low) {
        Pair x[Wide<T>::kCount / 2];
#pragma unroll
        for (int i = 0; i < Wide<T>::kCount / 2; ++i) x[i] = Wide<T>::pair_of(q, i);
        add(x, low);
    }

    __device__ __forceinline__ RowSums total() const { return {max, sum.f.x + sum.f.y, dot.f.x + dot.f.y}; }
};

struct LogprobsArgs {
    const void *logits;
    int64_t rows, row_stride;
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

    __device__ __forceinline__ const uint4 *address(uint32_t v) const { return reinterpret_cast<const uint4 *>(row - shift) + v; }
    __device__ __forceinline__ uint4 load(uint32_t v) const { return __ldcs(address(v)); }

    // Element that lane `i` takes of the row's ends (up to kCount - 1 at each
    // end do not fill a vector; without a full vector it is the whole row);
    // `end` where there is none.
    __device__ __forceinline__ uint32_t edge(uint32_t i) const {
        const bool some = full_end > full_begin;
        const uint32_t head = some ? full_begin * Wide<T>::kCount : end;
        const uint32_t e = shift + i;
        if (e < head) return e;
        return min(end, e - head + (some ? full_end * Wide<T>::kCount : end));
    }
};

// Smallest and largest of a thread's logits, NaN left out.
template <typename T, int U> __device__ __forceinline__ float2 logit_range(const uint4 (&q)[U]) {
    float lo = __uint_as_float(q[0].x), hi = lo;
#pragma unroll
    for (int i = 1; i < 4 * U; ++i) {
        const float x = __uint_as_float((&q[i / 4].x)[i % 4]);
        lo = fminf(lo, x);
        hi = fmaxf(hi, x);
    }
    return make_float2(lo, hi);
}

// 16-bit types: two at a time, before they are widened.
template <typename T2, int U> __device__ __forceinline__ float2 logit_range2(const uint4 (&q)[U]) {
    T2 lo = *reinterpret_cast<const T2 *>(&q[0].x), hi = lo;
#pragma unroll
    for (int i = 1; i < 4 * U; ++i) {
        const T2 x = *reinterpret_cast<const T2 *>(&q[i / 4].x + i % 4);
        lo = __hmin2(lo, x);
        hi = __hmax2(hi, x);
    }
    return make_float2(fminf(to_f32(lo.x), to_f32(lo.y)), fmaxf(to_f32(hi.x), to_f32(hi.y)));
}

template <> __device__ __forceinline__ float2 logit_range<__nv_bfloat16>(const uint4 (&q)[kLpVectors]) {
    return logit_range2<__nv_bfloat162>(q);
}

template <> __device__ __forceinline__ float2 logit_range<__half>(const uint4 (&q)[kLpVectors]) {
    return logit_range2<__half2>(q);
}

// A thread's logits above `bound`, as bits; hit_element gives a bit's element.
template <typename T, int U> __device__ __forceinline__ uint32_t hits_above(const uint4 (&q)[U], float bound) {
    uint32_t hits = 0;
#pragma unroll
    for (int i = 0; i < 4 * U; ++i) hits |= __uint_as_float((&q[i / 4].x)[i % 4]) > bound ? 1u << i : 0u;
    return hits;
}

// 16-bit types: two at a time (against the next value of the type at or below the
// bound); word i has bits i and i + 16.
template <typename T2, int U> __device__ __forceinline__ uint32_t hits_above2(const uint4 (&q)[U], T2 bound) {
    uint32_t hits = 0;
#pragma unroll
    for (int i = 0; i < 4 * U; ++i) hits |= __hgt2_mask(*reinterpret_cast<const T2 *>(&q[i / 4].x + i % 4), bound) & (0x00010001u << i);
    return hits;
}

template <> __device__ __forceinline__ uint32_t hits_above<__nv_bfloat16>(const uint4 (&q)[kLpVectors], float bound) {
    return hits_above2(q, __bfloat162bfloat162(__float2bfloat16_rd(bound)));
}

template <> __device__ __forceinline__ uint32_t hits_above<__half>(const uint4 (&q)[kLpVectors], float bound) {
    return hits_above2(q, __half2half2(__float2half_rd(bound)));
}

template <typename T> __device__ __forceinline__ int hit_element(int bit) {
    return sizeof(T) == 4 ? bit : 2 * (bit & 15) + (bit >> 4);
}

// TEAM threads hold a row (or a part of one): the CTA, or for short rows a warp.
template <typename T, bool TOP, int TEAM>
__global__ void __launch_bounds__(kLpThreads, kLpCtas) k_logprobs(const LogprobsArgs a) {
    constexpr int N = Wide<T>::kCount;
    constexpr int kTeams = kLpThreads / TEAM;
    constexpr uint32_t kStep = TEAM * kLpVectors, kRoom = kCandidates / kTeams;
    constexpr int kGroupLanes = TEAM / 32;                     // 32 groups of lanes give the first threshold
    __shared__ RowSums s_sums[kLpWarps], s_cluster[kMaxCluster];
    __shared__ __align__(16) uint32_t s_groups[kTeams][32];    // the groups' largest keys
    __shared__ uint32_t s_keys[TOP && TEAM > 32 ? kLpWarps : 1][32];
    __shared__ uint64_t s_list[TOP ? kLpWarps : 1][32];        // the warps' lists
    __shared__ uint64_t s_remote[TOP ? kMaxCluster : 1][32];   // the cluster's lists
    __shared__ uint64_t s_buffers[TOP ? kCandidates : 1];
    __shared__ uint32_t s_counts[kTeams];

    const int tid = threadIdx.x % TEAM, lane = tid & 31, warp = tid >> 5, team = threadIdx.x / TEAM;   // within the team
    uint32_t *s_group = s_groups[team], &s_count = s_counts[team];
    uint64_t *s_buffer = s_buffers + (TOP ? team * kRoom : 0);
    auto sync = [] {
        if (TEAM == 32) __syncwarp();
        else __syncthreads();
    };
    const uint32_t unit = blockIdx.x * kTeams + team;
    const int64_t row = unit / a.split;
    const uint32_t part = unit % a.split;
    if (row >= a.rows) return;       // a whole warp: other teams have no barrier with it
    if (TEAM > 32 && a.split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

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

    LaneSums mine;
    float threshold = kNegInf;
    uint64_t kept = 0;           // the warp's list, descending
    if (TOP && tid == 0) s_count = 0;

    // sorts the warp's share of the buffer into its list
    auto take = [&](uint32_t have) {
        for (uint32_t b = warp * 32; b < have; b += TEAM) {
            const uint64_t c = bitonic_sort_desc(b + lane < have ? s_buffer[b + lane] : 0, lane);
            kept = __any_sync(kFullMask, kept != 0) ? merge_lists(kept, c, lane) : c;
        }
    };

    // With alternatives a row stops at its first step and at its end, and the
    // other CTAs' loads do not fill the gap: the step after next is on its way
    // into L2 (4096 x 100003 bf16: 158 -> 148 us when it came; no gain elsewhere).
    auto prefetch = [&](uint32_t v) {
        if (TOP && tid == 0 && v < last)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(view.address(v)), "r"(min(kStep, last - v) * 16) : "memory");
    };
    prefetch(first + kStep);
    for (uint32_t base = first; base < last; base += kStep) {
        prefetch(base + 2 * kStep);
        uint4 now[kLpVectors];
        const uint32_t v0 = base + tid;
#pragma unroll
        for (int u = 0; u < kLpVectors; ++u) {
            constexpr uint32_t w = Wide<T>::kNegInfWord;
            now[u] = make_uint4(w, w, w, w);
            if (v0 + u * TEAM < last) now[u] = view.load(v0 + u * TEAM);
        }
        const float2 range = logit_range<T>(now);
        mine.raise(range.y);
        float bound = threshold;     // candidates are above it
        if (TOP && base == first) {
            // `top` logits reach the top-th largest of the largest logits of some groups
            uint32_t cut;
            if (a.top <= kFewTop) {
                // 32 groups of threads, whose ranks are counted
                float hi = range.y > kNegInf ? range.y : kNegInf;
#pragma unroll
                for (int o = kGroupLanes / 2; o > 0; o >>= 1) hi = fmaxf(hi, __shfl_xor_sync(kFullMask, hi, o));
                // the key's last five bits make room for the group's number, so that no two are equal
                const uint32_t group = tid / kGroupLanes;
                if (tid % kGroupLanes == 0) s_group[group] = hi > kNegInf ? (order_key(hi) & ~31u) | group : 0u;
                sync();
                const uint32_t key = s_group[lane];
                uint32_t above = 0;
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const uint4 o = *reinterpret_cast<const uint4 *>(s_group + i);
                    above += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
                }
                cut = __reduce_max_sync(kFullMask, above == static_cast<uint32_t>(a.top - 1) ? key : 0u) & ~31u;
            } else if (TEAM == 32) {
                // every vector is a group
                uint32_t keys[kLpVectors];
#pragma unroll
                for (int u = 0; u < kLpVectors; ++u) {
                    float hi = kNegInf;
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        const Pair p = Wide<T>::pair_of(now[u], i);
                        hi = fmaxf(hi, fmaxf(p.f.x, p.f.y));
                    }
                    keys[u] = sort_keys_desc(hi > kNegInf ? order_key(hi) : 0u, lane);
                }
                sync();              // s_count is set
                cut = __shfl_sync(kFullMask, join_keys(keys, lane), a.top - 1);
            } else {
                // every thread is a group: each warp sorts its own, then joins all
                s_keys[warp][lane] = sort_keys_desc(range.y > kNegInf ? order_key(range.y) : 0u, lane);
                sync();
                uint32_t keys[kLpWarps];
#pragma unroll
                for (int w = 0; w < kLpWarps; ++w) keys[w] = s_keys[w][lane];
                cut = __shfl_sync(kFullMask, join_keys(keys, lane), a.top - 1);
            }
            // logits of this step that equal it may belong to the best; later ones have
            // higher indices: only a greater logit displaces one of this step
            threshold = cut ? order_key_value(cut) : kNegInf;
            bound = cut ? order_key_value(cut - (cut == 0x80000000u ? 2u : 1u)) : kNegInf;   // the key below zero's is unused
        }
        uint32_t hits = 0;       // the thread's candidates
        if (TOP && range.y > bound) hits = hits_above<T>(now, bound);
        if (range.x - mine.max > kLowLogit) {
#pragma unroll
            for (int u = 0; u < kLpVectors; ++u) mine.template add_vector<T>(now[u], false);
        } else {
#pragma unroll
            for (int u = 0; u < kLpVectors; ++u) mine.template add_vector<T>(now[u], true);
        }
        if (TOP) {
            auto element = [&](int bit) {
                const int b = hit_element<T>(bit);
                return (v0 + b / N * TEAM) * N + b % N;
            };
            uint32_t lost = 0;   // candidates that found the buffer full
            if (hits != 0) {
                uint32_t at = atomicAdd(&s_count, static_cast<uint32_t>(__popc(hits)));
                const bool one = (hits & (hits - 1)) == 0;     // mostly: it is the thread's largest
                for (; hits != 0; hits &= hits - 1, ++at) {
                    const uint32_t e = element(__ffs(hits) - 1);
                    if (at < kRoom) s_buffer[at] = candidate(one ? range.y : to_f32((view.row - view.shift)[e]), e - view.shift);
                    else lost |= hits & (~hits + 1);
                }
            }
            if (__any_sync(kFullMask, lost != 0)) {
                // rare: the warp sorts them into a list of its own, which raises its threshold
#pragma unroll 1
                for (int b = 0; b < kLpVectors * N; ++b) {
                    uint64_t c = 0;
                    if ((lost >> b) & 1u) c = candidate(to_f32((view.row - view.shift)[element(b)]), element(b) - view.shift);
                    if (__any_sync(kFullMask, c != 0)) kept = merge_lists(kept, bitonic_sort_desc(c, lane), lane);
                }
                const uint64_t c = __shfl_sync(kFullMask, kept, a.top - 1);
                if (c) threshold = fmaxf(threshold, order_key_value(static_cast<uint32_t>(c >> 32)));
            }
        }
        if (TOP && TEAM == 32) {
            // a warp's buffer is small, and nobody else waits: sorting it now raises the
            // threshold (8192 x 12000 bf16 with 20 alternatives: 149 us without, 71)
            __syncwarp();
            const uint32_t have = s_count;
            if (have >= kRefresh) {
                take(min(have, kRoom));
                __syncwarp();
                if (lane == 0) s_count = 0;
                __syncwarp();
                const uint64_t c = __shfl_sync(kFullMask, kept, a.top - 1);
                if (c) threshold = fmaxf(threshold, order_key_value(static_cast<uint32_t>(c >> 32)));
            }
        }
    }

    if (TOP && first >= last) sync();     // s_count is set; with a step, its barrier has come
    // the row's ends
    if (part == 0 && warp == 0) {
        const uint32_t e = view.edge(lane);
        const float x = e < view.end ? to_f32((view.row - view.shift)[e]) : kNegInf;
        mine.raise(x);
        const Pair one[1] = {pair(x, kNegInf)};
        mine.add(one, true);
        if (TOP) {
            const uint64_t c = x > kNegInf && x >= threshold ? candidate(x, e - view.shift) : 0;
            if (__any_sync(kFullMask, c != 0)) kept = merge_lists(kept, bitonic_sort_desc(c, lane), lane);
        }
    }

    RowSums s = warp_join(mine.total());
    if (TEAM > 32 && lane == 0) s_sums[warp] = s;
    sync();
    if (TOP) {
        // each warp sorts its share of the buffer into its list; warp 0 joins the lists
        const uint32_t have = min(s_count, kRoom);
        take(have);
        if (TEAM > 32) {
            const int lists = s_count > kRoom ? kLpWarps : min(kLpWarps, static_cast<int>((have + 31) / 32));
            if (lists > 1) {
                s_list[warp][lane] = kept;
                __syncthreads();
                if (warp == 0) kept = join_lists(s_list, lists, lane);
            }
        }
    }
    if (TEAM > 32 && warp == 0) s = warp_join(lane < kLpWarps ? s_sums[lane] : RowSums{kNegInf, 0.0f, 0.0f});

    if (TEAM > 32 && a.split > 1) {
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
            if (TOP) kept = join_lists(s_remote, static_cast<int>(a.split), lane);
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
    int64_t rows;
    uint32_t blocks_per_row;   // CTAs to a row where its threads are the CTA, else 1
};

// A row's gradient as a function of x: with e = 2^y, y = (x - m) log2(e),
//   -p (g + h (ln p + H)) = e * (q1 y + q0),  q1 = -h ln2 / S,  q0 = -(g + h (H - ln S)) / S
// A 16-bit gradient rounds to 2^-9 or 2^-12 of itself: there the product in y may
// round too (up to (m - x) 2^-23 of e).  A 32-bit one keeps what it lost; the
// memory bounds it all the same.
template <typename T> struct RowGradient {
    Pair minus, q0, q1;

    // FLAT: q1 = 0, no entropy in the loss
    template <bool FLAT> __device__ __forceinline__ Pair at(Pair x) const {
        const Pair d = add2(x, minus);
        Pair y;
        if (sizeof(T) == 4) {
            const Pair e = exp_exact2(d, y);
            return mul2(e, FLAT ? q0 : fma2(q1, y, q0));
        }
        y = mul2(d, pair(kLog2e, kLog2e));
        if (FLAT) return mul2(pair(exp2_approx(y.f.x), exp2_approx(y.f.y)), q0);
        y = pair(max_nan(y.f.x, kTinyExponent), max_nan(y.f.y, kTinyExponent));
        return mul2(pair(exp2_approx(y.f.x), exp2_approx(y.f.y)), fma2(q1, y, q0));
    }

    template <bool FLAT> __device__ __forceinline__ uint4 vector(const uint4 &x) const {
        uint4 o;
#pragma unroll
        for (int i = 0; i < Wide<T>::kCount / 2; ++i) Wide<T>::set_pair(o, i, at<FLAT>(Wide<T>::pair_of(x, i)));
        return o;
    }
};

// LANES threads are side by side on a row: the CTA, or for short rows some warps
// of it (8192 x 1000 bf16: 6 us, 16 with a CTA to a row).
template <typename T, int LANES>
__global__ void __launch_bounds__(kGradThreads) k_logprobs_backward(const LogprobsBackwardArgs a) {
    constexpr int N = Wide<T>::kCount;
    const uint32_t tid = threadIdx.x % LANES;
    const int64_t row = static_cast<int64_t>(blockIdx.x / a.blocks_per_row) * (kGradThreads / LANES) + threadIdx.x / LANES;
    const uint32_t block = blockIdx.x % a.blocks_per_row;
    if (row >= a.rows) return;
    const RowView<T> view(static_cast<const T *>(a.logits) + row * a.row_stride, a.vocab);
    T *out = static_cast<T *>(a.grad_logits) + row * a.grad_stride;
    // the gradient's rows move as vectors where they lie as the logits' do
    const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(view.row) & 15);
    out -= view.shift;

    uint4 x[kGradVectors];
    const uint32_t v0 = view.full_begin + block * (kGradThreads * kGradVectors) + tid;
#pragma unroll
    for (int u = 0; u < kGradVectors; ++u)
        if (v0 + u * LANES < view.full_end) x[u] = view.load(v0 + u * LANES);

    const float2 stats = reinterpret_cast<const float2 *>(a.stats)[row];
    float g = a.grad_logprobs != nullptr ? a.grad_logprobs[row] : 0.0f;
    const float h = a.grad_entropy != nullptr ? a.grad_entropy[row] : 0.0f;
    int64_t t = -1;
    if (a.targets != nullptr) t = target_of(a.targets, a.wide_targets, row);
    if (t < 0) g = 0.0f;
    if (t >= static_cast<int64_t>(a.vocab)) g = __int_as_float(0x7FC00000);
    const bool empty = stats.y == 0.0f;      // every logit is -inf: -inf - 0 stays -inf, and e = 0
    const float m = empty ? 0.0f : stats.x, inv = empty ? 0.0f : -1.0f / stats.y;
    const float q0 = empty ? 0.0f : (h == 0.0f ? g : g + h * (a.entropy[row] - logf(stats.y))) * inv, q1 = h * kLn2 * inv;
    RowGradient<T> f;
    f.minus = pair(-m, -m);
    f.q0 = pair(q0, q0);
    f.q1 = pair(q1, q1);
    // the target's element; 0xFFFFFFFF: none
    const uint32_t at = t >= 0 && t < static_cast<int64_t>(a.vocab) && !empty ? static_cast<uint32_t>(t) + view.shift : 0xFFFFFFFFu;

    // read before the stores: they may be to the same memory
    const uint32_t tv = at / N;
    const bool own = tv >= v0 && tv < view.full_end && (tv - v0) % LANES == 0 && (tv - v0) / LANES < kGradVectors;
    float xt = 0.0f;
    if (own) xt = to_f32((view.row - view.shift)[at]);

#pragma unroll
    for (int u = 0; u < kGradVectors; ++u) {
        const uint32_t v = v0 + u * LANES;
        if (v < view.full_end) {
            const uint4 o = h == 0.0f ? f.template vector<true>(x[u]) : f.template vector<false>(x[u]);
            if (same) {
                __stcs(reinterpret_cast<uint4 *>(out) + v, o);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) out[v * N + i] = Wide<T>::element(o, i);
            }
        }
    }
    if (own) {                                   // over this thread's own vector, rounded once
        const Pair p = pair(xt, kNegInf);
        out[at] = from_f32<T>((h == 0.0f ? f.template at<true>(p) : f.template at<false>(p)).f.x + g);
    }
    if (block == 0 && tid < 32) {        // the row's ends
        const uint32_t e = view.edge(tid);
        if (e < view.end) {
            const Pair p = pair(to_f32((view.row - view.shift)[e]), kNegInf);
            const Pair d = h == 0.0f ? f.template at<true>(p) : f.template at<false>(p);
            out[e] = from_f32<T>(d.f.x + (e == at ? g : 0.0f));
        }
    }
}

template <typename T, bool TOP, int TEAM> int start_logprobs(const LogprobsLaunch &L, const LogprobsArgs &a) {
    constexpr int64_t kTeams = kLpThreads / TEAM;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<uint32_t>((L.rows * a.split + kTeams - 1) / kTeams));
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {a.split, 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = a.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_logprobs<T, TOP, TEAM>, a) == cudaSuccess ? GSORT_OK : GSORT_ECUDA;
}

}  // namespace

int launch_logprobs(const LogprobsLaunch &L) {
    LogprobsArgs a{};
    a.logits = L.logits;
    a.rows = L.rows;
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
    const int64_t vectors = L.vocab * float_bytes(L.dtype) / 16;
    // A warp to a row where it is short, so that rows wait for no CTA-wide barrier
    // (8192 x 1000 bf16 with 5 alternatives: 14 us, 51 with a CTA each), and up to
    // four times as long where rows fill the device, 24 to an SM.  bf16, a warp / a
    // CTA to a row in us:
    //   8192 x 6000 22 / 35, with 20 alternatives 46 / 64; x 12000 36 / 50, 70 / 86
    //   3660 x 6000 with 20 alternatives 28 / 31; x 12000 42 / 41; x 16000 52 / 44
    //   1824 x 6000 with 20 alternatives 19 / 18; x 12000 29 / 23; x 16000 36 / 25
    // One limit for all: by length and alternatives the two cross between 1824 rows
    // (x 6000 without alternatives 9.2 / 10.2) and 4864 (x 16000 with 20 53 / 56).
    const bool warps = vectors <= 512 || (vectors <= 2048 && L.rows >= 24 * L.sm_count);
    // Otherwise a row is split while CTAs do not fill the device and a part has 512
    // vectors: up to 3 CTAs to an SM before the last halving.  131072 bf16 with 20
    // alternatives, with 1 / 3 / 12 to an SM: 76 rows 13.8 / 12.4 / 12.4 us, 152 21.7 /
    // 17.6 / 20.6, 304 26 / 24 / 35, 380 32 / 28 / 42, 450 32 / 36 / 48.
    a.split = 1;
    while (!warps && a.split < kMaxCluster && L.rows * a.split < 3 * L.sm_count && vectors / (2 * a.split) >= 512) a.split *= 2;
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        if (warps) return L.top > 0 ? start_logprobs<T, true, 32>(L, a) : start_logprobs<T, false, 32>(L, a);
        return L.top > 0 ? start_logprobs<T, true, kLpThreads>(L, a) : start_logprobs<T, false, kLpThreads>(L, a);
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
        constexpr int64_t per_thread = static_cast<int64_t>(kGradVectors) * Wide<T>::kCount, per_block = kGradThreads * per_thread;
        a.rows = L.rows;
        const int lanes = L.vocab <= 32 * per_thread ? 32 : L.vocab <= 128 * per_thread ? 128 : kGradThreads;
        a.blocks_per_row = lanes < kGradThreads ? 1 : static_cast<uint32_t>((L.vocab + per_block - 1) / per_block);
        const int64_t in_block = kGradThreads / lanes, blocks = (L.rows + in_block - 1) / in_block * a.blocks_per_row;
        if (blocks > 0x7FFFFFFF) return static_cast<int>(GSORT_ETOOBIG);
        const uint32_t grid = static_cast<uint32_t>(blocks);
        if (lanes == 32) k_logprobs_backward<T, 32><<<grid, kGradThreads, 0, L.stream>>>(a);
        else if (lanes == 128) k_logprobs_backward<T, 128><<<grid, kGradThreads, 0, L.stream>>>(a);
        else k_logprobs_backward<T, kGradThreads><<<grid, kGradThreads, 0, L.stream>>>(a);
        return cudaGetLastError() == cudaSuccess ? static_cast<int>(GSORT_OK) : static_cast<int>(GSORT_ECUDA);
    });
}

}  // namespace gsort
