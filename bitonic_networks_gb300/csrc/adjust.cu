// adjust.cu -- logits before an answer is chosen: penalties for tokens that were
// there before, biases of single tokens, and a mask of the tokens that may follow.
//
// Per row x of V logits, with c the times that a token comes up in the generated
// part of the row's history, and "seen" where it comes up in the history at all:
//   y = seen ? (x > 0 ? x / r : x * r) : x            repetition r
//   y = y - (f * c + p * [c > 0])                     frequency f, presence p
//   y = y + b                                         the row's last bias of the token
//   out = y where the token's bit of the mask is set (or there is no mask), else -inf
// and the gradient by x: 0 where the mask's bit is clear, else d * (seen ? (x > 0 ? 1 / r
// : r) : 1).
//
// A CTA holds a piece of a row: counts of its tokens in shared memory, made by
// one look over the row's whole history (which the caches hold for the row's
// other CTAs), then one pass over its logits.  A bit for every token says
// whether history or biases name it, so that the others cost no more than a copy.  The
// memory bounds it: logits in, logits out.  In place, vectors in which nothing
// changes are neither read nor written.
#include <algorithm>

#include "model_ops.cuh"

namespace gsort {
namespace {

constexpr int kAdjustThreads = 256;
constexpr int kAdjustVectors = 4;                 // 16-byte vectors per thread and step
constexpr size_t kAdjustMaxSmem = 128 * 1024;     // of a CTA
constexpr uint32_t kSeenBefore = 0x80000000u;     // of a count: the token is in the prompt

template <typename T> struct AdjustArgs {
    const T *logits;         // the gradient's: null where no history is given
    const T *in;             // what is adjusted: the logits, or the gradient by the adjusted logits
    T *out;
    int64_t logits_stride, in_stride, out_stride;
    uint32_t rows, vocab;
    const void *history;
    int64_t history_stride;
    uint32_t length;
    int history_bytes;
    const int32_t *prompt;
    const float *repetition, *presence, *frequency;
    const void *bias_tokens;
    const float *bias;
    int64_t bias_stride;     // of both
    uint32_t biases;
    int bias_bytes;
    const uint32_t *allowed;
    int64_t allowed_stride;
    uint32_t pieces, steps;  // pieces of a row, of `steps` * 1024 vectors each
    bool vectors;            // rows of in and out lie the same way to 16 bytes
    bool in_place;
};

__device__ __forceinline__ int64_t int_at(const void *p, int bytes, int64_t i) {
    return bytes == 8 ? static_cast<const int64_t *>(p)[i] : static_cast<const int32_t *>(p)[i];
}

// What a CTA knows of its piece of a row.
struct Piece {
    const uint32_t *named;     // a bit for every token: history or biases name it
    const uint32_t *counts;    // null: no history
    const uint32_t *biased;    // entry + 1 of the token's bias, 0: none; null: no biases
    const float *bias;
    const uint32_t *allowed;   // the row's mask; null: none
    float repetition, presence, frequency;
    int32_t first;             // the piece's first token (a vector may begin before the row)
    uint32_t vocab;

    __device__ __forceinline__ uint32_t bits(const uint32_t *words, int32_t at, int n) const {   // n <= 8 bits from `at` on
        const uint32_t w = static_cast<uint32_t>(at) >> 5, s = at & 31;
        uint32_t b = words[w] >> s;
        if (s + n > 32) b |= words[w + 1] << (32 - s);
        return b & ((1u << n) - 1);
    }
};

__device__ __forceinline__ float adjusted(const Piece &p, float x, int32_t e) {
    const uint32_t at = static_cast<uint32_t>(e - p.first);
    if (p.counts != nullptr) {
        const uint32_t c = p.counts[at];
        if (c != 0) {
            x = x > 0.0f ? x / p.repetition : x * p.repetition;
            const uint32_t n = c & ~kSeenBefore;
            if (n != 0) x -= fmaf(p.frequency, static_cast<float>(n), p.presence);
        }
    }
    if (p.biased != nullptr) {
        const uint32_t b = p.biased[at];
        if (b != 0) x += p.bias[b - 1];
    }
    return x;
}

template <typename T, bool BACK>
__global__ void __launch_bounds__(kAdjustThreads) k_adjust(const AdjustArgs<T> a) {
    constexpr int N = Wide<T>::kCount;
    extern __shared__ __align__(16) uint32_t s_words[];
    const uint32_t row = blockIdx.x / a.pieces, piece = blockIdx.x % a.pieces, tid = threadIdx.x;
    const uint32_t tokens = a.steps * (kAdjustThreads * kAdjustVectors * N);       // of a piece
    const T *in = a.in + static_cast<int64_t>(row) * a.in_stride;
    T *out = a.out + static_cast<int64_t>(row) * a.out_stride;
    // elements between the 16-byte boundary at or before the row and the row
    const int32_t shift = a.vectors ? static_cast<int32_t>((reinterpret_cast<uintptr_t>(in) & 15) / sizeof(T)) : 0;
    const int64_t low = static_cast<int64_t>(piece) * tokens - shift;
    if (low >= a.vocab) return;
    const int32_t first = static_cast<int32_t>(low);
    const int32_t begin = max(first, 0), end = static_cast<int32_t>(min(low + tokens, static_cast<int64_t>(a.vocab)));
    const bool history = a.history != nullptr, biases = !BACK && a.biases > 0;

    // shared memory: a bit for each token, then counts and biases where there are any
    uint32_t *named = s_words, *counts = named + tokens / 32, *biased = counts + (history && !BACK ? tokens : 0);
    if (history || biases) {
        const uint32_t words = tokens / 32 + (history && !BACK ? tokens : 0) + (biases ? tokens : 0);
        for (uint32_t i = tid * 4; i < words; i += kAdjustThreads * 4) *reinterpret_cast<uint4 *>(s_words + i) = make_uint4(0, 0, 0, 0);
        __syncthreads();
        if (history) {
            const uint32_t prompt = a.prompt ? static_cast<uint32_t>(max(a.prompt[row], 0)) : 0;
            const int64_t base = static_cast<int64_t>(row) * a.history_stride;
#pragma unroll 8
            for (uint32_t i = tid; i < a.length; i += kAdjustThreads) {
                const int64_t t = int_at(a.history, a.history_bytes, base + i);
                if (t >= begin && t < end) {
                    const uint32_t at = static_cast<uint32_t>(static_cast<int32_t>(t) - first);
                    atomicOr(named + at / 32, 1u << (at & 31));
                    if (!BACK) {
                        if (i < prompt) atomicOr(counts + at, kSeenBefore);
                        else atomicAdd(counts + at, 1u);
                    }
                }
            }
        }
        if (biases) {
            const int64_t base = static_cast<int64_t>(row) * a.bias_stride;
            for (uint32_t i = tid; i < a.biases; i += kAdjustThreads) {
                const int64_t t = int_at(a.bias_tokens, a.bias_bytes, base + i);
                if (t >= begin && t < end) {
                    const uint32_t at = static_cast<uint32_t>(static_cast<int32_t>(t) - first);
                    atomicOr(named + at / 32, 1u << (at & 31));
                    atomicMax(biased + at, i + 1);
                }
            }
        }
        __syncthreads();
    }
    Piece p;
    p.named = history || biases ? named : nullptr;
    p.counts = history ? counts : nullptr;
    p.biased = biases ? biased : nullptr;
    p.bias = biases ? a.bias + static_cast<int64_t>(row) * a.bias_stride : nullptr;
    p.allowed = a.allowed ? a.allowed + static_cast<int64_t>(row) * a.allowed_stride : nullptr;
    p.repetition = a.repetition ? a.repetition[row] : 1.0f;
    p.presence = a.presence ? a.presence[row] : 0.0f;
    p.frequency = a.frequency ? a.frequency[row] : 0.0f;
    p.first = first;
    p.vocab = a.vocab;
    const T *logits = BACK && history ? a.logits + static_cast<int64_t>(row) * a.logits_stride : nullptr;

    auto one = [&](float x, int32_t e, bool name, bool allow) {
        if (BACK) {
            if (!allow) return 0.0f;
            if (!name) return x;
            return to_f32(logits[e]) > 0.0f ? x * (1.0f / p.repetition) : x * p.repetition;
        }
        return !allow ? kNegInf : name ? adjusted(p, x, e) : x;
    };
    if (!a.vectors) {          // rows that lie differently: element by element
        for (int32_t e = begin + static_cast<int32_t>(tid); e < end; e += kAdjustThreads) {
            const bool name = p.named && p.bits(p.named, e - first, 1), allow = !p.allowed || p.bits(p.allowed, e, 1);
            out[e] = from_f32<T>(one(to_f32(in[e]), e, name, allow));
        }
        return;
    }
    for (uint32_t step = 0; step < a.steps; ++step) {
        uint4 q[kAdjustVectors];
        uint32_t name[kAdjustVectors], allow[kAdjustVectors];
        int32_t at[kAdjustVectors];
#pragma unroll
        for (int u = 0; u < kAdjustVectors; ++u) {
            const uint32_t v = (step * kAdjustVectors + u) * kAdjustThreads + tid;
            const int32_t e = first + static_cast<int32_t>(v * N);
            at[u] = e;
            name[u] = 0;
            allow[u] = (1u << N) - 1;
            if (e < 0 || e + N > end) continue;
            if (p.named) name[u] = p.bits(p.named, e - first, N);
            if (p.allowed) allow[u] = p.bits(p.allowed, e, N);
            if (a.in_place && name[u] == 0 && allow[u] == (1u << N) - 1) continue;
            q[u] = *reinterpret_cast<const uint4 *>(in + e);
        }
#pragma unroll
        for (int u = 0; u < kAdjustVectors; ++u) {
            const int32_t e = at[u];
            if (e < 0 || e + N > end) {        // the row's first and last elements
                for (int i = 0; i < N; ++i) {
                    const int32_t k = e + i;
                    if (k < begin || k >= end) continue;
                    const bool n1 = p.named && p.bits(p.named, k - first, 1), a1 = !p.allowed || p.bits(p.allowed, k, 1);
                    if (a.in_place && !n1 && a1) continue;
                    out[k] = from_f32<T>(one(to_f32(in[k]), k, n1, a1));
                }
                continue;
            }
            if (name[u] == 0 && allow[u] == (1u << N) - 1) {
                if (!a.in_place) *reinterpret_cast<uint4 *>(out + e) = q[u];
                continue;
            }
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const Pair x = Wide<T>::pair_of(q[u], i);
                Wide<T>::set_pair(q[u], i, pair(one(x.f.x, e + 2 * i, name[u] >> (2 * i) & 1, allow[u] >> (2 * i) & 1),
                                                one(x.f.y, e + 2 * i + 1, name[u] >> (2 * i + 1) & 1, allow[u] >> (2 * i + 1) & 1)));
            }
            *reinterpret_cast<uint4 *>(out + e) = q[u];
        }
    }
}

}  // namespace

int launch_adjust(const AdjustLaunch &L) {
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int N = Wide<T>::kCount;
        constexpr uint32_t kStep = kAdjustThreads * kAdjustVectors * N;     // tokens of a step
        AdjustArgs<T> a{};
        a.logits = static_cast<const T *>(L.logits);
        a.in = static_cast<const T *>(L.in);
        a.out = static_cast<T *>(L.out);
        a.logits_stride = L.logits_stride;
        a.in_stride = L.in_stride;
        a.out_stride = L.out_stride;
        a.rows = static_cast<uint32_t>(L.rows);
        a.vocab = static_cast<uint32_t>(L.vocab);
        a.history = L.history;
        a.history_stride = L.history_stride;
        a.length = static_cast<uint32_t>(L.length);
        a.history_bytes = L.history_bytes;
        a.prompt = L.prompt;
        a.repetition = L.repetition;
        a.presence = L.presence;
        a.frequency = L.frequency;
        a.bias_tokens = L.bias_tokens;
        a.bias = L.bias;
        a.bias_stride = L.bias_stride;
        a.biases = static_cast<uint32_t>(L.biases);
        a.bias_bytes = L.bias_bytes;
        a.allowed = L.allowed;
        a.allowed_stride = L.allowed_stride;
        a.in_place = L.in == L.out;
        // a row has the distance from the boundary of its array and `row` strides
        a.vectors = ((reinterpret_cast<uintptr_t>(L.in) ^ reinterpret_cast<uintptr_t>(L.out)) & 15) == 0 &&
                    (L.rows == 1 || (L.in_stride - L.out_stride) % N == 0);
        a.steps = 1;
        const uint32_t tokens = a.steps * kStep;
        a.pieces = static_cast<uint32_t>((L.vocab + (a.vectors ? N - 1 : 0) + tokens - 1) / tokens);
        const int64_t blocks = L.rows * a.pieces;
        if (blocks > 0x7FFFFFFF) return static_cast<int>(GSORT_ETOOBIG);
        const bool history = a.history != nullptr, biases = !L.backward && a.biases > 0;
        size_t smem = 0;
        if (history || biases) smem = (tokens / 32 + (history && !L.backward ? tokens : 0) + (biases ? tokens : 0)) * 4;
        const void *kernel = L.backward ? reinterpret_cast<const void *>(k_adjust<T, true>) : reinterpret_cast<const void *>(k_adjust<T, false>);
        if (smem > 48 * 1024 && set_smem_limit(kernel, kAdjustMaxSmem) != cudaSuccess) return static_cast<int>(GSORT_ECUDA);
        if (L.backward) k_adjust<T, true><<<static_cast<uint32_t>(blocks), kAdjustThreads, smem, L.stream>>>(a);
        else k_adjust<T, false><<<static_cast<uint32_t>(blocks), kAdjustThreads, smem, L.stream>>>(a);
        return cudaGetLastError() == cudaSuccess ? static_cast<int>(GSORT_OK) : static_cast<int>(GSORT_ECUDA);
    });
}

}  // namespace gsort
