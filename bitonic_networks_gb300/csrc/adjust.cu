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
// A CTA holds a piece of a row, a whole one where rows are many.  The tokens that
// history or biases name in it are a set in shared memory: a bit for every token of
// the piece, and the named ones before each word of bits, so that a named token has a
// slot and the slots are no more than the history is long.  Counts are made in the slots by a
// second look over the history.  The mask's words are laid beside the set's, so that a
// vector's bits are all at one place.  Then the logits pass by once: a vector without a
// bit costs a look at its bits and no more than a copy.  The memory bounds it: logits in,
// logits out.  In place, vectors in which nothing changes are neither read nor
// written.
#include <algorithm>

#include "model_ops.cuh"

namespace gsort {
namespace {

constexpr int kAdjustThreads = 512;
constexpr int kAdjustVectors = 4;                 // 16-byte vectors in flight per thread, and as many of the next step
constexpr int kHistoryLoads = 8;                  // tokens of the history in flight per thread
constexpr size_t kAdjustMaxSmem = 112 * 1024;     // two CTAs to an SM
constexpr int64_t kAdjustCtas = 304;              // that rows are cut into, where they are fewer
constexpr uint32_t kSeenBefore = 0x80000000u;     // of a count: the token is in the prompt
constexpr uint32_t kNowhere = 0xFFFFFFFFu;

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
    uint32_t pieces, tokens; // pieces of a row, of so many tokens (a multiple of 256) each
    uint32_t slots, bias_slots;      // words of the sets' slots
    bool vectors;            // rows of in and out lie the same way to 16 bytes
    bool in_place;
};

__device__ __forceinline__ int64_t int_at(const void *p, int bytes, int64_t i) {
    return bytes == 8 ? static_cast<const int64_t *>(p)[i] : static_cast<const int32_t *>(p)[i];
}

// n bits of a string of words from bit `at` on, all of one word.
__device__ __forceinline__ uint32_t bits_at(const uint32_t *words, uint32_t at, int n) {
    return words[at >> 5] >> (at & 31) & ((1u << n) - 1);
}

// Tokens of a piece, by their distance from its first one, in shared memory.  With
// less than 32768 members the words `before` and the counts in the slots take 16 bits.
struct TokenSet {
    uint32_t *bits;      // null: no set
    uint32_t *before;    // members before each word of bits
    uint32_t *slots;     // one for each member
    bool narrow;

    __device__ __forceinline__ bool has(uint32_t at) const { return bits != nullptr && (bits[at >> 5] >> (at & 31) & 1); }
    __device__ __forceinline__ uint32_t member(uint32_t at) const {      // its number
        const uint32_t w = at >> 5;
        return (narrow ? reinterpret_cast<const uint16_t *>(before)[w] : before[w]) + __popc(bits[w] & ((1u << (at & 31)) - 1));
    }
    __device__ __forceinline__ void add(uint32_t at) const {
        const uint32_t bit = 1u << (at & 31);
        if (at != kNowhere && !(*const_cast<const volatile uint32_t *>(bits + (at >> 5)) & bit)) atomicOr(bits + (at >> 5), bit);
    }
    // A token once more, in the prompt or behind it.
    __device__ __forceinline__ void count(uint32_t at, bool prompt) const {
        const uint32_t m = member(at), half = narrow ? 16 * (m & 1) : 0;
        uint32_t *word = slots + (narrow ? m / 2 : m);
        if (prompt) atomicOr(word, (narrow ? 0x8000u : kSeenBefore) << half);
        else atomicAdd(word, 1u << half);
    }
    __device__ __forceinline__ uint32_t counted(uint32_t at) const {     // how often behind the prompt
        const uint32_t m = member(at);
        return narrow ? reinterpret_cast<const uint16_t *>(slots)[m] & 0x7FFFu : slots[m] & ~kSeenBefore;
    }
};

__host__ __device__ constexpr bool is_narrow(int64_t members) { return members < 32768; }

// Counts the members before each word, and clears their slots (words of 1 or 2 to a
// slot word).  Called by the whole CTA.
__device__ __forceinline__ void number_members(const TokenSet &set, uint32_t words, uint32_t per_slot_word) {
    __shared__ uint32_t s_sum[kAdjustThreads / 32];
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t per = (words + kAdjustThreads - 1) / kAdjustThreads, begin = min(tid * per, words), end = min(begin + per, words);
    uint32_t mine = 0;
    for (uint32_t w = begin; w < end; ++w) mine += __popc(set.bits[w]);
    const uint32_t upto = warp_inclusive_scan(mine, lane);
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    uint32_t sum = upto - mine, total = 0;
#pragma unroll
    for (int i = 0; i < kAdjustThreads / 32; ++i) {
        const uint32_t n = s_sum[i];
        if (i < static_cast<int>(warp)) sum += n;
        total += n;
    }
    for (uint32_t w = begin; w < end; ++w) {
        if (set.narrow) reinterpret_cast<uint16_t *>(set.before)[w] = static_cast<uint16_t>(sum);
        else set.before[w] = sum;
        sum += __popc(set.bits[w]);
    }
    for (uint32_t i = tid; i * per_slot_word < total; i += kAdjustThreads) set.slots[i] = 0;
    __syncthreads();
}

// The tokens `base` + thread, + threads, ... of a list, as distances from the piece's first one.
__device__ __forceinline__ void load_tokens(const void *list, int bytes, int64_t row, uint32_t length, uint32_t base, int32_t begin,
                                            int32_t end, int32_t first, uint32_t (&at)[kHistoryLoads]) {
    uint32_t t[kHistoryLoads];       // what is no 32-bit number is no token
    const uint32_t i0 = base + threadIdx.x;
    if (bytes == 4) {
        const uint32_t *p = static_cast<const uint32_t *>(list) + row + i0;
#pragma unroll
        for (int k = 0; k < kHistoryLoads; ++k) t[k] = i0 + k * kAdjustThreads < length ? p[k * kAdjustThreads] : kNowhere;
    } else {
        const uint64_t *p = static_cast<const uint64_t *>(list) + row + i0;
#pragma unroll
        for (int k = 0; k < kHistoryLoads; ++k) {
            const uint64_t x = i0 + k * kAdjustThreads < length ? p[k * kAdjustThreads] : ~0ull;
            t[k] = x >> 32 ? kNowhere : static_cast<uint32_t>(x);
        }
    }
    const uint32_t span = static_cast<uint32_t>(end - begin);        // end <= 2^30: kNowhere is outside
#pragma unroll
    for (int k = 0; k < kHistoryLoads; ++k) at[k] = t[k] - static_cast<uint32_t>(begin) < span ? t[k] - static_cast<uint32_t>(first) : kNowhere;
}

// What a CTA knows of its piece of a row.
struct Piece {
    TokenSet seen, biased;
    const float *bias;
    uint32_t *allowed;         // bits of the piece's tokens, in shared memory; null: no mask
    float repetition, presence, frequency;
    int32_t first, begin, end; // the piece's first token (a vector may begin before the row), and its tokens
};

__device__ __forceinline__ float adjusted(const Piece &p, float x, uint32_t at) {
    if (p.seen.has(at)) {
        const uint32_t n = p.seen.counted(at);
        x = x > 0.0f ? x / p.repetition : x * p.repetition;
        if (n != 0) x -= fmaf(p.frequency, static_cast<float>(n), p.presence);
    }
    if (p.biased.has(at)) x += p.bias[p.biased.slots[p.biased.member(at)] - 1];
    return x;
}

// Elements whose bit is clear become -inf (or 0).
template <typename T, bool ZERO> __device__ __forceinline__ void mask_vector(uint4 &q, uint32_t bits) {
    uint32_t *w = &q.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t keep;
        if (sizeof(T) == 4) keep = bits >> i & 1 ? 0xFFFFFFFFu : 0u;
        else keep = ((bits >> (2 * i) | bits << 15 >> (2 * i)) & 0x00010001u) * 0xFFFFu;
        w[i] = ZERO ? w[i] & keep : (w[i] & keep) | (Wide<T>::kNegInfWord & ~keep);
    }
}

template <typename T, bool BACK>
__global__ void __launch_bounds__(kAdjustThreads, 2) k_adjust(const AdjustArgs<T> a) {
    constexpr int N = Wide<T>::kCount, U = kAdjustVectors;
    constexpr uint32_t kAll = (1u << N) - 1;
    extern __shared__ __align__(16) uint32_t s_words[];
    const uint32_t row = blockIdx.x / a.pieces, piece = blockIdx.x % a.pieces, tid = threadIdx.x;
    const T *in = a.in + static_cast<int64_t>(row) * a.in_stride;
    T *out = a.out + static_cast<int64_t>(row) * a.out_stride;
    // elements between the 16-byte boundary at or before the row and the row
    const int32_t shift = a.vectors ? static_cast<int32_t>((reinterpret_cast<uintptr_t>(in) & 15) / sizeof(T)) : 0;
    const int64_t low = static_cast<int64_t>(piece) * a.tokens - shift;
    if (low >= a.vocab) return;
    Piece p{};
    p.first = static_cast<int32_t>(low);
    p.begin = max(p.first, 0);
    p.end = static_cast<int32_t>(min(low + a.tokens, static_cast<int64_t>(a.vocab)));
    // vectors of the piece that are whole: not those that the row's start or end cuts
    const uint32_t low_v = p.first < 0 ? 1 : 0, high_v = static_cast<uint32_t>(p.end - p.first) / N;

    // the first vectors are on their way while the sets are made
    uint4 q[U];
    auto load = [&](uint32_t v0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t v = v0 + u * kAdjustThreads;
            if (v >= low_v && v < high_v) q[u] = reinterpret_cast<const uint4 *>(in + p.first)[v];
        }
    };
    const bool ahead = a.vectors && !a.in_place;
    if (ahead) load(tid);

    const uint32_t words = a.tokens / 32;
    uint32_t *space = s_words;
    if (a.history != nullptr) {
        p.seen.narrow = is_narrow(a.length);
        p.seen.bits = space;
        p.seen.before = space + words;
        p.seen.slots = p.seen.before + (p.seen.narrow ? words / 2 : words);
        space = BACK ? p.seen.before : p.seen.slots + a.slots;
    }
    if (!BACK && a.biases > 0) {
        p.biased.narrow = is_narrow(a.biases);
        p.biased.bits = space;
        p.biased.before = space + words;
        p.biased.slots = p.biased.before + (p.biased.narrow ? words / 2 : words);
        p.bias = a.bias + static_cast<int64_t>(row) * a.bias_stride;
        space = p.biased.slots + a.bias_slots;
    }
    if (a.allowed != nullptr) {      // word w: the bits of the piece's tokens 32 w ..
        const uint32_t *mask = a.allowed + static_cast<int64_t>(row) * a.allowed_stride;
        const int32_t last = static_cast<int32_t>((a.vocab - 1) / 32);
        p.allowed = space;
#pragma unroll 4
        for (uint32_t w = tid; w < words; w += kAdjustThreads) {
            const int32_t at = p.first + static_cast<int32_t>(w * 32), k = at >> 5;      // -8 < at
            const uint32_t here = k >= 0 && k <= last ? mask[k] : 0, next = (at & 31) != 0 && k < last ? mask[k + 1] : 0;
            space[w] = __funnelshift_r(here, next, at & 31);
        }
        if (!p.seen.bits && !p.biased.bits) __syncthreads();
    }
    if (p.seen.bits || p.biased.bits) {
        for (uint32_t w = tid; w < words; w += kAdjustThreads) {
            if (p.seen.bits) p.seen.bits[w] = 0;
            if (p.biased.bits) p.biased.bits[w] = 0;
        }
        __syncthreads();
        const int64_t history_row = static_cast<int64_t>(row) * a.history_stride, bias_row = static_cast<int64_t>(row) * a.bias_stride;
        uint32_t at[kHistoryLoads];
        constexpr uint32_t kStep = kAdjustThreads * kHistoryLoads;
        if (p.seen.bits) {
            for (uint32_t base = 0; base < a.length; base += kStep) {
                load_tokens(a.history, a.history_bytes, history_row, a.length, base, p.begin, p.end, p.first, at);
#pragma unroll
                for (int k = 0; k < kHistoryLoads; ++k) p.seen.add(at[k]);
            }
        }
        if (p.biased.bits) {
            for (uint32_t i = tid; i < a.biases; i += kAdjustThreads) {
                const int64_t t = int_at(a.bias_tokens, a.bias_bytes, bias_row + i);
                if (t >= p.begin && t < p.end) p.biased.add(static_cast<uint32_t>(t - p.first));
            }
        }
        __syncthreads();
        if (!BACK) {
            if (p.seen.bits) {
                number_members(p.seen, words, p.seen.narrow ? 2 : 1);
                const uint32_t prompt = a.prompt ? static_cast<uint32_t>(max(a.prompt[row], 0)) : 0;
                for (uint32_t base = 0; base < a.length; base += kStep) {
                    // a history of one step is still there
                    if (a.length > kStep) load_tokens(a.history, a.history_bytes, history_row, a.length, base, p.begin, p.end, p.first, at);
#pragma unroll
                    for (int k = 0; k < kHistoryLoads; ++k) {
                        if (at[k] != kNowhere) p.seen.count(at[k], base + k * kAdjustThreads + tid < prompt);
                    }
                }
            }
            if (p.biased.bits) {
                number_members(p.biased, words, 1);
                for (uint32_t i = tid; i < a.biases; i += kAdjustThreads) {
                    const int64_t t = int_at(a.bias_tokens, a.bias_bytes, bias_row + i);
                    if (t >= p.begin && t < p.end) atomicMax(p.biased.slots + p.biased.member(static_cast<uint32_t>(t - p.first)), i + 1);
                }
            }
            __syncthreads();
        }
    }
    p.repetition = a.repetition ? a.repetition[row] : 1.0f;
    p.presence = a.presence ? a.presence[row] : 0.0f;
    p.frequency = a.frequency ? a.frequency[row] : 0.0f;
    const T *logits = BACK && p.seen.bits ? a.logits + static_cast<int64_t>(row) * a.logits_stride : nullptr;

    // the value of a token that history or biases name
    auto named = [&](float x, int32_t e) {
        if (!BACK) return adjusted(p, x, static_cast<uint32_t>(e - p.first));
        return to_f32(logits[e]) > 0.0f ? x * (1.0f / p.repetition) : x * p.repetition;
    };
    auto single = [&](int32_t e) {
        const uint32_t at = static_cast<uint32_t>(e - p.first);
        const float x = to_f32(in[e]);
        const bool allow = !p.allowed || bits_at(p.allowed, at, 1);
        out[e] = from_f32<T>(!allow ? (BACK ? 0.0f : kNegInf) : p.seen.has(at) || p.biased.has(at) ? named(x, e) : x);
    };
    // Single elements: the whole piece where rows lie differently, else those of the two
    // vectors that the row's start and end cut.
    const int32_t whole = a.vectors ? p.first + static_cast<int32_t>(low_v) * N : p.end;
    for (int32_t e = p.begin + static_cast<int32_t>(tid); e < min(whole, p.end); e += kAdjustThreads) single(e);
    if (!a.vectors) return;
    const int32_t rest = max(p.first + static_cast<int32_t>(high_v) * N, whole);
    if (rest + static_cast<int32_t>(tid) < p.end) single(rest + static_cast<int32_t>(tid));
    for (uint32_t v0 = tid; v0 < high_v; v0 += kAdjustThreads * U) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = q[u];
        if (ahead) load(v0 + kAdjustThreads * U);
        // Vectors are masked and written as a whole; the few named tokens are gathered
        // and written after them (their code stands here once: in the unrolled part, 32
        // times, it did not fit the instruction cache, 2048 x 131072 490 us).
        uint32_t names = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t v = v0 + u * kAdjustThreads;
            if (v < low_v || v >= high_v) continue;
            uint32_t name = 0, allow = kAll;
            if (p.seen.bits) name = bits_at(p.seen.bits, v * N, N);
            if (p.biased.bits) name |= bits_at(p.biased.bits, v * N, N);
            if (p.allowed) allow = bits_at(p.allowed, v * N, N);
            names |= (name & allow) << (u * N);
            if (a.in_place) {
                if (allow == kAll) continue;
                x[u] = reinterpret_cast<const uint4 *>(in + p.first)[v];
            }
            if (p.allowed) mask_vector<T, BACK>(x[u], allow);
            reinterpret_cast<uint4 *>(out + p.first)[v] = x[u];
        }
        while (names != 0) {
            const uint32_t b = __ffs(names) - 1;
            names &= names - 1;
            const int32_t e = p.first + static_cast<int32_t>((v0 + b / N * kAdjustThreads) * N + b % N);
            out[e] = from_f32<T>(named(to_f32(in[e]), e));     // in place, it holds its value still
        }
    }
}

}  // namespace

int launch_adjust(const AdjustLaunch &L) {
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int N = Wide<T>::kCount;
        constexpr int64_t kLeast = kAdjustThreads * N;      // tokens of a piece: a vector for every thread
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
        // pieces that fill the device, smaller ones where their sets would take too much room
        const int64_t want = std::max<int64_t>(kAdjustCtas / L.rows, 1), most = (L.vocab + kLeast - 1) / kLeast;
        const int64_t pieces = std::min(want, most), span = L.vocab + (a.vectors ? N - 1 : 0);
        int64_t tokens = std::max<int64_t>(256, (std::min<int64_t>(span / pieces + 1, 1 << 18) + 255) / 256 * 256);
        auto smem_bytes = [&] {
            const int64_t words = tokens / 32;
            a.tokens = static_cast<uint32_t>(tokens);
            a.slots = static_cast<uint32_t>((std::min(tokens, L.length) + 1) / (is_narrow(L.length) ? 2 : 1));
            a.bias_slots = static_cast<uint32_t>(std::min(tokens, L.biases));
            int64_t all = L.allowed != nullptr ? words : 0;
            if (a.history != nullptr) all += words + (L.backward ? 0 : (is_narrow(L.length) ? words / 2 : words) + a.slots);
            if (!L.backward && L.biases > 0) all += words + (is_narrow(L.biases) ? words / 2 : words) + a.bias_slots;
            return static_cast<size_t>(all) * 4;
        };
        while (smem_bytes() > kAdjustMaxSmem) tokens = (tokens / 2 + 255) / 256 * 256;
        a.pieces = static_cast<uint32_t>((span + tokens - 1) / tokens);
        const int64_t blocks = L.rows * a.pieces;
        if (blocks > 0x7FFFFFFF) return static_cast<int>(GSORT_ETOOBIG);
        const size_t smem = smem_bytes();
        const void *kernel = L.backward ? reinterpret_cast<const void *>(k_adjust<T, true>) : reinterpret_cast<const void *>(k_adjust<T, false>);
        if (smem > 48 * 1024 && set_smem_limit(kernel, kAdjustMaxSmem) != cudaSuccess) return static_cast<int>(GSORT_ECUDA);
        if (L.backward) k_adjust<T, true><<<static_cast<uint32_t>(blocks), kAdjustThreads, smem, L.stream>>>(a);
        else k_adjust<T, false><<<static_cast<uint32_t>(blocks), kAdjustThreads, smem, L.stream>>>(a);
        return cudaGetLastError() == cudaSuccess ? static_cast<int>(GSORT_OK) : static_cast<int>(GSORT_ECUDA);
    });
}

}  // namespace gsort
