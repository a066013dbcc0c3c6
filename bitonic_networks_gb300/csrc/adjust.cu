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
// A CTA holds a piece of a row, a whole one where rows are many.  Some of its warps pass
// the logits by once, through a ring of bulk copies, and mask them.  The others meanwhile make
// the set of the history's tokens in shared memory: a bit for every token of
// the piece, and the members before each word of bits, so that a token has a
// slot and the slots are no more than the history is long; counts are made in the slots
// by a second look over the history, biases go to a hash table.  When the piece
// is written, each token of the set is taken once, and its logit (from the caches) is
// written anew.  In place, vectors in which nothing is masked are neither read nor written.
//
// The memory bounds large calls: logits in, logits out.  2048 x 131072 bf16 with histories of 1024,
// 64 biases and a mask take 376 us with their gradient (5.8 TB/s of what is counted so); 64 x
// 131072 f32 with histories of 2048 16.4 us, of which 13.5 are what the call takes with nothing to adjust.  Long
// histories take longer than the logits: 256 x 100003 bf16 with 16384 tokens 54 us, the memory's
// part 18: an SM has two rows one after the other, and writes the named tokens of one before the next begins.
// In place, what is masked is read too, behind the mask's words: where a grammar leaves one token of
// 1000, 64 x 131072 f32 take 20.6 us in place and 14.5 with an output of their own.
#include <algorithm>

#include "model_ops.cuh"

namespace gsort {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kStageVectors = 2;                  // vectors of a stage of the ring for each thread of the CTA; 1 where room is short
constexpr int kMostStages = 4;
constexpr uint32_t kChunk = 1024, kChunks = 4;    // tokens of a chunk of a long history, and chunks on their way at once
constexpr uint32_t kQueue = 64;                   // members of the set that a warp has room for, at least
// A CTA of 512 threads has half an SM, one of 1024 a whole one: for histories that do not
// fit beside the rest in the half.
constexpr size_t kHalfSmem = 108 * 1024, kWholeSmem = 218 * 1024;
constexpr int64_t kHalfCtas = 304, kWholeCtas = 152;      // that rows are cut into, where they are fewer
constexpr uint32_t kSeenBefore = 0x80000000u;     // of a count: the token is in the prompt
constexpr uint32_t kNowhere = 0xFFFFFFFFu;
constexpr uint32_t kWaitLimit = 1u << 20;         // polls of a copy's barrier before its room is used anew

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
    uint32_t slots, table;   // words of the set's slots; entries of the biases' table, a power of two
    uint32_t stages;         // of the ring; 0: none
    uint32_t stage_vectors;  // of a stage for each thread
    uint32_t ring_words;     // of shared memory, for the ring and after it the queues
    uint32_t streamers;      // threads that pass the logits by; the others see to what is named
    bool history_whole;      // the history has room in shared memory
    bool narrow;             // counts and numbers of members in 16 bits
    bool vectors;            // rows of in and out lie the same way to 16 bytes
    bool in_place;
    Waits waits;             // for the ring's copies
};

__device__ __forceinline__ int64_t int_at(const void *p, int bytes, int64_t i) {
    return bytes == 8 ? static_cast<const int64_t *>(p)[i] : static_cast<const int32_t *>(p)[i];
}

// n bits of a string of words from bit `at` on, all of one word.
__device__ __forceinline__ uint32_t bits_at(const uint32_t *words, uint32_t at, int n) {
    return words[at >> 5] >> (at & 31) & ((1u << n) - 1);
}

// Histories whose counts fit 15 bits.
constexpr bool is_narrow(int64_t length) { return length < 32768; }

// Tokens of a piece, by their distance from its first one, in shared memory.
struct TokenSet {
    uint32_t *bits;      // null: no set
    uint32_t *before;    // members before each word of bits
    uint32_t *slots;     // a count for each member
    bool narrow;         // `before` and counts in 16 bits

    __device__ __forceinline__ bool has(uint32_t at) const { return bits != nullptr && (bits[at >> 5] >> (at & 31) & 1); }
    __device__ __forceinline__ uint32_t member(uint32_t at) const {      // its number
        const uint32_t w = at >> 5;
        return (narrow ? reinterpret_cast<const uint16_t *>(before)[w] : before[w]) + __popc(bits[w] & ((1u << (at & 31)) - 1));
    }
    __device__ __forceinline__ void add(uint32_t at) const {
        const uint32_t bit = 1u << (at & 31);
        if (at != kNowhere && !(*const_cast<const volatile uint32_t *>(bits + (at >> 5)) & bit)) atomicOr(bits + (at >> 5), bit);
    }
    // A token of the history once more, in the prompt or behind it.
    __device__ __forceinline__ void count(uint32_t at, bool prompt) const {
        const uint32_t m = member(at), half = narrow ? 16 * (m & 1) : 0;
        uint32_t *word = slots + (narrow ? m / 2 : m);
        if (prompt) atomicOr(word, (narrow ? 0x8000u : kSeenBefore) << half);
        else atomicAdd(word, 1u << half);
    }
    // How often behind the prompt, with kSeenBefore; kNowhere for all but one of those who ask.
    __device__ __forceinline__ uint32_t take(uint32_t at) const {
        const uint32_t m = member(at);
        if (!narrow) return atomicExch(slots + m, kNowhere);
        const uint32_t half = 16 * (m & 1), c = atomicOr(slots + m / 2, 0xFFFFu << half) >> half & 0xFFFFu;
        return c == 0xFFFFu ? kNowhere : (c & 0x7FFFu) | (c & 0x8000u) << 16;      // fewer than 32768: 0xFFFF is no count
    }
    // The same, of a member that one thread asks for.
    __device__ __forceinline__ uint32_t counted(uint32_t at) const {
        const uint32_t m = member(at);
        if (!narrow) return slots[m];
        const uint32_t c = reinterpret_cast<const uint16_t *>(slots)[m];
        return (c & 0x7FFFu) | (c & 0x8000u) << 16;
    }
    // Whether the token was there still: the gradient needs no counts.
    __device__ __forceinline__ bool take_bit(uint32_t at) const {
        const uint32_t bit = 1u << (at & 31);
        return atomicAnd(bits + (at >> 5), ~bit) & bit;
    }
};

// Some warps of the CTA, for a barrier of their own.
struct Crew {
    uint32_t id, threads, rank;      // barrier, threads, and this thread among them
    __device__ __forceinline__ void sync() const { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
    // The same, and whether x holds for any thread.
    __device__ __forceinline__ bool sync_any(bool x) const {
        uint32_t any;
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                     : "=r"(any) : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(x)) : "memory");
        return any != 0;
    }
};

// Counts the members before each word, and clears their slots.  Called by the whole crew.
__device__ __forceinline__ void number_members(const TokenSet &set, uint32_t words, const Crew &crew) {
    __shared__ uint32_t s_sum[kMaxThreads / 32];
    const uint32_t threads = crew.threads, tid = crew.rank, lane = tid & 31, warp = tid >> 5;
    const uint32_t per = (words + threads - 1) / threads, begin = min(tid * per, words), end = min(begin + per, words);
    uint32_t mine = 0;
    for (uint32_t w = begin; w < end; ++w) mine += __popc(set.bits[w]);
    const uint32_t upto = warp_inclusive_scan(mine, lane);
    if (lane == 31) s_sum[warp] = upto;
    crew.sync();
    const uint32_t warps = warp_inclusive_scan(lane < threads / 32 ? s_sum[lane] : 0, lane);      // sums up to each warp
    const uint32_t total = __shfl_sync(kFullMask, warps, 31), earlier = __shfl_sync(kFullMask, warps, (warp + 31) & 31);
    uint32_t sum = upto - mine + (warp > 0 ? earlier : 0);
    for (uint32_t w = begin; w < end; ++w) {
        if (set.narrow) reinterpret_cast<uint16_t *>(set.before)[w] = static_cast<uint16_t>(sum);
        else set.before[w] = sum;
        sum += __popc(set.bits[w]);
    }
    const uint32_t slot_words = set.narrow ? (total + 1) / 2 : total;
    for (uint32_t i = tid; i < slot_words; i += threads) set.slots[i] = 0;
    crew.sync();
}

// The biased tokens of a piece, each with its last entry: an open hash table, at most three quarters full.
struct BiasTable {
    uint2 *entries;      // token (kNowhere: free), entry + 1; null: no biases
    uint32_t mask;

    __device__ __forceinline__ uint32_t start(uint32_t at) const { return (at * 2654435761u >> 12) & mask; }
    __device__ __forceinline__ void add(uint32_t at, uint32_t entry) const {
        if (at == kNowhere) return;
        for (uint32_t h = start(at), n = 0; n <= mask; h = (h + 1) & mask, ++n) {
            const uint32_t was = atomicCAS(&entries[h].x, kNowhere, at);
            if (was != kNowhere && was != at) continue;
            atomicMax(&entries[h].y, entry + 1);
            return;
        }
    }
    __device__ __forceinline__ uint32_t find(uint32_t at) const {        // entry + 1, 0: none
        for (uint32_t h = start(at), n = 0; n <= mask; h = (h + 1) & mask, ++n) {
            const uint2 e = entries[h];
            if (e.x == at) return e.y;
            if (e.x == kNowhere) return 0;
        }
        return 0;
    }
};

// A piece of a row: its first token (a vector may begin before the row), and its tokens.
struct Range {
    int32_t first, begin, end;
};

// The history in shared memory, whole or in chunks.  A thread copies tokens rank, rank +
// threads, ... without registers, and looks at no others, so that it waits for its own copies
// alone.
struct History {
    const char *row;         // the row's tokens
    uint32_t *data;
    uint32_t length, words;  // tokens; words of each
    bool whole;              // a chunk is all of it

    __device__ __forceinline__ uint32_t chunk() const { return whole ? length : kChunk; }
    __device__ __forceinline__ uint32_t chunks() const { return whole ? 1 : (length + kChunk - 1) / kChunk; }
    __device__ __forceinline__ uint32_t size(uint32_t c) const { return min(chunk(), length - c * kChunk); }
    __device__ __forceinline__ uint32_t *slot(uint32_t c, uint32_t i) const { return data + ((c % kChunks) * kChunk + i) * words; }
    __device__ __forceinline__ void fetch(uint32_t c, uint32_t rank, uint32_t threads) const {
        if (c < chunks()) {
            const char *from = row + static_cast<size_t>(c) * kChunk * words * 4;
            for (uint32_t i = rank; i < size(c); i += threads) {
                if (words == 1) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(slot(c, i))), "l"(from + i * 4) : "memory");
                else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(slot(c, i))), "l"(from + i * 8) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void start(uint32_t rank, uint32_t threads) const {
        for (uint32_t c = 0; c + 1 < kChunks; ++c) fetch(c, rank, threads);
    }
    // The next chunk is asked for, and chunk c there.
    __device__ __forceinline__ void next(uint32_t c, uint32_t rank, uint32_t threads) const {
        fetch(c + kChunks - 1, rank, threads);
        asm volatile("cp.async.wait_group %0;" ::"n"(kChunks - 1) : "memory");
    }
    // A token as its distance from the piece's first one.  What is no 32-bit number is no token.
    __device__ __forceinline__ uint32_t read(uint32_t c, uint32_t i, const Range &r) const {
        const uint32_t *p = slot(c, i), t = p[0];
        const bool inside = (words == 1 || p[1] == 0) && t - static_cast<uint32_t>(r.begin) < static_cast<uint32_t>(r.end - r.begin);
        return inside ? t - static_cast<uint32_t>(r.first) : kNowhere;
    }
};

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
__global__ void __launch_bounds__(kMaxThreads, 1) k_adjust(const AdjustArgs<T> a) {
    constexpr int N = Wide<T>::kCount;
    constexpr uint32_t kAll = (1u << N) - 1;
    extern __shared__ __align__(128) uint32_t s_words[];
    __shared__ __align__(8) uint64_t s_full[kMostStages];
    const uint32_t row = blockIdx.x / a.pieces, piece = blockIdx.x % a.pieces, tid = threadIdx.x, threads = blockDim.x;
    const T *in = a.in + static_cast<int64_t>(row) * a.in_stride;
    T *out = a.out + static_cast<int64_t>(row) * a.out_stride;
    // elements between the 16-byte boundary at or before the row and the row
    const int32_t shift = a.vectors ? static_cast<int32_t>((reinterpret_cast<uintptr_t>(in) & 15) / sizeof(T)) : 0;
    const int64_t low = static_cast<int64_t>(piece) * a.tokens - shift;
    if (low >= a.vocab) return;
    Range r;
    r.first = static_cast<int32_t>(low);
    r.begin = max(r.first, 0);
    r.end = static_cast<int32_t>(min(low + a.tokens, static_cast<int64_t>(a.vocab)));

    // shared memory: the ring (later the queues), the mask, then what is named
    const uint32_t words = a.tokens / 32;
    uint4 *const ring = reinterpret_cast<uint4 *>(s_words);
    uint32_t *const allowed = a.allowed ? s_words + a.ring_words : nullptr;
    BiasTable biased{nullptr, a.table - 1};
    TokenSet seen{nullptr, nullptr, nullptr, a.narrow};
    uint32_t *space = s_words + a.ring_words + (a.allowed ? words : 0);
    if (!BACK && a.biases > 0) {
        biased.entries = reinterpret_cast<uint2 *>(space);
        space += 2 * a.table;
    }
    if (a.history != nullptr) {
        seen.bits = space;
        seen.before = space + words;
        seen.slots = seen.before + (a.narrow ? words / 2 : words);
        space = BACK ? seen.before : seen.slots + a.slots;
    }
    const History history{static_cast<const char *>(a.history) + static_cast<int64_t>(row) * a.history_stride * a.history_bytes,
                          space + (space - s_words) % 2, a.length, static_cast<uint32_t>(a.history_bytes) / 4, a.history_whole};
    const int64_t bias_row = static_cast<int64_t>(row) * a.bias_stride;
    auto bias_at = [&](uint32_t i) {           // an entry's token as a distance from the piece's first one
        const int64_t t = int_at(a.bias_tokens, a.bias_bytes, bias_row + i);
        return t >= r.begin && t < r.end ? static_cast<uint32_t>(t - r.first) : kNowhere;
    };

    if (tid < a.streamers) {
        // ------------------------------------------------ the logits, masked
        const Crew crew{1, a.streamers, tid};
        // vectors that are whole: not those that the row's start or end cuts
        const uint32_t low_v = r.first < 0 ? 1 : 0, high_v = a.vectors ? static_cast<uint32_t>(r.end - r.first) / N : 0;
        const uint4 *in_v = reinterpret_cast<const uint4 *>(in + r.first);     // read from low_v on
        uint4 *out_v = reinterpret_cast<uint4 *>(out + r.first);
        const uint32_t per_stage = threads * a.stage_vectors;
        auto copy = [&](uint32_t k) {          // the ring's stage k: vectors low_v + k * per_stage ...; thread 0
            const uint32_t from = low_v + k * per_stage;
            if (from >= high_v) return;
            const uint32_t bytes = min(per_stage, high_v - from) * 16, stage = k % a.stages;
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(&s_full[stage], bytes);
            bulk_load(ring + stage * per_stage, in_v + from, bytes, &s_full[stage]);
        };
        // the mask's words ask first: behind the ring's copies each load takes microseconds
        const uint32_t *mask = a.allowed + static_cast<int64_t>(row) * a.allowed_stride;
        const int32_t last = static_cast<int32_t>((a.vocab - 1) / 32);
        const uint32_t off = static_cast<uint32_t>(r.first) & 31;
        const int32_t k0 = r.first >> 5;       // -1 where the first vector begins before the row
        for (uint32_t w = tid * 32; allowed && w < words + 32; w += 32 * a.streamers)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(mask + min(max(k0 + static_cast<int32_t>(w), 0), last)));
        if (tid == 0) {
            for (uint32_t k = 0; k < a.stages; ++k) mbar_init(&s_full[k], 1);
            for (uint32_t k = 0; k < a.stages; ++k) copy(k);
        }
        if (allowed != nullptr) {              // word w: the bits of the piece's tokens 32 w ..
            // words beside the mask's hold no token of the piece
            for (uint32_t w0 = tid; w0 < words; w0 += 8 * a.streamers) {
                uint32_t here[8], next[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int32_t k = k0 + static_cast<int32_t>(w0 + j * a.streamers);
                    here[j] = mask[min(max(k, 0), last)];
                    next[j] = off != 0 ? mask[min(max(k + 1, 0), last)] : 0;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t w = w0 + j * a.streamers;
                    if (w < words) allowed[w] = __funnelshift_r(here[j], next[j], off);
                }
            }
        }
        crew.sync();
        // single elements: of the whole piece where rows lie differently, else of the two
        // vectors that the row's start and end cut
        const int32_t whole = a.vectors ? min(r.first + static_cast<int32_t>(low_v) * N, r.end) : r.end;
        const int32_t rest = a.vectors ? max(r.first + static_cast<int32_t>(high_v) * N, whole) : r.end;
        auto single = [&](int32_t e) { out[e] = !allowed || bits_at(allowed, e - r.first, 1) ? in[e] : from_f32<T>(BACK ? 0.0f : kNegInf); };
        for (int32_t e = r.begin + static_cast<int32_t>(tid); e < whole; e += a.streamers) single(e);
        for (int32_t e = rest + static_cast<int32_t>(tid); e < r.end; e += a.streamers) single(e);
        for (uint32_t k = 0, v0 = low_v; v0 < high_v; ++k, v0 += per_stage) {
            const uint4 *data = ring;
            bool there = true;
            if (a.stages > 0) {
                data += k % a.stages * per_stage;
                there = mbar_wait_bounded(&s_full[k % a.stages], (k / a.stages) & 1, a.waits.of_cta());
            }
#pragma unroll 4
            for (uint32_t i = tid; i < min(per_stage, high_v - v0); i += a.streamers) {
                const uint32_t v = v0 + i, allow = allowed ? bits_at(allowed, v * N, N) : kAll;
                if (a.stages == 0 && allow == kAll) continue;      // in place
                uint4 x = a.stages > 0 ? data[i] : in_v[v];
                if (allowed) mask_vector<T, BACK>(x, allow);
                out_v[v] = x;
            }
            if (a.stages > 0) {
                if (crew.sync_any(!there)) {       // a copy that does not come: what is left is no number
                    for (uint32_t v = v0 + tid; v < high_v; v += a.streamers) out_v[v] = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
                    for (uint32_t i = k; i < k + a.stages && low_v + i * per_stage < high_v; ++i)
                        mbar_wait_bounded(&s_full[i % a.stages], (i / a.stages) & 1, kWaitLimit);
                    break;
                }
                if (tid == 0) copy(k + a.stages);
            }
        }
    } else {
        // ------------------------------------------------ what is named
        const Crew crew{2, threads - a.streamers, tid - a.streamers};
        const uint32_t step = crew.threads, chunks = seen.bits ? history.chunks() : 0;
        if (chunks > 0) history.start(crew.rank, step);
        for (uint32_t w = crew.rank; seen.bits && w < words; w += step) seen.bits[w] = 0;
        for (uint32_t i = crew.rank; biased.entries && i < a.table; i += step) biased.entries[i] = make_uint2(kNowhere, 0);
        crew.sync();
        for (uint32_t c = 0; c < chunks; ++c) {
            history.next(c, crew.rank, step);
#pragma unroll 4
            for (uint32_t i = crew.rank; i < history.size(c); i += step) seen.add(history.read(c, i, r));
        }
        for (uint32_t i = crew.rank; biased.entries && i < a.biases; i += step) biased.add(bias_at(i), i);
        if (chunks > 0 && !history.whole) history.start(crew.rank, step);
        crew.sync();
        if (!BACK && chunks > 0) {
            const uint32_t prompt = a.prompt ? static_cast<uint32_t>(max(a.prompt[row], 0)) : 0;
            number_members(seen, words, crew);
            for (uint32_t c = 0; c < chunks; ++c) {
                if (!history.whole) history.next(c, crew.rank, step);
#pragma unroll 4
                for (uint32_t i = crew.rank; i < history.size(c); i += step) {
                    const uint32_t at = history.read(c, i, r);
                    if (at != kNowhere) seen.count(at, c * kChunk + i < prompt);
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    if (a.streamers == threads) return;

    // ---------------------------------------------- named tokens, anew
    const float repetition = a.repetition ? a.repetition[row] : 1.0f;
    const float presence = !BACK && a.presence ? a.presence[row] : 0.0f, frequency = !BACK && a.frequency ? a.frequency[row] : 0.0f;
    const T *logits = BACK ? a.logits + static_cast<int64_t>(row) * a.logits_stride : nullptr;
    __syncthreads();
    const uint32_t lane = tid & 31;
    // A warp queues its tokens, and asks for their logits, before it writes any: one after another
    // they would each wait for memory.
    const uint32_t room = a.ring_words / 2 / (threads / 32);
    uint32_t queued = 0;
    uint2 *const queue = reinterpret_cast<uint2 *>(s_words) + (tid >> 5) * room;      // where the ring was
    auto serve = [&] {
        __syncwarp();
        for (uint32_t i = lane; i < queued; i += 32) {
            const uint2 q = queue[i];
            const int32_t e = r.first + static_cast<int32_t>(q.x);
            float x = to_f32(in[e]);                           // in place, it holds its value still
            if (BACK) {
                x *= to_f32(logits[e]) > 0.0f ? 1.0f / repetition : repetition;
            } else {
                const uint32_t count = q.y == kNowhere ? seen.counted(q.x) : q.y, times = count & ~kSeenBefore;
                const uint32_t b = biased.entries ? biased.find(q.x) : 0;
                const float by = b != 0 ? a.bias[bias_row + b - 1] : 0.0f;
                if (count != 0) x = x > 0.0f ? x / repetition : x * repetition;
                if (times != 0) x -= fmaf(frequency, static_cast<float>(times), presence);
                if (b != 0) x += by;
            }
            out[e] = from_f32<T>(x);
        }
        queued = 0;
        __syncwarp();
    };
    auto ask = [&](uint32_t token) {
        asm volatile("prefetch.global.L1 [%0];" ::"l"(in + r.first + static_cast<int32_t>(token)));
        if (BACK) asm volatile("prefetch.global.L1 [%0];" ::"l"(logits + r.first + static_cast<int32_t>(token)));
    };
    auto push = [&](uint32_t token, uint32_t count) {          // kNowhere: none
        const bool real = token != kNowhere && (allowed == nullptr || bits_at(allowed, token, 1));
        const uint32_t active = __ballot_sync(kFullMask, real);
        if (real) {
            queue[queued + __popc(active & lanemask_lt())] = make_uint2(token, count);
            ask(token);
        }
        queued += __popc(active);
        if (queued + 32 > room) serve();
    };
    if (seen.bits && a.length <= threads * 4) {  // a short history: the first of a token's places takes it
        for (uint32_t i = tid; i - tid < a.length; i += threads) {
            uint32_t token = i < a.length ? history.read(0, i, r) : kNowhere, count = 0;
            if (token != kNowhere) {
                if (BACK) {
                    if (!seen.take_bit(token)) token = kNowhere;
                } else {
                    count = seen.take(token);
                    if (count == kNowhere) token = kNowhere;
                }
            }
            push(token, count);
        }
    } else if (seen.bits) {
        // of a long one, a thread queues a word's members, whose counts are looked up when the queue is
        // served (a push for each bit of the 32 words, few lanes at a time: 61 us where this takes 53)
        for (uint32_t w = tid; w - lane < words; w += threads) {
            uint32_t bits = w < words ? seen.bits[w] & (allowed ? allowed[w] : ~0u) : 0;
            while (__any_sync(kFullMask, bits != 0)) {
                const uint32_t upto = warp_inclusive_scan(__popc(bits), lane), from = queued;
                const bool fits = from + upto <= room;         // of the first lane that has any, at least
                if (fits)
                    for (uint32_t at = from + upto - __popc(bits); bits != 0; bits &= bits - 1)
                        queue[at++] = make_uint2(w * 32 + __ffs(bits) - 1, kNowhere);
                queued = __reduce_max_sync(kFullMask, fits ? from + upto : from);
                __syncwarp();
                for (uint32_t i = from + lane; i < queued; i += 32) ask(queue[i].x);
                if (queued + 32 > room) serve();
            }
        }
    }
    if (!BACK && biased.entries) {             // biased tokens that are not in the history, by their last entry
        for (uint32_t base = 0; base < a.biases; base += threads) {
            uint32_t token = base + tid < a.biases ? bias_at(base + tid) : kNowhere;
            if (token != kNowhere && (seen.has(token) || biased.find(token) != base + tid + 1)) token = kNowhere;
            push(token, 0);
        }
    }
    serve();
}

}  // namespace

int launch_adjust(const AdjustLaunch &L) {
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int N = Wide<T>::kCount;
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
        a.waits = L.waits;
        // a row has the distance from the boundary of its array and `row` strides
        a.vectors = ((reinterpret_cast<uintptr_t>(L.in) ^ reinterpret_cast<uintptr_t>(L.out)) & 15) == 0 &&
                    (L.rows == 1 || (L.in_stride - L.out_stride) % N == 0);
        const bool history = a.history != nullptr, biases = !L.backward && L.biases > 0, ring = a.vectors && !a.in_place;
        const int64_t span = L.vocab + (a.vectors ? N - 1 : 0);
        int64_t tokens = 0;
        uint32_t threads = 0;
        size_t most_smem = 0, queues = 0;
        auto set_bytes = [&] {
            const int64_t words = tokens / 32, members = std::min(tokens, L.length);
            a.tokens = static_cast<uint32_t>(tokens);
            a.narrow = is_narrow(L.length);
            a.slots = static_cast<uint32_t>(a.narrow ? (members + 1) / 2 : members);
            a.table = 1;
            while (biases && 3 * a.table < 4 * std::min(tokens, L.biases)) a.table *= 2;
            int64_t all = (L.allowed != nullptr ? words : 0) + (biases ? 2 * a.table : 0);
            if (history) all += words + (L.backward ? 0 : (a.narrow ? words / 2 : words) + a.slots);
            if (history) all += 1 + (a.history_whole ? L.length : kChunks * kChunk) * (L.history_bytes / 4);
            return static_cast<size_t>(all) * 4;
        };
        auto stage_bytes = [&] { return static_cast<size_t>(threads) * a.stage_vectors * 16; };
        auto fits = [&] { return set_bytes() + std::max(ring ? 2 * stage_bytes() : 0, queues) <= most_smem; };
        // Pieces that fill the device; false where their sets take too much room.
        auto plan = [&](uint32_t n, size_t smem, int64_t ctas) {
            threads = n;
            most_smem = smem;
            queues = history || biases ? threads / 32 * kQueue * 8 : 0;
            const int64_t least = static_cast<int64_t>(threads) * N;         // a vector for every thread
            const int64_t pieces = std::min(std::max<int64_t>(ctas / L.rows, 1), (L.vocab + least - 1) / least);
            tokens = std::max<int64_t>(256, (std::min<int64_t>(span / pieces + 1, 1 << 18) + 255) / 256 * 256);
            a.stage_vectors = kStageVectors;
            if (!fits()) a.stage_vectors = 1;
            return fits();
        };
        a.history_whole = true;
        if (!plan(512, kHalfSmem, kHalfCtas) && !plan(1024, kWholeSmem, kWholeCtas)) {
            a.history_whole = L.length <= kChunks * kChunk;
            while (!fits()) tokens = (tokens / 2 + 255) / 256 * 256;
        }
        // what is named takes longer where the history is long (256 x 100003 bf16, histories of 16384: 57 us
        // with a quarter of 1024 threads for the logits, 59 with half; 2048 x 131072 with 1024 and its
        // gradient: 376 with half of 512, 385 with a quarter; graph replays)
        a.streamers = !history && !biases ? threads : threads == 1024 ? threads / 4 : threads / 2;
        const size_t sets = set_bytes(), stage = stage_bytes();
        if (ring) {
            const size_t stages = std::min<size_t>((most_smem - sets) / stage, kMostStages);
            a.stages = static_cast<uint32_t>(std::min<size_t>(stages, (tokens / N * 16 + stage - 1) / stage));
        }
        const size_t ring_bytes = std::max(a.stages * stage, queues);
        a.ring_words = static_cast<uint32_t>(ring_bytes / 4);
        a.pieces = static_cast<uint32_t>((span + tokens - 1) / tokens);
        const int64_t blocks = L.rows * a.pieces;
        if (blocks > 0x7FFFFFFF) return static_cast<int>(GSORT_ETOOBIG);
        const size_t smem = sets + ring_bytes;
        const void *kernel = L.backward ? reinterpret_cast<const void *>(k_adjust<T, true>) : reinterpret_cast<const void *>(k_adjust<T, false>);
        if (smem > 40 * 1024 && set_smem_limit(kernel, kWholeSmem) != cudaSuccess) return static_cast<int>(GSORT_ECUDA);
        if (L.backward) k_adjust<T, true><<<static_cast<uint32_t>(blocks), threads, smem, L.stream>>>(a);
        else k_adjust<T, false><<<static_cast<uint32_t>(blocks), threads, smem, L.stream>>>(a);
        return cudaGetLastError() == cudaSuccess ? static_cast<int>(GSORT_OK) : static_cast<int>(GSORT_ECUDA);
    });
}

}  // namespace gsort
