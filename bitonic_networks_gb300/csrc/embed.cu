// embed.cu -- rows of an embedding table by token, and the table's gradient.
//
//   lookup     out[t] = scale * table[tokens[t]], zeros for a token that is not
//              in 0 .. vocab - 1
//   gradient   d_table[v] = scale * sum over t with tokens[t] = v of d_out[t],
//              zeros for a token that does not occur; or, accumulated,
//              d_table[v] += scale * sum, other rows left as they are
//
// The gradient sorts the positions by token (stable, so that the order of every
// sum is given by the input) and sums runs of equal tokens.  The sorted positions
// are cut into equal pieces whatever the tokens are: frequent tokens make long
// runs (in a text one position in twenty may hold the same token), rare ones a run
// of one position, and a piece costs the same either way.  Within a piece a group
// of lanes walks its positions with several rows' loads in flight; runs that cross
// its ends leave partial sums, which are joined in shared memory within a CTA, in the
// order of the positions, and through the workspace between CTAs, in an order that is
// fixed as well (below).  Every row of d_out is read once and every row of d_table
// written once, so the memory bounds it: 65536 rows of 4096 bf16 into 131072 take 270 us (6.0 TB/s), their
// lookup 111 (6.3).  Sums are 32-bit, rounded once.  Rows of tokens that do not
// occur are filled with zeros while the tokens are sorted, which takes few SMs, and
// while the sums run.
#include <algorithm>

#include "row_access.cuh"

namespace gsort {
namespace {

constexpr uint32_t kNoKey = 0xFFFFFFFFu;
constexpr int kEmbedThreads = kRowThreads;
constexpr int kMinLogLanes = 3, kMaxLogLanes = 5;   // lanes side by side on a row
constexpr uint32_t kMaxPer = 128;                   // positions of a group of lanes
constexpr uint32_t kMaxChunk = 1024;                // positions of a CTA
constexpr uint32_t kFillCtas = 608;                 // CTAs that keep a GB300 busy: 4 to an SM

// A CTA that fills rows takes so many bytes: a table of 1 GB of 8 KB rows takes 146 us, 144 with
// half, 151 with twice as many; with 65536 tokens, which make runs of absent rows short, the gradient
// takes 384 us with its lookup, 393 with half.
constexpr int64_t kFillBytes = 128 << 10, kWideRow = 2048;
// Bytes that are filled while the tokens are sorted, by counting or in a cluster; what
// is left is filled beside the sums.
constexpr int64_t kBesideFew = 32 << 20, kBesideCounting = 64 << 20, kBesideCluster = 128 << 20;

// Rows in flight per thread; a shifted one takes two vectors of registers.
template <int MODE> constexpr int kLoads = MODE == kShifted ? 4 : 8;

__device__ __forceinline__ int64_t token_at(const void *tokens, int bytes, int64_t i) {
    return bytes == 8 ? static_cast<const int64_t *>(tokens)[i] : static_cast<const int32_t *>(tokens)[i];
}

// A token as a sort key: what is no token comes last.
__device__ __forceinline__ uint32_t token_key(int64_t token, uint32_t vocab) {
    return static_cast<uint64_t>(token) < vocab ? static_cast<uint32_t>(token) : vocab;
}

// ------------------------------------------------------------------ lookup
template <typename T> struct EmbedArgs {
    const T *table;
    const uint4 *safe;       // 32 bytes that can be read in place of others
    T *out;
    const void *tokens;
    int64_t row_stride;
    float scale;
    int token_bytes;
    uint32_t n, vocab, width, vectors, log_lanes, chunks;
};

template <typename T, int MODE, bool SCALED, int U>
__global__ void __launch_bounds__(kEmbedThreads) k_embed(const EmbedArgs<T> a) {
    constexpr int N = Wide<T>::kCount;
    const uint32_t lanes = 1u << a.log_lanes;
    const uint32_t group = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
    const uint32_t t = group * (kEmbedThreads >> a.log_lanes) + (threadIdx.x >> a.log_lanes);
    if (t >= a.n) return;
    const uint32_t v0 = chunk * lanes * U + (threadIdx.x & (lanes - 1));
    const uint32_t key = token_key(token_at(a.tokens, a.token_bytes, t), a.vocab);
    const bool there = key < a.vocab;
    const uint32_t k = there ? key : 0;
    const InRow<T> in{a.table + static_cast<int64_t>(k) * a.row_stride, k > 0 && k + 1 < a.vocab};
    const OutRow<T, MODE> out(a.out + static_cast<int64_t>(t) * a.width);
    Loaded x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)     // no branch around the loads
        x[u] = start_read<T, MODE>(in, out.at(min(v0 + u * lanes, a.vectors - 1)), a.width, a.safe);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t v = v0 + u * lanes;
        if (v >= a.vectors) continue;
        const int32_t e = out.at(v);
        uint4 q = end_read<T, MODE>(x[u], in, e, a.width);
        if (!there) {
            q = make_uint4(0, 0, 0, 0);
        } else if (SCALED) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) Wide<T>::set_pair(q, i, mul2(pair(a.scale, a.scale), Wide<T>::pair_of(q, i)));
        }
        // what is written is not read here again: the table's rows stay in L2 for tokens that come up again
        if (MODE != kSingle && out.whole(e, a.width)) __stcs(reinterpret_cast<uint4 *>(out.row + e), q);
        else out.write(e, a.width, q);
    }
}

// ------------------------------------------------------------ order by token
// Every token as a key, with its position; and its bit, where they are asked for.
__global__ void __launch_bounds__(256) k_token_keys(const void *tokens, int bytes, uint32_t n, uint32_t vocab, uint32_t *keys,
                                                    uint32_t *positions, uint32_t *bits, uint32_t *counters, uint32_t count) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    for (uint32_t c = i; c < count; c += gridDim.x * 256) counters[c] = 0;
    if (i >= n) return;
    const uint32_t key = token_key(token_at(tokens, bytes, i), vocab);
    keys[i] = key;
    positions[i] = i;
    // frequent tokens find their bit set
    if (bits != nullptr && key < vocab && !(ld_relaxed(bits + key / 32) >> (key & 31) & 1)) atomicOr(bits + key / 32, 1u << (key & 31));
}

// --------------------------------------------- rows of tokens that do not occur
struct FillArgs {
    char *table;
    int64_t stride, row_bytes;     // in bytes, even
    uint32_t vocab;
    uint32_t rows;                 // of a CTA, at most 256
    uint32_t first;                // CTA's number of the grid's first one
    const uint32_t *bits;          // a bit for each token that occurs; null: the CTA looks at the tokens itself
    const void *tokens;
    int token_bytes;
    uint32_t n;
};

// THREADS threads write a span of bytes with what `word` has twice.
template <uint32_t THREADS> __device__ __forceinline__ void fill_span(char *p, int64_t bytes, uint32_t word) {
    const uint32_t rank = threadIdx.x % THREADS;
    const int64_t head = min(static_cast<int64_t>(-reinterpret_cast<intptr_t>(p) & 15), bytes);
    const int64_t vectors = (bytes - head) / 16, tail = head + vectors * 16;
    if (rank < head / 2) reinterpret_cast<uint16_t *>(p)[rank] = static_cast<uint16_t>(word);
    uint4 *v = reinterpret_cast<uint4 *>(p + head);
#pragma unroll 4
    for (int64_t i = rank; i < vectors; i += THREADS) v[i] = make_uint4(word, word, word, word);
    if (rank < (bytes - tail) / 2) reinterpret_cast<uint16_t *>(p + tail)[rank] = static_cast<uint16_t>(word);
}

// Fills the absent rows of CTA number `block`.  The CTA writes a run of them as a whole (400 MB
// of rows of 4004 bytes take 57 us so, 7.0 TB/s, and 63 with a run to each warp), short rows by
// warps.
__device__ __forceinline__ void fill_absent(const FillArgs &a, uint32_t block) {
    __shared__ uint32_t s_bits[9];     // of 256 tokens, from any bit of the first word on
    const uint32_t base = block * a.rows, rows = min(a.rows, a.vocab - base), tid = threadIdx.x;
    const uint32_t shift = a.bits != nullptr ? base & 31 : 0;      // the bit of token `base`
    if (tid < 9) s_bits[tid] = a.bits != nullptr && base / 32 + tid < (a.vocab + 31) / 32 ? a.bits[base / 32 + tid] : 0;
    __syncthreads();
    if (a.bits == nullptr) {
#pragma unroll 8
        for (uint32_t i = tid; i < a.n; i += kEmbedThreads) {
            const int64_t t = token_at(a.tokens, a.token_bytes, i) - base;
            if (t >= 0 && t < rows) atomicOr(s_bits + t / 32, 1u << (t & 31));
        }
        __syncthreads();
    }
    // the first row from r on that is present (or absent), `to` at most
    auto find = [&](uint32_t r, uint32_t to, bool present) {
        while (r < to) {
            const uint32_t at = shift + r, left = 32 - (at & 31);
            const uint32_t w = (present ? s_bits[at / 32] : ~s_bits[at / 32]) >> (at & 31);
            if (w != 0) return min(r + __ffs(w) - 1, to);          // zeros are shifted in
            r += left;
        }
        return to;
    };
    auto fill = [&](auto team, uint32_t from, uint32_t to) {
        for (uint32_t r = find(from, to, false); r < to;) {
            const uint32_t end = find(r, to, true), run = a.stride == a.row_bytes ? end - r : 1;   // without gaps, rows are one span
            for (; r < end; r += run)
                fill_span<decltype(team)::value>(a.table + (base + static_cast<int64_t>(r)) * a.stride, run * a.row_bytes, 0);
            r = find(end, to, false);
        }
    };
    if (a.row_bytes >= kWideRow) {
        fill(std::integral_constant<uint32_t, kEmbedThreads>{}, 0, rows);
    } else {
        const uint32_t per = (rows + 7) / 8, from = min(tid / 32 * per, rows);
        fill(std::integral_constant<uint32_t, 32>{}, from, min(from + per, rows));
    }
}

// Beside the kernel that precedes it in the stream: neither needs the other.  What follows
// waits for both.
__global__ void __launch_bounds__(256) k_fill_absent(const FillArgs a) {
    fill_absent(a, a.first + blockIdx.x);
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Few tokens are sorted by counting: a token's place is the number of tokens that
// are smaller, or equal and before it.  A lane holds a token, a warp compares
// its 32 tokens with an eighth of all (a broadcast from shared memory each).  The
// CTAs behind those of the tokens fill absent rows.
constexpr uint32_t kRankMax = 8192;
// Up to so many tokens, and more of them where few CTAs fill, each CTA that fills looks at the
// tokens itself: two launches instead of five (3500 tokens, a table of 2890 x 120 f32: 18 us, 24 with five).
constexpr uint32_t kFewTokens = 2048, kFewFills = 1216;

__global__ void __launch_bounds__(256) k_token_rank(const void *tokens, int bytes, uint32_t n, uint32_t vocab, uint32_t *keys,
                                                    uint32_t *order, uint32_t *status, uint32_t *counters, uint32_t count,
                                                    const FillArgs fill) {
    extern __shared__ __align__(16) uint32_t s_keys[];   // n rounded up to 32
    __shared__ uint32_t s_rank[8][32];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, groups = (n + 31) / 32;
    if (blockIdx.x >= groups) {
        fill_absent(fill, blockIdx.x - groups);
        return;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;              // of the call: this sort cannot fail
    for (uint32_t c = blockIdx.x * 256 + threadIdx.x; c < count; c += groups * 256) counters[c] = 0;
    for (uint32_t i = threadIdx.x; i < groups * 32; i += 256)
        s_keys[i] = i < n ? token_key(token_at(tokens, bytes, i), vocab) : kNoKey;   // behind every token
    __syncthreads();
    const uint32_t i = blockIdx.x * 32 + lane, mine = s_keys[i];
    uint32_t rank = 0;
    for (uint32_t g = warp; g < groups; g += 8) {
        const uint4 *q = reinterpret_cast<const uint4 *>(s_keys + g * 32);
        if (g < blockIdx.x) {              // equal ones are before
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint4 k = q[j];
                rank += (k.x <= mine) + (k.y <= mine) + (k.z <= mine) + (k.w <= mine);
            }
        } else if (g > blockIdx.x) {       // equal ones are behind
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint4 k = q[j];
                rank += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
            }
        } else {
#pragma unroll
            for (uint32_t j = 0; j < 32; ++j) {
                const uint32_t k = s_keys[g * 32 + j];
                rank += k < mine || (k == mine && j < lane);
            }
        }
    }
    s_rank[warp][lane] = rank;
    __syncthreads();
    if (warp == 0 && i < n) {
        rank = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) rank += s_rank[w][lane];
        keys[rank] = mine;
        order[rank] = i;
    }
}

// More of them are sorted in two steps.  Runs of 256 tokens, by counting within the run; bits, where they
// are asked for, and the call's counters and status on the way.
constexpr uint32_t kRun = 256;

__global__ void __launch_bounds__(kRun) k_token_runs(const void *tokens, int bytes, uint32_t n, uint32_t vocab, uint32_t *keys, uint32_t *order,
                                                     uint32_t *bits, uint32_t *status, uint32_t *counters, uint32_t count) {
    __shared__ __align__(16) uint32_t s_keys[kRun];
    const uint32_t tid = threadIdx.x, base = blockIdx.x * kRun, i = base + tid, group = tid / 32, lane = tid & 31;
    for (uint32_t c = i; c < count; c += gridDim.x * kRun) counters[c] = 0;
    if (i == 0) *status = 0;             // this sort cannot fail
    const uint32_t mine = i < n ? token_key(token_at(tokens, bytes, i), vocab) : kNoKey;       // behind every token
    s_keys[tid] = mine;
    if (bits != nullptr && mine < vocab && !(ld_relaxed(bits + mine / 32) >> (mine & 31) & 1)) atomicOr(bits + mine / 32, 1u << (mine & 31));
    __syncthreads();
    uint32_t rank = 0;
#pragma unroll 2
    for (uint32_t g = 0; g < kRun / 32; ++g) {
        const uint4 *q = reinterpret_cast<const uint4 *>(s_keys + g * 32);
        const uint32_t limit = mine + (g < group);         // equal ones before are counted
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
            const uint4 k = q[j];
            if (g == group) {
                rank += (k.x < mine || (k.x == mine && 4 * j < lane)) + (k.y < mine || (k.y == mine && 4 * j + 1 < lane)) +
                        (k.z < mine || (k.z == mine && 4 * j + 2 < lane)) + (k.w < mine || (k.w == mine && 4 * j + 3 < lane));
            } else {
                rank += (k.x < limit) + (k.y < limit) + (k.z < limit) + (k.w < limit);
            }
        }
    }
    if (i < n) {
        keys[base + rank] = mine;
        order[base + rank] = i;
    }
}

// Joins the runs: a token's place is the number of tokens before it in every run, found by
// halving.  A lane holds a token, a warp looks at an eighth of the runs.  (8000 tokens added to a
// table of 32000 x 512 bf16 take 25 us so, 29 by counting among all of them.)
__global__ void __launch_bounds__(256) k_token_join(const uint32_t *run_keys, const uint32_t *run_order, uint32_t n, uint32_t *keys, uint32_t *order) {
    extern __shared__ __align__(16) uint32_t s_keys[];       // n
    __shared__ uint32_t s_rank[8][32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");       // rows are filled meanwhile
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, runs = (n + kRun - 1) / kRun;
#pragma unroll 8
    for (uint32_t i = threadIdx.x; i < n; i += 256) s_keys[i] = run_keys[i];
    __syncthreads();
    const uint32_t i = blockIdx.x * 32 + lane, own = blockIdx.x * 32 / kRun, mine = i < n ? s_keys[i] : 0;
    uint32_t rank = 0;
#pragma unroll 2
    for (uint32_t b = warp; b < runs; b += 8) {
        const uint32_t *run = s_keys + b * kRun;
        const uint32_t size = min(kRun, n - b * kRun), limit = mine + (b < own);       // equal ones of earlier runs are before
        if (b == own) {
            rank += i - own * kRun;
            continue;
        }
        uint32_t low = 0;                  // keys of the run below the limit
#pragma unroll
        for (uint32_t step = kRun / 2; step > 0; step /= 2)
            if (low + step <= size && run[low + step - 1] < limit) low += step;
        if (low < size && run[low] < limit) ++low;
        rank += low;
    }
    s_rank[warp][lane] = rank;
    __syncthreads();
    if (warp == 0 && i < n) {
        rank = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) rank += s_rank[w][lane];
        keys[rank] = mine;
        order[rank] = run_order[i];
    }
}

// ---------------------------------------------------------------- gradient
template <typename T> struct EmbedSumArgs {
    const T *d;
    const uint4 *safe;
    T *out;
    const uint32_t *keys, *order;    // sorted
    const void *tokens;
    const uint32_t *status;          // of the sort; null: it cannot fail
    float *partials;                 // [chunks][2][slabs * lanes][N]: sums up to a chunk's end and from its start
    uint32_t *counters;              // [chunks][slabs], zeros: parts of a run that began in the chunk
    int64_t d_stride, out_stride;
    float scale;
    bool accumulate, wide;           // wide: tokens of 8 bytes (as an int of its own it made ptxas spill: shifted rows 3 % slower)
    uint32_t n, vocab, width, vectors;
    uint32_t log_lanes, slabs;       // 2^log_lanes lanes hold a vector each; slabs of them make a row
    uint32_t per;                    // positions of a group of lanes
    uint32_t chunks;                 // of (256 >> log_lanes) * per positions
};

template <typename T, int MODE> struct RowSum {
    static constexpr int N = Wide<T>::kCount;
    Pair p[N / 2];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) p[i] = pair(0.0f, 0.0f);
    }
    __device__ __forceinline__ void add(const uint4 &q) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) p[i] = add2(p[i], Wide<T>::pair_of(q, i));
    }
    __device__ __forceinline__ void add(const float *f) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) add4(i, reinterpret_cast<const float4 *>(f)[i]);
    }
    __device__ __forceinline__ void add_other(const float *f) {       // of another CTA: from L2
#pragma unroll
        for (int i = 0; i < N / 4; ++i) add4(i, __ldcg(reinterpret_cast<const float4 *>(f) + i));
    }
    __device__ __forceinline__ void add4(int i, const float4 &x) {
        {
            p[2 * i] = add2(p[2 * i], pair(x.x, x.y));
            p[2 * i + 1] = add2(p[2 * i + 1], pair(x.z, x.w));
        }
    }
    __device__ __forceinline__ void store(float *f) const {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            reinterpret_cast<float4 *>(f)[i] = make_float4(p[2 * i].f.x, p[2 * i].f.y, p[2 * i + 1].f.x, p[2 * i + 1].f.y);
    }
    // The run's sum to its row of the table.
    __device__ __forceinline__ void write(const EmbedSumArgs<T> &a, uint32_t key, uint32_t v) const {
        const OutRow<T, MODE> out(a.out + static_cast<int64_t>(key) * a.out_stride);
        const int32_t e = out.at(v);
        uint4 q;
        if (a.accumulate) {
            if (MODE != kSingle && out.whole(e, a.width)) {
                q = *reinterpret_cast<const uint4 *>(out.row + e);
            } else {
                float f[N];
#pragma unroll
                for (int i = 0; i < N; ++i)
                    f[i] = static_cast<uint32_t>(e + i * kStep<MODE>) < a.width ? to_f32(out.row[e + i * kStep<MODE>]) : 0.0f;
#pragma unroll
                for (int i = 0; i < N / 2; ++i) Wide<T>::set_pair(q, i, pair(f[2 * i], f[2 * i + 1]));
            }
#pragma unroll
            for (int i = 0; i < N / 2; ++i) Wide<T>::set_pair(q, i, fma2(p[i], pair(a.scale, a.scale), Wide<T>::pair_of(q, i)));
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) Wide<T>::set_pair(q, i, mul2(p[i], pair(a.scale, a.scale)));
        }
        out.write(e, a.width, q);
    }
};

// Rows of tokens that occur become NaN.
template <typename T> __device__ __forceinline__ void void_rows(const EmbedSumArgs<T> &a) {
    for (uint32_t i = blockIdx.x; i < a.n; i += gridDim.x) {
        const uint32_t key = token_key(token_at(a.tokens, a.wide ? 8 : 4, i), a.vocab);
        if (key < a.vocab)
            fill_span<kEmbedThreads>(reinterpret_cast<char *>(a.out + static_cast<int64_t>(key) * a.out_stride),
                                     static_cast<int64_t>(a.width) * sizeof(T), 0x7FFF7FFFu);
    }
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kEmbedThreads, 4) k_embed_sum(const EmbedSumArgs<T> a) {
    constexpr int N = Wide<T>::kCount, U = kLoads<MODE>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");       // rows are filled meanwhile
    if (a.status != nullptr && *a.status != 0) {       // the sort gave up, its results are void: rows of tokens that occur are NaN
        void_rows(a);
        return;
    }
    __shared__ uint32_t s_key[kMaxChunk + 2], s_order[kMaxChunk];   // s_key[0]: the key before the chunk
    __shared__ __align__(16) float s_head[kEmbedThreads][N];
    __shared__ uint32_t s_last;
    const uint32_t chunk = blockIdx.x / a.slabs, slab = blockIdx.x % a.slabs;
    const uint32_t lanes = 1u << a.log_lanes, units = kEmbedThreads >> a.log_lanes, size = units * a.per;
    const uint32_t base = chunk * size, count = min(size, a.n - base), tid = threadIdx.x;
    // keys at the ends of the chunks before and behind, to find where runs begin and end
    const uint64_t behind_at = (static_cast<uint64_t>(chunk) + 1 + tid) * size;
    const uint32_t key_before = tid + 1 < chunk ? a.keys[static_cast<size_t>(chunk - 1 - tid) * size - 1] : kNoKey;
    const uint32_t key_behind = behind_at < a.n ? a.keys[behind_at] : kNoKey;
    for (uint32_t i = tid; i < count + 2; i += kEmbedThreads) {
        const uint32_t p = base + i - 1;
        s_key[i] = p < a.n ? a.keys[p] : kNoKey;
    }
    for (uint32_t i = tid; i < count; i += kEmbedThreads) s_order[i] = a.order[base + i];
    __syncthreads();
    const uint32_t unit = tid >> a.log_lanes, v = slab * lanes + (tid & (lanes - 1)), vv = min(v, a.vectors - 1);
    const uint32_t begin = unit * a.per, end = min(begin + a.per, count);
    const bool any = begin < end && s_key[begin + 1] < a.vocab;
    uint32_t key = any ? s_key[begin + 1] : kNoKey;
    const bool head = any && s_key[begin] == key;      // the run began before this unit
    bool first = head;
    RowSum<T, MODE> sum;
    sum.clear();
    if (any) {
        for (uint32_t p0 = begin; p0 < end; p0 += U) {
            Loaded x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t p = min(p0 + u, end - 1), k = s_key[p + 1], o = s_order[p];
                const uint32_t row = o < a.n ? o : 0;
                const OutRow<T, MODE> out(a.out + static_cast<int64_t>(k < a.vocab ? k : 0) * a.out_stride);
                x[u] = start_read<T, MODE>(InRow<T>{a.d + static_cast<int64_t>(row) * a.d_stride, row > 0 && row + 1 < a.n}, out.at(vv),
                                           a.width, a.safe);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t p = p0 + u;
                if (p >= end) continue;
                const uint32_t k = s_key[p + 1], o = s_order[p];
                if (k != key) {
                    if (key < a.vocab) {
                        if (first) sum.store(s_head[tid]);
                        else if (v < a.vectors) sum.write(a, key, v);
                    }
                    first = false;
                    key = k;
                    sum.clear();
                }
                if (k >= a.vocab) continue;
                const uint32_t row = o < a.n ? o : 0;
                const OutRow<T, MODE> out(a.out + static_cast<int64_t>(k) * a.out_stride);
                sum.add(end_read<T, MODE>(x[u], InRow<T>{a.d + static_cast<int64_t>(row) * a.d_stride, row > 0 && row + 1 < a.n}, out.at(vv),
                                          a.width));
            }
        }
        if (key >= a.vocab) key = kNoKey;
        if (key != kNoKey && first) sum.store(s_head[tid]);    // the whole unit is a part of one run
    }
    __syncthreads();
    // Runs that go on behind the unit they began in: that unit joins their parts.
    // The chunk's first unit does so for a run that began before the chunk.
    const bool onward = any && key != kNoKey && s_key[end + 1] == key;
    const size_t row = static_cast<size_t>(a.slabs) * lanes * N;           // of partial sums
    float *const mine = a.partials + static_cast<size_t>(chunk) * 2 * row + static_cast<size_t>(v) * N;
    if (any && unit == 0 && head) {
        const uint32_t k0 = s_key[1];
        RowSum<T, MODE> part;
        part.clear();
        part.add(s_head[tid]);
        if (first && onward) {             // the run covers this unit
            for (uint32_t i = 1; i < units && i * a.per < count && s_key[i * a.per + 1] == k0; ++i) {
                part.add(s_head[(i << a.log_lanes) + (tid & (lanes - 1))]);
                if (s_key[min((i + 1) * a.per, count)] != k0) break;
            }
        }
        part.store(mine + row);
    }
    if (any && key != kNoKey && !first) {  // a run that began here
        bool leaves = onward;              // the chunk
        for (uint32_t i = unit + 1; leaves && i < units && i * a.per < count; ++i) {
            sum.add(s_head[(i << a.log_lanes) + (tid & (lanes - 1))]);
            const uint32_t stop = min((i + 1) * a.per, count);
            leaves = s_key[stop] == key && s_key[stop + 1] == key;
        }
        if (leaves) sum.store(mine);
        else if (v < a.vectors) sum.write(a, key, v);
    }
    // A run that crosses ends of chunks has a part in each of them.  The CTA that
    // writes the last of these joins them: each group of lanes every units-th part, then the
    // groups' sums one after the other.  Tokens and sizes give that order, not the CTAs' times.
    const uint32_t front = s_key[1], back = s_key[count], next = s_key[count + 1];
    const bool before = s_key[0] == front && front < a.vocab;
    const bool behind = next == back && back < a.vocab;
    for (int r = 0; r < 2; ++r) {          // the run at the chunk's start, and another one at its end
        if (r == 0 ? !before : !(behind && !(before && front == back))) continue;
        const uint32_t k = r == 0 ? front : back;
        uint32_t from = chunk, to = chunk;
        if (r == 0) {                      // the chunk it began in
            for (from = chunk - 1;; from -= kEmbedThreads) {
                const uint32_t c = from - tid;
                const uint32_t held = __syncthreads_count(from == chunk - 1 ? key_before == k
                                                                           : tid < from && a.keys[static_cast<size_t>(c) * size - 1] == k);
                if (held < kEmbedThreads) {
                    from -= held;
                    break;
                }
            }
        }
        if (r == 1 || (behind && front == back)) {       // the chunk it ends in
            for (;; to += kEmbedThreads) {
                const uint64_t p = static_cast<uint64_t>(to + 1 + tid) * size;
                const uint32_t held = __syncthreads_count(to == chunk ? key_behind == k : p < a.n && a.keys[p] == k);
                if (held < kEmbedThreads) {
                    to += held;
                    break;
                }
            }
        }
        __threadfence();                   // this thread's part, before the count
        __syncthreads();
        if (tid == 0) s_last = atomicAdd(a.counters + static_cast<size_t>(from) * a.slabs + slab, 1u) == to - from;
        __syncthreads();
        if (!s_last) continue;
        __threadfence();
        sum.clear();
        const float *parts = a.partials + static_cast<size_t>(v) * N;
        if (unit == 0) sum.add_other(parts + static_cast<size_t>(from) * 2 * row);
#pragma unroll 4
        for (uint32_t c = from + 1 + unit; c <= to; c += units) sum.add_other(parts + (static_cast<size_t>(c) * 2 + 1) * row);
        sum.store(s_head[tid]);
        __syncthreads();
        if (unit == 0) {
            for (uint32_t i = 1; i < min(units, to - from); ++i) sum.add(s_head[(i << a.log_lanes) + tid]);
            if (v < a.vectors) sum.write(a, k, v);
        }
        __syncthreads();
    }
}

// A launch that may start while the kernel before it in the stream runs, as soon as that allows it.
template <typename A> int launch_early(void (*kernel)(const A), uint32_t ctas, cudaStream_t stream, const A &a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kEmbedThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? GSORT_OK : GSORT_ECUDA;
}

// ------------------------------------------------------------------- plans
// How the gradient's work is cut: by sizes alone, so that the order of every sum
// depends on nothing else.
struct EmbedPlan {
    uint32_t vectors_max, log_lanes, slabs, per, chunks;
    size_t keys, order, keys_in, order_in, radix, bits, partials, counters, total;
};

EmbedPlan embed_plan(uint32_t n, uint32_t vocab, uint32_t width, int size) {
    EmbedPlan p{};
    const uint32_t count = 16 / size;
    // a row touches so many vectors at most, however it lies
    p.vectors_max = size == 4 ? (width + 127) / 128 * 32 : (width + 2 * (count - 1)) / count;
    p.log_lanes = kMinLogLanes;
    while (p.log_lanes < kMaxLogLanes && (1u << p.log_lanes) < p.vectors_max) ++p.log_lanes;
    const uint32_t lanes = 1u << p.log_lanes, units = kEmbedThreads / lanes;
    p.slabs = (p.vectors_max + lanes - 1) / lanes;
    // longer pieces leave fewer partial sums, shorter ones fill the device
    p.per = std::min(kMaxPer, kMaxChunk / units);
    while (p.per > 8 && static_cast<uint64_t>((n + units * p.per - 1) / (units * p.per)) * p.slabs < kFillCtas) p.per /= 2;
    p.chunks = (n + units * p.per - 1) / (units * p.per);
    const size_t bytes = align_up(static_cast<size_t>(n) * 4, kWsAlign);
    size_t at = 0;
    if (n > kRankMax) {          // the sort's header comes first: its status is the call's
        p.radix = at;
        at += align_up(radix_layout(n, true, 4).total, kWsAlign);
    } else {
        at += kWsAlign;          // the status alone
    }
    if (n > kFewTokens) {
        p.keys_in = at;
        at += bytes;
        p.order_in = at;
        at += bytes;
        p.bits = at;
        at += align_up((static_cast<size_t>(vocab) + 31) / 32 * 4, kWsAlign);
    }
    p.keys = at;
    at += bytes;
    p.order = at;
    at += bytes;
    p.partials = at;
    if (p.chunks > 1) at += static_cast<size_t>(p.chunks) * 2 * p.slabs * lanes * (16 / size) * 4;
    p.counters = at;
    if (p.chunks > 1) at += static_cast<size_t>(p.chunks) * p.slabs * 4;
    p.total = align_up(at, kWsAlign);
    return p;
}

}  // namespace

size_t embed_workspace_bytes(int64_t tokens, int64_t vocab, int64_t width, int dtype) {
    return embed_plan(static_cast<uint32_t>(tokens), static_cast<uint32_t>(vocab), static_cast<uint32_t>(width), float_bytes(dtype)).total;
}

int launch_embed(const EmbedLaunch &L) {
    using std::integral_constant;
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int N = Wide<T>::kCount;
        EmbedArgs<T> a{};
        a.table = static_cast<const T *>(L.in);
        a.safe = safe_in(L.in);
        a.out = static_cast<T *>(L.out);
        a.tokens = L.tokens;
        a.token_bytes = L.token_bytes;
        a.row_stride = L.in_stride;
        a.scale = L.scale;
        a.n = static_cast<uint32_t>(L.n);
        a.vocab = static_cast<uint32_t>(L.vocab);
        a.width = static_cast<uint32_t>(L.width);
        auto start = [&](auto m) {
            constexpr int MODE = decltype(m)::value, U = 4;
            a.log_lanes = lanes_for(a.vectors, U);
            const uint32_t step = U << a.log_lanes, rows = kEmbedThreads >> a.log_lanes;
            a.chunks = (a.vectors + step - 1) / step;
            const int64_t blocks = static_cast<int64_t>((a.n + rows - 1) / rows) * a.chunks;
            if (blocks > 0x7FFFFFFF) return static_cast<int>(GSORT_ETOOBIG);
            const dim3 grid(static_cast<uint32_t>(blocks));
            if (L.scale == 1.0f) k_embed<T, MODE, false, U><<<grid, kEmbedThreads, 0, L.stream>>>(a);
            else k_embed<T, MODE, true, U><<<grid, kEmbedThreads, 0, L.stream>>>(a);
            return launch_status();
        };
        if (L.width % N == 0 && aligned(L.in, 16) && aligned(L.out, 16) && L.in_stride % N == 0) {
            a.vectors = a.width / N;
            return start(integral_constant<int, kAligned>{});
        }
        a.vectors = (a.width + 2 * (N - 1)) / N;
        if (L.width * sizeof(T) >= 64) return start(integral_constant<int, kShifted>{});
        return start(integral_constant<int, kElements>{});
    });
}

int launch_embed_backward(const EmbedBackwardLaunch &L) {
    using std::integral_constant;
    const uint32_t n = static_cast<uint32_t>(L.n), vocab = static_cast<uint32_t>(L.vocab);
    const EmbedPlan plan = embed_plan(n, vocab, static_cast<uint32_t>(L.width), float_bytes(L.dtype));
    uint32_t *keys = reinterpret_cast<uint32_t *>(L.ws + plan.keys), *order = reinterpret_cast<uint32_t *>(L.ws + plan.order);
    FillArgs fill{};
    fill.table = static_cast<char *>(L.d_table);
    fill.row_bytes = L.width * float_bytes(L.dtype);
    fill.stride = L.table_stride * float_bytes(L.dtype);
    fill.vocab = vocab;
    fill.tokens = L.tokens;
    fill.token_bytes = L.token_bytes;
    fill.n = n;
    // fewer of a small table, to fill the device
    fill.rows = static_cast<uint32_t>(std::max<int64_t>(1, std::min({static_cast<int64_t>(256), kFillBytes / fill.row_bytes, std::max<int64_t>(8, vocab / kFillCtas)})));
    const uint32_t fill_ctas = L.accumulate ? 0 : (vocab + fill.rows - 1) / fill.rows;
    uint32_t *counters = reinterpret_cast<uint32_t *>(L.ws + plan.counters), *status = reinterpret_cast<uint32_t *>(L.ws + kHdrStatus);
    const uint64_t sums = static_cast<uint64_t>(plan.chunks) * plan.slabs;
    const uint32_t count = plan.chunks > 1 ? static_cast<uint32_t>(sums) : 0;
    if (sums > 0x7FFFFFFF) return GSORT_ETOOBIG;
    const uint32_t groups = (n + 31) / 32;
    auto start_fill = [&](uint32_t from, uint32_t to) {
        fill.first = from;
        return from < to ? launch_early(k_fill_absent, to - from, L.stream, fill) : static_cast<int>(GSORT_OK);
    };
    const bool few = n <= kFewTokens || (n <= 2 * kFewTokens && static_cast<int64_t>(fill_ctas) * n <= static_cast<int64_t>(kFewFills) * kFewTokens);
    // of the CTAs that fill, those before the sums
    const int64_t beside = few ? kBesideFew : n <= kRankMax ? kBesideCounting : cluster_sort_applies(n, 4, 0, L.waits.stall, 1) ? kBesideCluster : 0;
    const uint32_t filled = n == 0 ? fill_ctas : static_cast<uint32_t>(std::min<int64_t>(fill_ctas, beside / (fill.row_bytes * fill.rows)));
    if (few) {
        if (groups == 0 && fill_ctas == 0) return GSORT_OK;
        k_token_rank<<<groups + filled, 256, groups * 32 * 4, L.stream>>>(L.tokens, L.token_bytes, n, vocab, keys, order, status, counters, count, fill);
        if (cudaGetLastError() != cudaSuccess) return GSORT_ECUDA;
    } else {
        uint32_t *keys_in = reinterpret_cast<uint32_t *>(L.ws + plan.keys_in);
        uint32_t *order_in = reinterpret_cast<uint32_t *>(L.ws + plan.order_in);
        uint32_t *bits = L.accumulate ? nullptr : reinterpret_cast<uint32_t *>(L.ws + plan.bits);
        if (bits && cudaMemsetAsync(bits, 0, (static_cast<size_t>(vocab) + 31) / 32 * 4, L.stream) != cudaSuccess) return GSORT_ECUDA;
        if (n <= kRankMax) {
            k_token_runs<<<(n + kRun - 1) / kRun, kRun, 0, L.stream>>>(L.tokens, L.token_bytes, n, vocab, keys_in, order_in, bits, status, counters, count);
            if (cudaGetLastError() != cudaSuccess) return GSORT_ECUDA;
            k_token_join<<<groups, 256, n * 4, L.stream>>>(keys_in, order_in, n, keys, order);
            if (cudaGetLastError() != cudaSuccess) return GSORT_ECUDA;
        } else {
            k_token_keys<<<(n + 255) / 256, 256, 0, L.stream>>>(L.tokens, L.token_bytes, n, vocab, keys_in, order_in, bits, counters, count);
            if (cudaGetLastError() != cudaSuccess) return GSORT_ECUDA;
            RadixLaunch R{};
            R.keys_in = keys_in;
            R.keys_out = keys;
            R.vals_in = order_in;
            R.vals_out = order;
            R.n = n;
            R.kind = GSORT_KEY_U32;
            R.end_bit = 32 - __builtin_clz(vocab);       // what is no token has the key `vocab`
            R.ws = L.ws + plan.radix;
            R.spin_limit = L.waits.polls;
            R.stall_tile = L.waits.stall;
            R.stream = L.stream;
            R.sm_count = L.sm_count;
            R.next_early = fill_ctas > 0;
            const int rc = launch_radix(R);
            if (rc != GSORT_OK) return rc;
        }
        fill.bits = bits;
        if (start_fill(0, filled) != GSORT_OK) return GSORT_ECUDA;
    }
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int N = Wide<T>::kCount;
        EmbedSumArgs<T> a{};
        a.d = static_cast<const T *>(L.d_out);
        a.safe = safe_in(L.d_out);
        a.out = static_cast<T *>(L.d_table);
        a.keys = keys;
        a.order = order;
        a.status = n > kRankMax ? status : nullptr;
        a.tokens = L.tokens;
        a.wide = L.token_bytes == 8;
        a.partials = reinterpret_cast<float *>(L.ws + plan.partials);
        a.counters = counters;
        a.d_stride = L.d_stride;
        a.out_stride = L.table_stride;
        a.scale = L.scale;
        a.accumulate = L.accumulate;
        a.n = n;
        a.vocab = vocab;
        a.width = static_cast<uint32_t>(L.width);
        a.log_lanes = plan.log_lanes;
        a.slabs = plan.slabs;
        a.per = plan.per;
        a.chunks = plan.chunks;
        auto start = [&](auto m) {
            constexpr int MODE = decltype(m)::value;
            if (a.chunks == 0) return static_cast<int>(GSORT_OK);
            k_embed_sum<T, MODE><<<a.chunks * a.slabs, kEmbedThreads, 0, L.stream>>>(a);
            if (cudaGetLastError() != cudaSuccess) return static_cast<int>(GSORT_ECUDA);
            return start_fill(filled, fill_ctas);
        };
        if (L.width % N == 0 && aligned(L.d_out, 16) && aligned(L.d_table, 16) && L.d_stride % N == 0 && L.table_stride % N == 0) {
            a.vectors = a.width / N;
            return start(integral_constant<int, kAligned>{});
        }
        a.vectors = plan.vectors_max;
        if constexpr (sizeof(T) == 4) {
            return start(integral_constant<int, kSingle>{});
        } else {
            if (L.width * sizeof(T) >= 64) return start(integral_constant<int, kShifted>{});
            return start(integral_constant<int, kElements>{});
        }
    });
}

}  // namespace gsort
