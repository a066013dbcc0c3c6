// norm.cu -- the Euclidean norm of many tensors together, and clipping by it.
//
//   norm   = |scale| * sqrt(sum over all tensors of g^2)
//   out    = g * scale * min(1, max_norm / norm)
//
// The tensors' addresses and sizes travel as a kernel parameter (up to 1000 of
// them in a launch), so that a call needs no copy to the device and can be captured
// in a graph.  What a tensor has between its first and last 16-byte boundary is cut into
// chunks, which resident CTAs take in turn, in steps of 16 KB: bulk copies bring the next
// two steps to shared memory while one is worked on, so that 4 CTAs keep up to 192 KB of an
// SM's loads under way.  The few elements before the first and behind the last boundary of
// each tensor are taken by a thread each, while the first copies run.
// A thread's squares of a step are summed in 32 bits, all else in 64; each CTA's sum goes
// to a slot of its own, so that the order is given by the sizes.  A step whose squares leave
// the 32-bit range is summed in 64 bits.
//
// The memory bounds both kernels.  Clipping reads everything twice, as the norm has to be
// known before the first product; it takes the chunks backwards, so that what was
// read last comes from the caches.  2^30 bf16 elements in 200 tensors: norm 312 us (6.9 TB/s),
// clipping 990 us in all (6.5 TB/s of three passes).  In place and not clipped nothing is written, but
// all is read twice: 615 us.
#include <algorithm>
#include <cmath>

#include "model_ops.cuh"

namespace gsort {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormVectors = 4;                   // vectors of a thread in a step
constexpr uint32_t kStep = kNormThreads * kNormVectors;     // vectors of a step
// Tensors of a launch.  A table of 1000 takes 28 KB, which cost 3 us more to launch than one of 32.
constexpr int kFewTensors = 32, kSomeTensors = 384, kManyTensors = 1000;
constexpr int kStages = 3;
constexpr uint32_t kNormCtas = 608;               // 4 to an SM of a GB300
constexpr uint32_t kWaitLimit = 1u << 20;         // polls of a copy's barrier before the CTA is left
constexpr uint64_t kSizeMask = (1ull << 56) - 1;
// below it a thread's sum of squares may have lost what is under the 32-bit range
constexpr float kTinySum = 1.2621774483536189e-29f;         // 2^-96
constexpr double kLeastNormal = 1.1754943508222875e-38;     // 2^-126
constexpr size_t kNormSmem = kStages * kStep * 16;

template <int M> struct TensorTable {
    const void *in[M];
    void *out[M];
    uint64_t size[M];        // elements; the type in the top byte
    uint32_t first[M + 1];   // chunks before the tensor
    uint32_t tensors;
    uint32_t steps;          // of a chunk
};

__host__ __device__ __forceinline__ uint32_t type_bytes(uint32_t type) { return type == GSORT_F32 ? 4 : 2; }

// How a tensor lies: bytes before its first 16-byte boundary, whole vectors from there on,
// bytes behind its last boundary.
struct Span {
    uint32_t type, head, tail;
    uint64_t vectors;
};

__host__ __device__ __forceinline__ Span span_of(const void *p, uint64_t word) {
    Span s;
    s.type = static_cast<uint32_t>(word >> 56);
    const uint64_t bytes = (word & kSizeMask) * type_bytes(s.type), before = -reinterpret_cast<uintptr_t>(p) & 15;
    s.head = static_cast<uint32_t>(before < bytes ? before : bytes);
    s.vectors = (bytes - s.head) / 16;
    s.tail = static_cast<uint32_t>(bytes - s.head - s.vectors * 16);
    return s;
}

// A step: `vectors` (0: the last one is behind) from a tensor's byte `begin` on.
struct Step {
    uint32_t tensor, type, vectors;
    int64_t begin;
};

constexpr uint32_t kAll = 0xFFFFFFFFu;

// The steps of a CTA, brought to shared memory in turn.
template <int M, bool BACKWARDS> struct Ring {
    const TensorTable<M> &t;
    uint4 (*data)[kStep];
    Step *steps;             // [kStages]
    uint64_t *full;          // [kStages], a barrier for each stage
    uint32_t chunk, step;    // of the next copy; thread 0

    __device__ __forceinline__ void start() {
        if (threadIdx.x == 0) {
            for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
            chunk = blockIdx.x;
            step = 0;
            for (int i = 0; i < kStages; ++i) copy(i);
        }
        __syncthreads();     // the barriers are there
    }
    // Thread 0: the next step.
    __device__ __forceinline__ Step next() {
        const uint32_t chunks = t.first[t.tensors];
        Step s{};
        while (s.vectors == 0 && chunk < chunks) {
            const uint32_t c = BACKWARDS ? chunks - 1 - chunk : chunk;
            uint32_t i = 0, high = t.tensors - 1;
            while (i < high) {
                const uint32_t mid = (i + high + 1) / 2;
                if (t.first[mid] <= c) i = mid;
                else high = mid - 1;
            }
            const Span span = span_of(t.in[i], t.size[i]);
            const uint64_t v = (static_cast<uint64_t>(c - t.first[i]) * t.steps + step) * kStep;
            if (v < span.vectors) {
                s.tensor = i;
                s.type = span.type;
                s.vectors = static_cast<uint32_t>(min(span.vectors - v, static_cast<uint64_t>(kStep)));
                s.begin = static_cast<int64_t>(span.head + v * 16);
            }
            if (++step == t.steps || v + kStep >= span.vectors) {
                step = 0;
                chunk += gridDim.x;
            }
        }
        return s;
    }
    // Thread 0: the next step's copy into a stage.
    __device__ __forceinline__ void copy(int stage) {
        const Step s = next();
        steps[stage] = s;
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(&full[stage], s.vectors * 16);
        if (s.vectors > 0) bulk_load(data[stage], static_cast<const char *>(t.in[s.tensor]) + s.begin, s.vectors * 16, &full[stage]);
    }
    // Calls f(step, vectors) for every step; the number of the first step whose copy did not come, or kAll.  All threads leave at the
    // same barrier: the end is read from the step, which was written before the last barrier, and a
    // wait that ran out for one thread counts for all.
    template <typename F> __device__ __forceinline__ uint32_t run(uint32_t polls, F &&f) {
        for (uint32_t k = 0;; ++k) {
            const int stage = k % kStages;
            const bool there = mbar_wait_bounded(&full[stage], (k / kStages) & 1, polls);
            if (steps[stage].vectors == 0) return kAll;
            if (there) f(steps[stage], data[stage]);
            if (__syncthreads_or(!there)) {        // leave once no copy can be under way any more
                for (uint32_t i = k; i < k + kStages; ++i) mbar_wait_bounded(&full[i % kStages], (i / kStages) & 1, kWaitLimit);
                return k;
            }
            if (threadIdx.x == 0) copy(stage);
        }
    }
    // After run has given up at step k: calls f(step) for it and all behind it.
    template <typename F> __device__ __forceinline__ void rest(uint32_t k, F &&f) {
        for (uint32_t i = k; i < k + kStages; ++i) f(steps[i % kStages]);
        for (;;) {
            __syncthreads();
            if (threadIdx.x == 0) steps[0] = next();
            __syncthreads();
            if (steps[0].vectors == 0) return;
            f(steps[0]);
        }
    }
};

template <int M, bool BACKWARDS> __device__ __forceinline__ Ring<M, BACKWARDS> make_ring(const TensorTable<M> &t) {
    extern __shared__ __align__(128) uint4 s_data[];
    __shared__ Step s_steps[kStages];
    __shared__ __align__(8) uint64_t s_full[kStages];
    return Ring<M, BACKWARDS>{t, reinterpret_cast<uint4 (*)[kStep]>(s_data), s_steps, s_full, 0, 0};
}

// Calls f(tensor, type, first element, elements) for the ends of tensors that this thread takes.
template <int M, typename F> __device__ __forceinline__ void for_ends(const TensorTable<M> &t, F &&f) {
    for (uint32_t i = blockIdx.x + gridDim.x * threadIdx.x; i < 2 * t.tensors; i += gridDim.x * kNormThreads) {
        const uint32_t tensor = i / 2;
        const Span s = span_of(t.in[tensor], t.size[tensor]);
        const uint32_t size = type_bytes(s.type);
        if (i % 2 == 0 && s.head > 0) f(tensor, s.type, static_cast<uint64_t>(0), s.head / size);
        if (i % 2 == 1 && s.tail > 0) f(tensor, s.type, (s.head + s.vectors * 16) / size, s.tail / size);
    }
}

// Calls f with a null pointer to the element type.
template <typename F> __device__ __forceinline__ void with_type(uint32_t type, F &&f) {
    switch (type) {
        case GSORT_F32: f(static_cast<float *>(nullptr)); break;
        case GSORT_BF16: f(static_cast<__nv_bfloat16 *>(nullptr)); break;
        default: f(static_cast<__half *>(nullptr)); break;
    }
}

// The sum of this thread's squares of a step.
template <typename T> __device__ __forceinline__ double square_sum(uint32_t vectors, const uint4 *data) {
    constexpr int N = Wide<T>::kCount;
    uint32_t any = 0;
    Pair sum[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll
    for (int u = 0; u < kNormVectors; ++u) {
        const uint32_t v = threadIdx.x + u * kNormThreads;
        const uint4 q = v < vectors ? data[v] : make_uint4(0, 0, 0, 0);
        any |= q.x | q.y | q.z | q.w;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const Pair y = Wide<T>::pair_of(q, i);
            sum[i % 2] = fma2(y, y, sum[i % 2]);
        }
    }
    const Pair both = add2(sum[0], sum[1]);
    const float total = both.f.x + both.f.y;
    if (total >= kTinySum && total < -kNegInf) return total;
    if ((any & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) == 0) return 0.0;
    double d = 0.0;          // squares beyond the 32-bit range, infinities and NaN
    for (uint32_t v = threadIdx.x; v < vectors; v += kNormThreads) {
        const uint4 q = data[v];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const double y = to_f32(Wide<T>::element(q, i));
            d = fma(y, y, d);
        }
    }
    return d;
}

// The CTA's sum, in every thread, in a fixed order.
__device__ __forceinline__ double cta_sum(double d) {
    __shared__ double s_sum[kNormThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(kFullMask, d, o);
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = d;
    __syncthreads();
    d = 0.0;
#pragma unroll
    for (int w = 0; w < kNormThreads / 32; ++w) d += s_sum[w];
    return d;
}

// A kernel may start while the one before it in the stream runs, up to its wait.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <int M>
__global__ void __launch_bounds__(kNormThreads, 4) k_square_sums(const __grid_constant__ TensorTable<M> t, double *slots, float *zero, const Waits waits) {
    let_next_start();
    Ring<M, false> ring = make_ring<M, false>(t);
    ring.start();
    double d = 0.0;
    for_ends(t, [&](uint32_t tensor, uint32_t type, uint64_t first, uint32_t count) {
        with_type(type, [&](auto *p) {
            using T = std::remove_pointer_t<decltype(p)>;
            for (uint32_t k = 0; k < count; ++k) {
                const double x = to_f32(static_cast<const T *>(t.in[tensor])[first + k]);
                d = fma(x, x, d);
            }
        });
    });
    const uint32_t lost = ring.run(waits.of_cta(), [&](const Step &s, const uint4 *data) {
        with_type(s.type, [&](auto *p) { d += square_sum<std::remove_pointer_t<decltype(p)>>(s.vectors, data); });
    });
    if (lost != kAll) d = __longlong_as_double(0x7FF8000000000000ll);      // a norm without all of its parts is none
    d = cta_sum(d);
    wait_for_last();         // so that who waits for this kernel has waited for those before it
    if (threadIdx.x == 0) slots[blockIdx.x] = d;
    if (zero != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *zero = 0.0f;
}

__device__ __forceinline__ double sum_of(const double *slots, uint32_t count) {
    double d = 0.0;
    for (uint32_t i = threadIdx.x; i < count; i += kNormThreads) d += slots[i];
    return cta_sum(d);
}

__device__ __forceinline__ double norm_of(double squares, float scale) { return fabs(static_cast<double>(scale)) * sqrt(squares); }

__global__ void __launch_bounds__(kNormThreads) k_norm(const double *slots, uint32_t count, float scale, float *out) {
    wait_for_last();
    const double squares = sum_of(slots, count);
    if (threadIdx.x == 0) *out = static_cast<float>(norm_of(squares, scale));
}

// What every element is multiplied by, one number after the other.  Where a norm is so far beyond its
// limit that the factor is no normal 32-bit number, rounding it would take its bits, or all of
// it: it is cut in two there, 2^-126 and a number that is not above 1.  The first product is exact, or
// below the normal range, where the second one is then too.
struct Factor {
    float first, by;

    __device__ __forceinline__ void set(double c) {
        const bool low = fabs(c) < kLeastNormal && c != 0.0;
        first = low ? static_cast<float>(kLeastNormal) : 1.0f;
        by = static_cast<float>(low ? c * (1.0 / kLeastNormal) : c);
    }
    __device__ __forceinline__ bool one() const { return first == 1.0f && by == 1.0f; }
    __device__ __forceinline__ float of(float x) const { return x * first * by; }
    __device__ __forceinline__ Pair of(Pair x) const { return mul2(mul2(x, pair(first, first)), pair(by, by)); }
};

template <typename T> __device__ __forceinline__ void scale_step(const Step &s, const uint4 *data, void *tensor, const Factor &c) {
    constexpr int N = Wide<T>::kCount;
    char *to = static_cast<char *>(tensor) + s.begin;
    if ((reinterpret_cast<uintptr_t>(to) & 15) != 0) {         // the output lies differently
        const T *from = reinterpret_cast<const T *>(data);
        for (uint32_t i = threadIdx.x; i < s.vectors * N; i += kNormThreads) reinterpret_cast<T *>(to)[i] = from_f32<T>(c.of(to_f32(from[i])));
        return;
    }
#pragma unroll
    for (int u = 0; u < kNormVectors; ++u) {
        const uint32_t v = threadIdx.x + u * kNormThreads;
        if (v >= s.vectors) break;
        uint4 q = data[v];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) Wide<T>::set_pair(q, i, c.of(Wide<T>::pair_of(q, i)));
        reinterpret_cast<uint4 *>(to)[v] = q;
    }
}

// The gradients of step k and behind did not come: results are no numbers, but for tensors that
// stay as they are (`same`: those that are their own output).
template <int M> __device__ __forceinline__ void void_rest(Ring<M, true> &ring, uint32_t k, bool same) {
    ring.rest(k, [&](const Step &s) {
        if (s.vectors == 0 || (same && ring.t.in[s.tensor] == ring.t.out[s.tensor])) return;
        uint16_t *to = reinterpret_cast<uint16_t *>(static_cast<char *>(ring.t.out[s.tensor]) + s.begin);
        for (uint32_t i = threadIdx.x; i < s.vectors * 8; i += kNormThreads) to[i] = 0x7FFF;
    });
}

// norm_out holds 0 before.  Its bits are only raised, so that the NaN of a CTA whose copies did not come
// stays: NaN is above all numbers, and a norm is not below 0.
template <int M>
__global__ void __launch_bounds__(kNormThreads, 4)
k_clip(const __grid_constant__ TensorTable<M> t, const double *slots, uint32_t count, float scale, float max_norm, float *norm_out,
       const Waits waits) {
    let_next_start();
    Ring<M, true> ring = make_ring<M, true>(t);
    ring.start();            // the gradients were there before the sums
    wait_for_last();
    __shared__ Factor s_factor;
    const double squares = sum_of(slots, count);
    uint32_t *const norm_bits = reinterpret_cast<uint32_t *>(norm_out);
    if (threadIdx.x == 0) {  // 64-bit operations are slow: 2^24 f32 elements in 300 tensors take 38.9 us so, 44.0 where every thread does them
        const double norm = norm_of(squares, scale);
        if (blockIdx.x == 0) atomicMax(norm_bits, __float_as_uint(static_cast<float>(norm)));
        // NaN stays: a gradient that is no number must not look like one
        const double part = norm > max_norm ? max_norm / norm : norm == norm ? 1.0 : norm;
        s_factor.set(scale * part);
    }
    __syncthreads();
    const Factor c = s_factor;
    auto changes = [&](uint32_t tensor) { return !c.one() || t.in[tensor] != t.out[tensor]; };     // else it is as it has to be
    for_ends(t, [&](uint32_t tensor, uint32_t type, uint64_t first, uint32_t n) {
        with_type(type, [&](auto *p) {
            using T = std::remove_pointer_t<decltype(p)>;
            for (uint32_t k = 0; changes(tensor) && k < n; ++k)
                static_cast<T *>(t.out[tensor])[first + k] = from_f32<T>(c.of(to_f32(static_cast<const T *>(t.in[tensor])[first + k])));
        });
    });
    const uint32_t lost = ring.run(waits.of_cta(), [&](const Step &s, const uint4 *data) {
        if (changes(s.tensor))
            with_type(s.type, [&](auto *p) { scale_step<std::remove_pointer_t<decltype(p)>>(s, data, t.out[s.tensor], c); });
    });
    if (lost == kAll) return;
    if (threadIdx.x == 0) atomicMax(norm_bits, 0x7FC00000u);
    void_rest(ring, lost, c.one());
}

// The tensors from `at` on, as many as fit, and how many of the list they are.
template <int M> int64_t fill_table(const NormLaunch &L, int64_t at, TensorTable<M> &t) {
    int64_t end = at;
    uint64_t bytes = 0;
    t.tensors = 0;
    for (; end < L.tensors && t.tensors < M; ++end) {
        if (L.sizes[end] == 0) continue;
        const uint32_t i = t.tensors++;
        t.in[i] = L.in[end];
        t.out[i] = L.out ? L.out[end] : nullptr;
        t.size[i] = static_cast<uint64_t>(L.sizes[end]) | static_cast<uint64_t>(L.dtypes[end]) << 56;
        bytes += static_cast<uint64_t>(L.sizes[end]) * float_bytes(L.dtypes[end]);
    }
    t.steps = bytes / (kStep * 16) >= 16 * kNormCtas ? 4 : 1;
    const uint64_t chunk_bytes = static_cast<uint64_t>(t.steps) * kStep * 16;
    uint64_t chunks = 0;
    for (uint32_t i = 0; i < t.tensors; ++i) {
        t.first[i] = static_cast<uint32_t>(chunks);
        chunks += (span_of(t.in[i], t.size[i]).vectors * 16 + chunk_bytes - 1) / chunk_bytes;
    }
    if (chunks > 0x7FFFFFFF) return -1;
    t.first[t.tensors] = static_cast<uint32_t>(chunks);
    return end - at;
}

// Ends alone have no chunks.
template <int M> uint32_t ctas_of(const TensorTable<M> &t) { return std::max(1u, std::min(t.first[t.tensors], kNormCtas)); }

template <typename K, typename... A> int launch(K kernel, uint32_t ctas, size_t smem, bool early, cudaStream_t stream, const A &...args) {
    if (smem > 0 && set_smem_limit(reinterpret_cast<const void *>(kernel), smem) != cudaSuccess) return GSORT_ECUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kNormThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? GSORT_OK : GSORT_ECUDA;
}

template <int M> int launch_tables(const NormLaunch &L) {
    static_assert(sizeof(TensorTable<M>) + 64 <= 32764, "kernel parameters");
    double *slots = reinterpret_cast<double *>(L.ws);
    TensorTable<M> t;
    uint32_t used = 0;
    int rc = GSORT_OK;
    int64_t at = 0;
    while (at < L.tensors) {
        const int64_t taken = fill_table(L, at, t);
        if (taken < 0) return GSORT_ETOOBIG;
        at += taken;
        if (t.tensors == 0) continue;
        const uint32_t ctas = ctas_of(t);
        rc = launch(k_square_sums<M>, ctas, kNormSmem, used > 0, L.stream, t, slots + used, L.out != nullptr && used == 0 ? L.norm : nullptr,
                    L.out == nullptr ? L.waits : Waits{});
        if (rc != GSORT_OK) return rc;
        used += ctas;
    }
    if (L.out == nullptr || used == 0)
        return launch(k_norm, 1, 0, used > 0, L.stream, static_cast<const double *>(slots), used, L.scale, L.norm);
    const bool one = L.tensors <= M;       // its table is still there
    for (at = 0; at < L.tensors;) {
        at += one ? L.tensors : fill_table(L, at, t);
        if (t.tensors == 0) continue;
        rc = launch(k_clip<M>, ctas_of(t), kNormSmem, true, L.stream, t, static_cast<const double *>(slots), used, L.scale,
                    L.max_norm, L.norm, L.waits);
        if (rc != GSORT_OK) return rc;
    }
    return GSORT_OK;
}

}  // namespace

size_t norm_workspace_bytes(int64_t tensors) {
    return static_cast<size_t>((tensors + kManyTensors - 1) / kManyTensors) * kNormCtas * sizeof(double);
}

int launch_norm(const NormLaunch &L) {
    if (L.tensors <= kFewTensors) return launch_tables<kFewTensors>(L);
    return L.tensors <= kSomeTensors ? launch_tables<kSomeTensors>(L) : launch_tables<kManyTensors>(L);
}

}  // namespace gsort
