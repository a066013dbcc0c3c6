// norm.cu -- the Euclidean norm of many tensors together, and clipping by it.
//
//   norm   = |scale| * sqrt(sum over all tensors of g^2)
//   out    = g * scale * min(1, max_norm / norm)
//
// The tensors' addresses and sizes travel as a kernel parameter (up to 1000 of
// them in a launch), so that a call needs no copy to the device and can be captured
// in a graph.  Tensors are cut into chunks of 16-byte vectors at 16-byte boundaries, and
// resident CTAs take them in turn, in steps of 16 KB of which the next one is loaded
// before the last is worked on.  A thread's squares of a step are summed in 32 bits, all else
// in 64; each CTA's sum goes to a slot of its own, so that the order is given by the
// sizes.  A step whose squares leave the 32-bit range is summed in 64 bits.
//
// The memory bounds both kernels.  Clipping reads everything twice, as the norm has to be
// known before the first product; it takes the chunks backwards, so that what was
// read last comes from the caches.
#include <algorithm>
#include <cmath>

#include "model_ops.cuh"

namespace gsort {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormVectors = 4;                   // vectors of a thread in a step
constexpr uint32_t kStep = kNormThreads * kNormVectors;     // vectors of a step
constexpr int kFewTensors = 32, kManyTensors = 1000;
constexpr uint32_t kNormCtas = 608;               // 4 to an SM of a GB300
constexpr uint64_t kSizeMask = (1ull << 56) - 1;
// below it a thread's sum of squares may have lost what is under the 32-bit range
constexpr float kTinySum = 1.2621774483536189e-29f;         // 2^-96

template <int M> struct TensorTable {
    const void *in[M];
    void *out[M];
    uint64_t size[M];        // elements; the type in the top byte
    uint32_t first[M + 1];   // chunks before the tensor
    uint32_t tensors;
    uint32_t steps;          // of a chunk
};

__host__ __device__ __forceinline__ int type_bytes(uint32_t type) { return type == GSORT_F32 ? 4 : 2; }

// A step: vectors [low, high) from `from` on are whole; the tensor's first and last
// vector may be cut by its start or end.
struct Step {
    const char *from;        // at a 16-byte boundary, at most 15 bytes before the tensor
    uint32_t tensor, type;
    uint32_t low, high, vectors;
    int64_t begin, size;     // bytes from the tensor's start to `from`, and of the tensor
};

// The steps of a CTA, one after another.
template <int M, bool BACKWARDS> struct Steps {
    const TensorTable<M> &t;
    uint32_t chunk, step;

    __device__ __forceinline__ explicit Steps(const TensorTable<M> &table) : t(table), chunk(blockIdx.x), step(0) {}

    __device__ __forceinline__ bool next(Step &s) {
        const uint32_t chunks = t.first[t.tensors];
        while (chunk < chunks) {
            const uint32_t c = BACKWARDS ? chunks - 1 - chunk : chunk;
            uint32_t i = 0, high = t.tensors - 1;
            while (i < high) {
                const uint32_t mid = (i + high + 1) / 2;
                if (t.first[mid] <= c) i = mid;
                else high = mid - 1;
            }
            const uint64_t word = t.size[i];
            s.tensor = i;
            s.type = static_cast<uint32_t>(word >> 56);
            s.size = static_cast<int64_t>(word & kSizeMask) * type_bytes(s.type);
            const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(t.in[i])) & 15;
            const int64_t v = (static_cast<int64_t>(c - t.first[i]) * t.steps + step) * kStep;
            const int64_t left = (s.size + shift + 15) / 16 - v;
            if (left > 0) {
                s.begin = v * 16 - shift;
                s.from = static_cast<const char *>(t.in[i]) + s.begin;
                s.vectors = static_cast<uint32_t>(min(left, static_cast<int64_t>(kStep)));
                s.low = s.begin < 0 ? 1 : 0;
                s.high = s.begin + static_cast<int64_t>(s.vectors) * 16 > s.size ? s.vectors - 1 : s.vectors;
                if (++step == t.steps) {
                    step = 0;
                    chunk += gridDim.x;
                }
                return true;
            }
            step = 0;
            chunk += gridDim.x;
        }
        return false;
    }
};

__device__ __forceinline__ void load_step(const Step &s, uint4 (&q)[kNormVectors]) {
#pragma unroll
    for (int u = 0; u < kNormVectors; ++u) {
        const uint32_t v = threadIdx.x + u * kNormThreads;
        q[u] = v >= s.low && v < s.high ? reinterpret_cast<const uint4 *>(s.from)[v] : make_uint4(0, 0, 0, 0);
    }
}

// The cut vector that this thread takes: threads 0 and 1 take the first and the last one.
__device__ __forceinline__ bool takes_cut(const Step &s, uint32_t &v) {
    v = threadIdx.x == 0 ? 0 : s.vectors - 1;
    return threadIdx.x == 0 ? s.low > 0 : threadIdx.x == 1 && s.high < s.vectors && (s.low == 0 || s.vectors > 1);
}

// The elements of a cut vector, zeros beside the tensor.
template <typename T> __device__ __forceinline__ uint4 cut_vector(const Step &s, uint32_t v) {
    constexpr int N = Wide<T>::kCount;
    const int64_t b = s.begin + static_cast<int64_t>(v) * 16;        // in bytes from the tensor's start
    const T *p = reinterpret_cast<const T *>(s.from) + v * N;
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t k = b + i * static_cast<int64_t>(sizeof(T));
        f[i] = k >= 0 && k < s.size ? to_f32(p[i]) : 0.0f;
    }
    uint4 q;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) Wide<T>::set_pair(q, i, pair(f[2 * i], f[2 * i + 1]));
    return q;
}

// The sum of this thread's squares of a step.
template <typename T> __device__ __forceinline__ double square_sum(const Step &s, const uint4 (&q)[kNormVectors]) {
    constexpr int N = Wide<T>::kCount;
    uint32_t cut, any = 0;
    uint4 edge = make_uint4(0, 0, 0, 0);
    if (takes_cut(s, cut)) edge = cut_vector<T>(s, cut);
    Pair sum[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
    auto add = [&](const uint4 &x) {
        any |= x.x | x.y | x.z | x.w;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const Pair y = Wide<T>::pair_of(x, i);
            sum[i % 2] = fma2(y, y, sum[i % 2]);
        }
    };
#pragma unroll
    for (int u = 0; u < kNormVectors; ++u) add(q[u]);
    add(edge);
    const Pair both = add2(sum[0], sum[1]);
    const float total = both.f.x + both.f.y;
    if (total >= kTinySum && total < -kNegInf) return total;
    if ((any & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) == 0) return 0.0;
    double d = 0.0;          // squares beyond the 32-bit range, infinities and NaN
    auto add_wide = [&](const uint4 &x) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const double y = to_f32(Wide<T>::element(x, i));
            d = fma(y, y, d);
        }
    };
#pragma unroll
    for (int u = 0; u < kNormVectors; ++u) add_wide(q[u]);
    add_wide(edge);
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
__global__ void __launch_bounds__(kNormThreads, 4) k_square_sums(const __grid_constant__ TensorTable<M> t, double *slots) {
    let_next_start();
    double d = 0.0;
    Steps<M, false> steps(t);
    Step now, then;
    uint4 q[kNormVectors];
    bool more = steps.next(now);
    if (more) load_step(now, q);
    while (more) {
        uint4 x[kNormVectors];
#pragma unroll
        for (int u = 0; u < kNormVectors; ++u) x[u] = q[u];
        more = steps.next(then);
        if (more) load_step(then, q);
        switch (now.type) {
            case GSORT_F32: d += square_sum<float>(now, x); break;
            case GSORT_BF16: d += square_sum<__nv_bfloat16>(now, x); break;
            default: d += square_sum<__half>(now, x); break;
        }
        now = then;
    }
    d = cta_sum(d);
    wait_for_last();         // so that who waits for this kernel has waited for those before it
    if (threadIdx.x == 0) slots[blockIdx.x] = d;
}

__device__ __forceinline__ double norm_of(const double *slots, uint32_t count, float scale) {
    double d = 0.0;
    for (uint32_t i = threadIdx.x; i < count; i += kNormThreads) d += slots[i];
    return fabs(static_cast<double>(scale)) * sqrt(cta_sum(d));
}

__global__ void __launch_bounds__(kNormThreads) k_norm(const double *slots, uint32_t count, float scale, float *out) {
    wait_for_last();
    const double norm = norm_of(slots, count, scale);
    if (threadIdx.x == 0) *out = static_cast<float>(norm);
}

template <typename T> __device__ __forceinline__ void scale_step(const Step &s, uint4 (&q)[kNormVectors], void *tensor, float by) {
    constexpr int N = Wide<T>::kCount;
    char *to = static_cast<char *>(tensor) + s.begin;
    const bool same = (reinterpret_cast<uintptr_t>(to) & 15) == 0;
    auto elements = [&](uint32_t v) {          // a vector's elements that are the tensor's, one by one
        const int64_t b = s.begin + static_cast<int64_t>(v) * 16;
        for (int i = 0; i < N; ++i) {
            const int64_t k = b + i * static_cast<int64_t>(sizeof(T));
            if (k >= 0 && k < s.size) reinterpret_cast<T *>(to)[v * N + i] = from_f32<T>(to_f32(reinterpret_cast<const T *>(s.from)[v * N + i]) * by);
        }
    };
    if (!same) {             // the output lies differently
        for (uint32_t v = threadIdx.x; v < s.vectors; v += kNormThreads) elements(v);
        return;
    }
#pragma unroll
    for (int u = 0; u < kNormVectors; ++u) {
        const uint32_t v = threadIdx.x + u * kNormThreads;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) Wide<T>::set_pair(q[u], i, mul2(Wide<T>::pair_of(q[u], i), pair(by, by)));
        if (v >= s.low && v < s.high) reinterpret_cast<uint4 *>(to)[v] = q[u];
    }
    uint32_t cut;
    if (takes_cut(s, cut)) elements(cut);
}

template <int M>
__global__ void __launch_bounds__(kNormThreads, 4)
k_clip(const __grid_constant__ TensorTable<M> t, const double *slots, uint32_t count, float scale, float max_norm, float *norm_out) {
    let_next_start();
    wait_for_last();
    const double norm = norm_of(slots, count, scale);
    if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
    // NaN stays: a gradient that is no number must not look like one
    const double part = norm > max_norm ? max_norm / norm : norm == norm ? 1.0 : norm;
    const float by = static_cast<float>(scale * part);
    Steps<M, true> steps(t);
    auto changes = [&](const Step &s) { return by != 1.0f || t.in[s.tensor] != t.out[s.tensor]; };     // else it is as it has to be
    Step now, then;
    uint4 q[kNormVectors];
    bool more = steps.next(now);
    if (more && changes(now)) load_step(now, q);
    while (more) {
        uint4 x[kNormVectors];
#pragma unroll
        for (int u = 0; u < kNormVectors; ++u) x[u] = q[u];
        more = steps.next(then);
        if (more && changes(then)) load_step(then, q);
        if (changes(now)) {
            void *out = t.out[now.tensor];
            switch (now.type) {
                case GSORT_F32: scale_step<float>(now, x, out, by); break;
                case GSORT_BF16: scale_step<__nv_bfloat16>(now, x, out, by); break;
                default: scale_step<__half>(now, x, out, by); break;
            }
        }
        now = then;
    }
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
        const uint64_t span = (reinterpret_cast<uintptr_t>(t.in[i]) & 15) + (t.size[i] & kSizeMask) * type_bytes(static_cast<uint32_t>(t.size[i] >> 56));
        chunks += (span + chunk_bytes - 1) / chunk_bytes;
    }
    if (chunks > 0x7FFFFFFF) return -1;
    t.first[t.tensors] = static_cast<uint32_t>(chunks);
    return end - at;
}

template <int M> uint32_t ctas_of(const TensorTable<M> &t) { return std::min(t.first[t.tensors], kNormCtas); }

template <typename K, typename... A> int launch(K kernel, uint32_t ctas, bool early, cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kNormThreads);
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
        if ((rc = launch(k_square_sums<M>, ctas, used > 0, L.stream, t, slots + used)) != GSORT_OK) return rc;
        used += ctas;
    }
    if (L.out == nullptr || used == 0)
        return launch(k_norm, 1, used > 0, L.stream, static_cast<const double *>(slots), used, L.scale, L.norm);
    float *norm = L.norm;
    const bool one = L.tensors <= M;       // its table is still there
    for (at = 0; at < L.tensors;) {
        at += one ? L.tensors : fill_table(L, at, t);
        if (t.tensors == 0) continue;
        rc = launch(k_clip<M>, ctas_of(t), true, L.stream, t, static_cast<const double *>(slots), used, L.scale,
                    L.max_norm, norm);
        if (rc != GSORT_OK) return rc;
        norm = nullptr;
    }
    return GSORT_OK;
}

}  // namespace

size_t norm_workspace_bytes(int64_t tensors) {
    return static_cast<size_t>((tensors + kManyTensors - 1) / kManyTensors) * kNormCtas * sizeof(double);
}

int launch_norm(const NormLaunch &L) {
    return L.tensors <= kFewTensors ? launch_tables<kFewTensors>(L) : launch_tables<kManyTensors>(L);
}

}  // namespace gsort
