// norm.cu -- the Euclidean norm of many tensors together, and clipping by it.
//
//   norm   = |scale| * sqrt(sum over all tensors of g^2)
//   out    = g * scale * min(1, max_norm / norm)
//
// The tensors' addresses and sizes travel as a kernel parameter (up to 1000 of
// them in a launch), so that a call needs no copy to the device and can be captured
// in a graph.  Tensors are cut into chunks, and a fixed number of CTAs takes them in turn;
// squares are summed in 32 bits within a thread's part of a chunk and in 64 bits
// from there on, each CTA's sum to a slot of its own: the order is given by the sizes.
// A part whose squares leave the 32-bit range is summed again in 64 bits.
//
// The memory bounds both steps.  Clipping reads everything twice, as the norm has to be
// known before the first product; it walks the chunks backwards, so that what the first
// step read last comes from the caches.
#include <algorithm>
#include <cmath>

#include "model_ops.cuh"

namespace gsort {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormVectors = 4;                   // 16-byte vectors in flight per thread
constexpr int kFewTensors = 32, kManyTensors = 1000;
constexpr uint32_t kMaxSlots = 1216;              // CTAs of a launch: 8 to an SM of a GB300
constexpr uint32_t kMaxChunk = 65536, kMinChunk = 4096;     // bytes
constexpr uint64_t kSizeMask = (1ull << 56) - 1;
// below it a thread's sum of squares may have lost what is under the 32-bit range
constexpr float kTinySum = 1.2621774483536189e-29f;         // 2^-96

template <int M> struct TensorTable {
    const void *in[M];
    void *out[M];
    uint64_t size[M];        // elements; the type in the top byte
    uint32_t first[M + 1];   // chunks before the tensor
    uint32_t tensors, chunk_bytes;
};

// The tensor that a chunk belongs to.
template <int M> __device__ __forceinline__ uint32_t tensor_of(const TensorTable<M> &t, uint32_t chunk) {
    uint32_t low = 0, high = t.tensors - 1;       // first[low] <= chunk
    while (low < high) {
        const uint32_t mid = (low + high + 1) / 2;
        if (t.first[mid] <= chunk) low = mid;
        else high = mid - 1;
    }
    return low;
}

// A chunk of a tensor: `vectors` 16-byte vectors from element `begin` on, which lies
// at a boundary; it may begin before the tensor and end behind it.
template <typename T> struct Chunk {
    const T *p;
    int64_t begin, size;
    uint32_t vectors;

    __device__ __forceinline__ bool whole(int64_t e) const { return e >= 0 && e + Wide<T>::kCount <= size; }
};

template <typename T, int M> __device__ __forceinline__ Chunk<T> chunk_of(const TensorTable<M> &t, uint32_t tensor, uint32_t chunk) {
    constexpr int N = Wide<T>::kCount;
    Chunk<T> c;
    c.p = static_cast<const T *>(t.in[tensor]);
    c.size = static_cast<int64_t>(t.size[tensor] & kSizeMask);
    c.vectors = t.chunk_bytes / 16;
    c.begin = static_cast<int64_t>(chunk - t.first[tensor]) * c.vectors * N - static_cast<int64_t>((reinterpret_cast<uintptr_t>(c.p) & 15) / sizeof(T));
    const int64_t left = (c.size - c.begin + N - 1) / N;
    if (left < c.vectors) c.vectors = static_cast<uint32_t>(left);
    return c;
}

// The elements of a vector, zeros beside the tensor.
template <typename T> __device__ __forceinline__ uint4 vector_of(const Chunk<T> &c, int64_t e) {
    constexpr int N = Wide<T>::kCount;
    if (c.whole(e)) return *reinterpret_cast<const uint4 *>(c.p + e);
    uint4 q;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const int64_t k = e + 2 * i;
        Wide<T>::set_pair(q, i, pair(k >= 0 && k < c.size ? to_f32(c.p[k]) : 0.0f, k + 1 >= 0 && k + 1 < c.size ? to_f32(c.p[k + 1]) : 0.0f));
    }
    return q;
}

// This thread's part of a chunk.
template <typename T> __device__ __forceinline__ double square_sum(const Chunk<T> &c) {
    constexpr int N = Wide<T>::kCount;
    Pair sum[kNormVectors];
    uint32_t any = 0;
#pragma unroll
    for (int u = 0; u < kNormVectors; ++u) sum[u] = pair(0.0f, 0.0f);
    for (uint32_t v0 = threadIdx.x; v0 < c.vectors; v0 += kNormThreads * kNormVectors) {
        uint4 q[kNormVectors];
#pragma unroll
        for (int u = 0; u < kNormVectors; ++u) {
            const uint32_t v = v0 + u * kNormThreads;
            q[u] = v < c.vectors ? vector_of(c, c.begin + static_cast<int64_t>(v) * N) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kNormVectors; ++u) {
            any |= q[u].x | q[u].y | q[u].z | q[u].w;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const Pair x = Wide<T>::pair_of(q[u], i);
                sum[u] = fma2(x, x, sum[u]);
            }
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < kNormVectors; ++u) s += sum[u].f.x + sum[u].f.y;
    if (s >= kTinySum && s < -kNegInf) return s;
    if ((any & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) == 0) return 0.0;
    double d = 0.0;          // squares beyond the 32-bit range, infinities and NaN
    for (uint32_t v = threadIdx.x; v < c.vectors; v += kNormThreads) {
        const uint4 q = vector_of(c, c.begin + static_cast<int64_t>(v) * N);
        for (int i = 0; i < N; ++i) {
            const double x = to_f32(Wide<T>::element(q, i));
            d = fma(x, x, d);
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

template <int M>
__global__ void __launch_bounds__(kNormThreads) k_square_sums(const __grid_constant__ TensorTable<M> t, double *slots) {
    double d = 0.0;
    for (uint32_t chunk = blockIdx.x; chunk < t.first[t.tensors]; chunk += gridDim.x) {
        const uint32_t i = tensor_of(t, chunk);
        switch (t.size[i] >> 56) {
            case GSORT_F32: d += square_sum(chunk_of<float>(t, i, chunk)); break;
            case GSORT_BF16: d += square_sum(chunk_of<__nv_bfloat16>(t, i, chunk)); break;
            default: d += square_sum(chunk_of<__half>(t, i, chunk)); break;
        }
    }
    d = cta_sum(d);
    if (threadIdx.x == 0) slots[blockIdx.x] = d;
}

__device__ __forceinline__ double norm_of(const double *slots, uint32_t count, float scale) {
    double d = 0.0;
    for (uint32_t i = threadIdx.x; i < count; i += kNormThreads) d += slots[i];
    return fabs(static_cast<double>(scale)) * sqrt(cta_sum(d));
}

__global__ void __launch_bounds__(kNormThreads) k_norm(const double *slots, uint32_t count, float scale, float *out) {
    const double norm = norm_of(slots, count, scale);
    if (threadIdx.x == 0) *out = static_cast<float>(norm);
}

template <typename T, int M>
__device__ __forceinline__ void scale_chunk(const TensorTable<M> &t, uint32_t tensor, uint32_t chunk, float by) {
    constexpr int N = Wide<T>::kCount;
    const Chunk<T> c = chunk_of<T>(t, tensor, chunk);
    T *out = static_cast<T *>(t.out[tensor]);
    const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(c.p)) & 15) == 0;
    for (uint32_t v0 = threadIdx.x; v0 < c.vectors; v0 += kNormThreads * kNormVectors) {
        uint4 q[kNormVectors];
#pragma unroll
        for (int u = 0; u < kNormVectors; ++u) {
            const uint32_t v = v0 + u * kNormThreads;
            if (v < c.vectors) q[u] = vector_of(c, c.begin + static_cast<int64_t>(v) * N);
        }
#pragma unroll
        for (int u = 0; u < kNormVectors; ++u) {
            const uint32_t v = v0 + u * kNormThreads;
            if (v >= c.vectors) continue;
            const int64_t e = c.begin + static_cast<int64_t>(v) * N;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) Wide<T>::set_pair(q[u], i, mul2(Wide<T>::pair_of(q[u], i), pair(by, by)));
            if (same && c.whole(e)) {
                *reinterpret_cast<uint4 *>(out + e) = q[u];
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (e + i >= 0 && e + i < c.size) out[e + i] = Wide<T>::element(q[u], i);
            }
        }
    }
}

template <int M>
__global__ void __launch_bounds__(kNormThreads)
k_clip(const __grid_constant__ TensorTable<M> t, const double *slots, uint32_t count, float scale, float max_norm, float *norm_out) {
    const double norm = norm_of(slots, count, scale);
    if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
    // NaN stays: a gradient that is no number must not look like one
    const double part = norm > max_norm ? max_norm / norm : norm == norm ? 1.0 : norm;
    const float by = static_cast<float>(scale * part);
    const uint32_t chunks = t.first[t.tensors];
    for (uint32_t n = blockIdx.x; n < chunks; n += gridDim.x) {
        const uint32_t chunk = chunks - 1 - n, i = tensor_of(t, chunk);
        if (by == 1.0f && t.in[i] == t.out[i]) continue;      // as it is
        switch (t.size[i] >> 56) {
            case GSORT_F32: scale_chunk<float>(t, i, chunk, by); break;
            case GSORT_BF16: scale_chunk<__nv_bfloat16>(t, i, chunk, by); break;
            default: scale_chunk<__half>(t, i, chunk, by); break;
        }
    }
}

// The tensors from `at` on, as many as fit, and how many of the list they are.
template <int M> int64_t fill_table(const NormLaunch &L, int64_t at, TensorTable<M> &t) {
    int64_t end = at;
    uint64_t bytes = 0;
    t.tensors = 0;
    while (end < L.tensors && t.tensors < M) {
        if (L.sizes[end] > 0) {
            t.in[t.tensors] = L.in[end];
            t.out[t.tensors] = L.out ? L.out[end] : nullptr;
            t.size[t.tensors++] = static_cast<uint64_t>(L.sizes[end]) | static_cast<uint64_t>(L.dtypes[end]) << 56;
            bytes += static_cast<uint64_t>(L.sizes[end]) * float_bytes(L.dtypes[end]);
        }
        ++end;
    }
    // small totals are cut finer, to fill the device
    t.chunk_bytes = kMaxChunk;
    while (t.chunk_bytes > kMinChunk && bytes / t.chunk_bytes < kMaxSlots) t.chunk_bytes /= 2;
    uint64_t chunks = 0;
    for (uint32_t i = 0; i < t.tensors; ++i) {
        t.first[i] = static_cast<uint32_t>(chunks);
        const uint64_t size = float_bytes(static_cast<int>(t.size[i] >> 56));
        const uint64_t span = (reinterpret_cast<uintptr_t>(t.in[i]) & 15) + (t.size[i] & kSizeMask) * size;
        chunks += (span + t.chunk_bytes - 1) / t.chunk_bytes;
    }
    if (chunks > 0x7FFFFFFF) return -1;
    t.first[t.tensors] = static_cast<uint32_t>(chunks);
    return end - at;
}

template <int M> int launch_tables(const NormLaunch &L) {
    static_assert(sizeof(TensorTable<M>) + 64 <= 32764, "kernel parameters");
    double *slots = reinterpret_cast<double *>(L.ws);
    TensorTable<M> t;
    uint32_t used = 0;
    for (int64_t at = 0; at < L.tensors;) {
        const int64_t taken = fill_table(L, at, t);
        if (taken < 0) return GSORT_ETOOBIG;
        at += taken;
        if (t.tensors == 0) continue;
        const uint32_t ctas = std::min(t.first[t.tensors], kMaxSlots);
        k_square_sums<M><<<ctas, kNormThreads, 0, L.stream>>>(t, slots + used);
        if (cudaGetLastError() != cudaSuccess) return GSORT_ECUDA;
        used += ctas;
    }
    if (L.out == nullptr || used == 0) {
        k_norm<<<1, kNormThreads, 0, L.stream>>>(slots, used, L.scale, L.norm);
        return cudaGetLastError() == cudaSuccess ? GSORT_OK : GSORT_ECUDA;
    }
    float *norm = L.norm;
    for (int64_t at = 0; at < L.tensors;) {
        at += fill_table(L, at, t);
        if (t.tensors == 0) continue;
        k_clip<M><<<std::min(t.first[t.tensors], kMaxSlots), kNormThreads, 0, L.stream>>>(t, slots, used, L.scale, L.max_norm, norm);
        if (cudaGetLastError() != cudaSuccess) return GSORT_ECUDA;
        norm = nullptr;
    }
    return GSORT_OK;
}

}  // namespace

size_t norm_workspace_bytes(int64_t tensors) {
    return static_cast<size_t>((tensors + kManyTensors - 1) / kManyTensors) * kMaxSlots * sizeof(double);
}

int launch_norm(const NormLaunch &L) {
    return L.tensors <= kFewTensors ? launch_tables<kFewTensors>(L) : launch_tables<kManyTensors>(L);
}

}  // namespace gsort
