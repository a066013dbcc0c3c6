// rows.cu -- rows to the experts and back, over the grouped layout.
//
//   dispatch          out[positions[t][j]] = x[t]; rows that no pair holds: 0
//   combine           out[t] = sum_j w[t][j] * y[positions[t][j]]
//   combine backward  dy[positions[t][j]] = w[t][j] * dout[t]; rows that no
//                     pair holds: 0;  dw[t][j] = <dout[t], y[positions[t][j]]>
// (dispatch's gradient is combine with w = 1.)  A position outside the layout
// takes no part.
//
// Every kernel walks the tokens, not the grouped rows: a token's row is read
// once and written to (or summed from) its k places, so the traffic is the
// algorithm's own.  Sums run over j in order, in 32 bits, rounded once.
#include <algorithm>

#include "model_ops.cuh"

namespace gsort {
namespace {

constexpr int kRowThreads = 256;
constexpr int kDotThreads = 128;

template <typename T> struct RowArgs {
    const T *by_token;
    const T *by_row;
    T *out;
    const int32_t *positions;
    const int32_t *rows;
    const float *weights;
    float *grad_weights;
    int64_t tokens, token_stride, row_stride, out_stride;
    uint32_t chosen, capacity, vectors;   // vectors per row
    uint32_t row_blocks;                  // CTAs that move rows; the rest fill with zeros
};

template <typename T, int N> __device__ __forceinline__ Vec<T, N> load_vec(const T *row, uint32_t v) {
    return reinterpret_cast<const Vec<T, N> *>(row)[v];
}

// Zeros the rows that no pair holds: a warp looks over 32 rows at a time.
template <typename T, int N>
__device__ __forceinline__ void fill_rows(const RowArgs<T> &a, uint32_t block) {
    Vec<T, N> zero;
#pragma unroll
    for (int i = 0; i < N; ++i) zero.e[i] = from_f32<T>(0.0f);
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t first = (block * (blockDim.x >> 5) + (threadIdx.x >> 5)) * 32;
    const uint32_t r = first + lane;
    uint32_t empty = __ballot_sync(kFullMask, r < a.capacity && a.rows[r] < 0);
    while (empty) {
        const uint32_t b = __ffs(empty) - 1;
        empty &= empty - 1;
        Vec<T, N> *o = reinterpret_cast<Vec<T, N> *>(a.out + static_cast<int64_t>(first + b) * a.out_stride);
        for (uint32_t v = lane; v < a.vectors; v += 32) o[v] = zero;
    }
}

template <typename T, int N>
__global__ void __launch_bounds__(kRowThreads) k_dispatch(const RowArgs<T> a) {
    if (blockIdx.x >= a.row_blocks) {
        fill_rows<T, N>(a, blockIdx.x - a.row_blocks);
        return;
    }
    const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
    const uint64_t t = i / a.vectors;
    const uint32_t v = static_cast<uint32_t>(i - t * a.vectors);
    if (t >= static_cast<uint64_t>(a.tokens)) return;
    const Vec<T, N> x = load_vec<T, N>(a.by_token + t * a.token_stride, v);
    const int32_t *pos = a.positions + t * a.chosen;
    for (uint32_t j = 0; j < a.chosen; ++j) {
        const uint32_t p = static_cast<uint32_t>(pos[j]);
        if (p < a.capacity) reinterpret_cast<Vec<T, N> *>(a.out + p * a.out_stride)[v] = x;
    }
}

template <typename T, int N>
__global__ void __launch_bounds__(kRowThreads) k_combine(const RowArgs<T> a) {
    const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
    const uint64_t t = i / a.vectors;
    const uint32_t v = static_cast<uint32_t>(i - t * a.vectors);
    if (t >= static_cast<uint64_t>(a.tokens)) return;
    const int32_t *pos = a.positions + t * a.chosen;
    const float *w = a.weights ? a.weights + t * a.chosen : nullptr;
    float acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
#pragma unroll 8
    for (uint32_t j = 0; j < a.chosen; ++j) {
        const uint32_t p = static_cast<uint32_t>(pos[j]);
        if (p < a.capacity) {
            const Vec<T, N> y = load_vec<T, N>(a.by_row + p * a.row_stride, v);
            const float wj = w ? w[j] : 1.0f;
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] = fmaf(wj, to_f32(y.e[e]), acc[e]);
        }
    }
    Vec<T, N> o;
#pragma unroll
    for (int e = 0; e < N; ++e) o.e[e] = from_f32<T>(acc[e]);
    reinterpret_cast<Vec<T, N> *>(a.out + t * a.out_stride)[v] = o;
}

// One CTA per token: dy rows are written and the dot products are summed over
// the CTA in a fixed order.
template <typename T, int N>
__global__ void __launch_bounds__(kDotThreads) k_combine_backward(const RowArgs<T> a) {
    if (blockIdx.x >= a.row_blocks) {
        fill_rows<T, N>(a, blockIdx.x - a.row_blocks);
        return;
    }
    __shared__ float s_dot[kDotThreads / 32];
    const int64_t t = blockIdx.x;
    const T *d_row = a.by_token + t * a.token_stride;
    for (uint32_t j = 0; j < a.chosen; ++j) {
        const uint32_t p = static_cast<uint32_t>(a.positions[t * a.chosen + j]);
        float dot = 0.0f;
        if (p < a.capacity) {
            const float w = a.weights[t * a.chosen + j];
            const T *y_row = a.by_row + p * a.row_stride;
            Vec<T, N> *o = reinterpret_cast<Vec<T, N> *>(a.out + p * a.out_stride);
            for (uint32_t v = threadIdx.x; v < a.vectors; v += kDotThreads) {
                const Vec<T, N> d = load_vec<T, N>(d_row, v), y = load_vec<T, N>(y_row, v);
                Vec<T, N> g;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float x = to_f32(d.e[e]);
                    dot = fmaf(x, to_f32(y.e[e]), dot);
                    g.e[e] = from_f32<T>(w * x);
                }
                o[v] = g;
            }
        }
        dot = warp_sum(dot);
        if ((threadIdx.x & 31) == 0) s_dot[threadIdx.x >> 5] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kDotThreads / 32; ++i) sum += s_dot[i];
            a.grad_weights[t * a.chosen + j] = sum;
        }
        __syncthreads();
    }
}

template <typename T> RowArgs<T> row_args(const RowsLaunch &L) {
    RowArgs<T> a{};
    a.by_token = static_cast<const T *>(L.by_token);
    a.by_row = static_cast<const T *>(L.by_row);
    a.out = static_cast<T *>(L.out);
    a.positions = L.positions;
    a.rows = L.rows;
    a.weights = L.weights;
    a.grad_weights = L.grad_weights;
    a.tokens = L.tokens;
    a.token_stride = L.token_stride;
    a.row_stride = L.row_stride;
    a.out_stride = L.width;
    a.chosen = L.chosen;
    a.capacity = static_cast<uint32_t>(L.capacity);
    return a;
}

// Elements that every row of every array can move at once: 16 bytes' worth
// where the bases, the strides and the width allow it, else less, down to one.
template <typename T> int vector_of(const RowsLaunch &L) {
    for (int n = 16 / sizeof(T); n > 1; n /= 2) {
        const size_t bytes = n * sizeof(T);
        auto fits = [&](const void *p, int64_t stride) {
            return p == nullptr || (aligned(p, bytes) && stride % n == 0);
        };
        if (L.width % n == 0 && fits(L.by_token, L.token_stride) && fits(L.by_row, L.row_stride) && fits(L.out, L.width))
            return n;
    }
    return 1;
}

template <typename F> int with_vector(const RowsLaunch &L, F &&f) {
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        switch (vector_of<T>(L)) {
            case 8: return f(t, std::integral_constant<int, 16 / sizeof(T)>{});
            case 4: return f(t, std::integral_constant<int, 4>{});
            case 2: return f(t, std::integral_constant<int, 2>{});
            default: return f(t, std::integral_constant<int, 1>{});
        }
    });
}

// CTAs that look for rows to zero, one row per thread.
uint32_t zero_blocks(const RowsLaunch &L, int threads) {
    return static_cast<uint32_t>((L.capacity + threads - 1) / threads);
}

int status() { return cudaGetLastError() == cudaSuccess ? GSORT_OK : GSORT_ECUDA; }

}  // namespace

int launch_dispatch(const RowsLaunch &L) {
    return with_vector(L, [&](auto t, auto n) {
        using T = decltype(t);
        constexpr int N = decltype(n)::value;
        RowArgs<T> a = row_args<T>(L);
        a.vectors = static_cast<uint32_t>(L.width / N);
        const int64_t blocks = (L.tokens * a.vectors + kRowThreads - 1) / kRowThreads;
        if (blocks + zero_blocks(L, kRowThreads) > 0x7FFFFFFF) return static_cast<int>(GSORT_ETOOBIG);
        a.row_blocks = static_cast<uint32_t>(blocks);
        k_dispatch<T, N><<<a.row_blocks + zero_blocks(L, kRowThreads), kRowThreads, 0, L.stream>>>(a);
        return status();
    });
}

int launch_combine(const RowsLaunch &L) {
    return with_vector(L, [&](auto t, auto n) {
        using T = decltype(t);
        constexpr int N = decltype(n)::value;
        RowArgs<T> a = row_args<T>(L);
        a.vectors = static_cast<uint32_t>(L.width / N);
        const int64_t blocks = (L.tokens * a.vectors + kRowThreads - 1) / kRowThreads;
        if (blocks > 0x7FFFFFFF) return static_cast<int>(GSORT_ETOOBIG);
        a.row_blocks = static_cast<uint32_t>(blocks);
        k_combine<T, N><<<a.row_blocks, kRowThreads, 0, L.stream>>>(a);
        return status();
    });
}

int launch_combine_backward(const RowsLaunch &L) {
    return with_vector(L, [&](auto t, auto n) {
        using T = decltype(t);
        constexpr int N = decltype(n)::value;
        RowArgs<T> a = row_args<T>(L);
        a.vectors = static_cast<uint32_t>(L.width / N);
        if (L.tokens + zero_blocks(L, kDotThreads) > 0x7FFFFFFF) return static_cast<int>(GSORT_ETOOBIG);
        a.row_blocks = static_cast<uint32_t>(L.tokens);
        k_combine_backward<T, N><<<a.row_blocks + zero_blocks(L, kDotThreads), kDotThreads, 0, L.stream>>>(a);
        return status();
    });
}

}  // namespace gsort
