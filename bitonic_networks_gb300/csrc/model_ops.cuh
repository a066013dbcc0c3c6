// Shared pieces of the language-model operators (expert routing, grouping,
// row movement, token log probabilities, embedding, adjusted logits, gradient
// norm): element types, 16-byte vectors,
// order keys and the launch descriptions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gsort_internal.cuh"

namespace gsort {

inline int float_bytes(int dtype) {
    return dtype == GSORT_F32 ? 4 : (dtype == GSORT_BF16 || dtype == GSORT_F16) ? 2 : 0;
}

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eRest = static_cast<float>(1.4426950408889634 - kLog2e);
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// Round to nearest even, once, where a result leaves the 32-bit arithmetic.
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// N elements that move as one aligned access.
template <typename T, int N> struct alignas(sizeof(T) * N) Vec {
    T e[N];
};
// Two 32-bit numbers that move through one packed instruction.
union Pair {
    uint64_t u;
    float2 f;
};

__device__ __forceinline__ Pair pair(float x, float y) {
    Pair p;
    p.f = make_float2(x, y);
    return p;
}

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

// 16-byte vectors as pairs of 32-bit numbers and back, two elements at a time.
template <typename T> struct Wide;

template <> struct Wide<float> {
    static constexpr int kCount = 4;
    static constexpr uint32_t kNegInfWord = 0xFF800000u;
    static __device__ __forceinline__ float element(const uint4 &q, int i) { return __uint_as_float((&q.x)[i]); }
    static __device__ __forceinline__ Pair pair_of(const uint4 &q, int i) {
        const uint32_t *w = &q.x;
        return pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
    static __device__ __forceinline__ void set_pair(uint4 &q, int i, Pair p) {
        uint32_t *w = &q.x;
        w[2 * i] = __float_as_uint(p.f.x);
        w[2 * i + 1] = __float_as_uint(p.f.y);
    }
};

template <> struct Wide<__nv_bfloat16> {
    static constexpr int kCount = 8;
    static constexpr uint32_t kNegInfWord = 0xFF80FF80u;
    static __device__ __forceinline__ __nv_bfloat16 element(const uint4 &q, int i) {
        return __ushort_as_bfloat16(static_cast<unsigned short>((&q.x)[i / 2] >> (16 * (i % 2))));
    }
    static __device__ __forceinline__ Pair pair_of(const uint4 &q, int i) {
        const uint32_t w = (&q.x)[i];
        return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ void set_pair(uint4 &q, int i, Pair p) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(p.f.x, p.f.y);
        (&q.x)[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
};

template <> struct Wide<__half> {
    static constexpr int kCount = 8;
    static constexpr uint32_t kNegInfWord = 0xFC00FC00u;
    static __device__ __forceinline__ __half element(const uint4 &q, int i) {
        return __ushort_as_half(static_cast<unsigned short>((&q.x)[i / 2] >> (16 * (i % 2))));
    }
    static __device__ __forceinline__ Pair pair_of(const uint4 &q, int i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&q.x + i));
        return pair(f.x, f.y);
    }
    static __device__ __forceinline__ void set_pair(uint4 &q, int i, Pair p) {
        const __half2 v = __floats2half2_rn(p.f.x, p.f.y);
        (&q.x)[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
};

// Order key of a float: greater floats have greater keys; both zeros have one
// key.  0 is below the key of every number and stands for "no candidate".
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float order_key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float exp2_approx(float x) {   // 2^x, ex2.approx: 2 ulp
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Maximum that keeps a NaN operand.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// e^d for d <= 0 where results stay in 32 bits.  2^(d log2(e)) with the product
// rounded would be off by |d| 2^-23 of itself (3 bits at d = -30); what the
// product lost is put back: e^d = 2^y (1 + r ln2), y + r = d log2(e).  Within 2
// ulp and 2^-24.  d is bounded where e^d is 0, so that r and y are numbers.
__device__ __forceinline__ Pair exp_exact2(Pair d, Pair &y) {
    constexpr float kZero = -178.0f;
    d = pair(max_nan(d.f.x, kZero), max_nan(d.f.y, kZero));
    y = mul2(d, pair(kLog2e, kLog2e));
    Pair r = fma2(d, pair(kLog2e, kLog2e), pair(-y.f.x, -y.f.y));
    r = fma2(d, pair(kLog2eRest, kLog2eRest), r);
    const Pair e = pair(exp2_approx(y.f.x), exp2_approx(y.f.y));
    return fma2(mul2(e, pair(kLn2, kLn2)), r, e);
}

__device__ __forceinline__ float exp_exact(float d) {     // the same for one number, NaN apart
    d = fmaxf(d, -178.0f);
    const float y = d * kLog2e, r = fmaf(d, kLog2eRest, fmaf(d, kLog2e, -y)), e = exp2_approx(y);
    return fmaf(e * kLn2, r, e);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

// The waits of a call's kernels for their bulk copies: polls of one, and (testing) the CTA whose
// waits run out at once.  Where a call sorts: polls of a look-back, and the tile that publishes nothing.
struct Waits {
    uint32_t polls = kDefaultSpinLimit, stall = kNoStall;
    __device__ __forceinline__ uint32_t of_cta() const { return blockIdx.x == stall ? 0 : polls; }
};

// --------------------------------------------------------- launch plans
struct RouteLaunch {
    const void *logits;
    int dtype;
    int64_t tokens, row_stride;
    int experts;
    const float *bias;     // null: none
    int score, groups, groups_kept, group_score, chosen;
    bool renormalise;
    float scale;
    float *weights;
    int32_t *experts_out;
    cudaStream_t stream;
};
int launch_route(const RouteLaunch &L);

struct RouteBackwardLaunch {
    const float *grad_weights;
    const void *logits;
    int dtype;
    int64_t tokens, row_stride;
    int experts;
    const int32_t *experts_in;
    int chosen, score;
    bool renormalise;
    float scale;
    void *grad_logits;     // [tokens][experts], contiguous
    cudaStream_t stream;
};
int launch_route_backward(const RouteBackwardLaunch &L);

struct GroupLaunch {
    const int32_t *experts_in;
    uint32_t pairs;
    int experts;
    uint32_t align;
    int32_t *offsets, *counts, *rows, *positions;
    uint32_t capacity;
    uint32_t *ws;          // u32[tiles][experts]
    cudaStream_t stream;
};
size_t group_workspace_bytes(uint32_t pairs, int experts);
int launch_group(const GroupLaunch &L);

struct RowsLaunch {
    int dtype;
    int64_t tokens, width;
    int chosen;
    int64_t capacity;
    const int32_t *positions;   // [tokens][chosen]
    const int32_t *rows;        // [capacity]; null where no row is written whole
    const float *weights;       // null: ones
    const void *by_token;       // [tokens][width], row stride token_stride
    int64_t token_stride;
    const void *by_row;         // [capacity][width], row stride row_stride
    int64_t row_stride;
    void *out;                  // contiguous
    float *grad_weights;
    cudaStream_t stream;
    int sm_count;
};
int launch_dispatch(const RowsLaunch &L);
int launch_combine(const RowsLaunch &L);
int launch_combine_backward(const RowsLaunch &L);

struct LogprobsLaunch {
    const void *logits;
    int dtype;
    int64_t rows, vocab, row_stride;
    const void *targets;     // null: none
    int target_bytes;        // 4 or 8
    int top;
    float *logprobs, *entropy, *stats;   // stats: [rows][2], maximum and sum
    float *top_logprobs;
    int32_t *top_ids;
    cudaStream_t stream;
    int sm_count;
};
int launch_logprobs(const LogprobsLaunch &L);

struct LogprobsBackwardLaunch {
    const float *grad_logprobs, *grad_entropy;   // null: zero
    const void *logits;
    int dtype;
    int64_t rows, vocab, row_stride;
    const void *targets;
    int target_bytes;
    const float *entropy, *stats;
    void *grad_logits;
    int64_t grad_stride;
    cudaStream_t stream;
};
int launch_logprobs_backward(const LogprobsBackwardLaunch &L);

struct EmbedLaunch {
    const void *in;          // the table
    int dtype;
    int64_t vocab, width, in_stride;
    const void *tokens;
    int token_bytes;         // 4 or 8
    int64_t n;
    float scale;
    void *out;               // [n][width], contiguous
    cudaStream_t stream;
};
int launch_embed(const EmbedLaunch &L);

struct EmbedBackwardLaunch {
    const void *d_out;
    int dtype;
    int64_t n, width, d_stride;
    const void *tokens;
    int token_bytes;
    int64_t vocab;
    float scale;
    bool accumulate;
    void *d_table;
    int64_t table_stride;
    unsigned char *ws;
    Waits waits;             // of the sort
    cudaStream_t stream;
    int sm_count;
};
size_t embed_workspace_bytes(int64_t tokens, int64_t vocab, int64_t width, int dtype);
int launch_embed_backward(const EmbedBackwardLaunch &L);

struct AdjustLaunch {
    bool backward;
    const void *logits;      // read by the gradient, where a history is given
    const void *in;
    void *out;
    int dtype;
    int64_t rows, vocab, logits_stride, in_stride, out_stride;
    const void *history;     // null: none
    int64_t history_stride, length;
    int history_bytes;
    const int32_t *prompt;   // each null: none
    const float *repetition, *presence, *frequency;
    const void *bias_tokens;
    const float *bias;
    int64_t bias_stride, biases;
    int bias_bytes;
    const uint32_t *allowed; // null: none
    int64_t allowed_stride;
    Waits waits;
    cudaStream_t stream;
};
int launch_adjust(const AdjustLaunch &L);

struct NormLaunch {
    const void *const *in;
    void *const *out;        // null: the norm alone
    const int64_t *sizes;
    const int *dtypes;
    int64_t tensors;
    float scale, max_norm;
    float *norm;
    unsigned char *ws;
    Waits waits;
    cudaStream_t stream;
};
size_t norm_workspace_bytes(int64_t tensors);
int launch_norm(const NormLaunch &L);

// Calls f with a value of the element type that `dtype` names.
template <typename F> int with_float_type(int dtype, F &&f) {
    switch (dtype) {
        case GSORT_F32: return f(float{});
        case GSORT_BF16: return f(__nv_bfloat16{});
        default: return f(__half{});
    }
}

}  // namespace gsort
