// Rows of elements that move in 16-byte vectors at any alignment, shared by the
// kernels that gather, scatter and sum rows.
//
// Where the width, a stride or a base is not a multiple of 16 bytes, rows start
// anywhere: a row that is written is cut at its own 16-byte boundaries (its first
// and last elements are written one by one), and a row that is read gives 16
// bytes at any element from the two aligned vectors around them.  Those may hold
// elements of the neighbouring rows, which are not used, but never bytes outside
// the array: at its ends elements are read one by one.
#pragma once

#include "model_ops.cuh"

namespace gsort {

constexpr int kRowThreads = 256;

// A row that is read.  inner: it is neither the first nor the last of its array,
// so that 64 bytes before and after it are the array's.
template <typename T> struct InRow {
    const T *row;
    bool inner;
};

// How rows move: every row starts and ends at 16 bytes; anywhere, in 16-byte
// vectors; anywhere, in single 32-bit elements that neighbouring threads hold
// side by side (for the sums of 32-bit rows: fewer instructions than shifting,
// 8191 x 6 rows of 1001: combine 39 us against 45, backward 81 against 84); or
// element by element, for rows of less than 64 bytes.
enum RowMode { kAligned, kShifted, kSingle, kElements };

// Where a thread's N elements of vector v of a row are: e, e + kStep, ...
// kSingle: a warp's threads are side by side, 32 apart.
template <int MODE> constexpr int kStep = MODE == kSingle ? 32 : 1;

template <typename T, int MODE> __device__ __forceinline__ int32_t element_of(uint32_t v, int32_t shift) {
    if (MODE == kSingle) return static_cast<int32_t>((v & ~31u) * Wide<T>::kCount + (v & 31u));
    return static_cast<int32_t>(v * Wide<T>::kCount) - shift;
}

// 16 bytes of a row from element e on, in two steps, so that several can be in
// flight: the loads, which do not branch, and the shift.  Elements outside the
// row have any value.
struct Loaded {
    uint4 q, r;
};

template <typename T> __device__ __forceinline__ uintptr_t address_of(const T *row, int32_t e) {
    return reinterpret_cast<uintptr_t>(row) + static_cast<int64_t>(e) * static_cast<int64_t>(sizeof(T));
}

template <typename T, int MODE>
__device__ __forceinline__ Loaded start_read(const InRow<T> &in, int32_t e, uint32_t width, const uint4 *safe) {
    Loaded x;
    if (MODE == kAligned) {
        x.q = *reinterpret_cast<const uint4 *>(in.row + e);
    } else if (MODE == kShifted) {
        const uint4 *p = in.inner ? reinterpret_cast<const uint4 *>(address_of(in.row, e) & ~static_cast<uintptr_t>(15)) : safe;
        x.q = p[0];
        x.r = p[1];
    } else if (MODE == kSingle) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(in.row) + e;
        const int32_t left = static_cast<int32_t>(width) - e;
        x.q = make_uint4(left > 0 ? w[0] : 0u, left > 32 ? w[32] : 0u, left > 64 ? w[64] : 0u, left > 96 ? w[96] : 0u);
    }
    return x;
}

template <typename T, int MODE>
__device__ __forceinline__ uint4 end_read(const Loaded &x, const InRow<T> &in, int32_t e, uint32_t width) {
    constexpr int N = Wide<T>::kCount;
    if (MODE == kAligned || MODE == kSingle) return x.q;
    uint4 q;
    if (MODE == kShifted) {
        const uint32_t at = static_cast<uint32_t>(address_of(in.row, e));
        uint32_t w[5] = {x.q.x, x.q.y, x.q.z, x.q.w, x.r.x};
        const bool two = at & 8, one = at & 4;
        w[0] = two ? x.q.z : x.q.x;
        w[1] = two ? x.q.w : x.q.y;
        w[2] = two ? x.r.x : x.q.z;
        w[3] = two ? x.r.y : x.q.w;
        w[4] = two ? x.r.z : x.r.x;
        const uint32_t after = two ? x.r.w : x.r.y;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = one ? w[i + 1] : w[i];
        w[4] = one ? after : w[4];
        if (sizeof(T) == 2) {
            const uint32_t bits = (at & 2) * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
        }
        q = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (MODE == kElements || !in.inner) {
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = static_cast<uint32_t>(e + i) < width ? to_f32(in.row[e + i]) : 0.0f;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) Wide<T>::set_pair(q, i, pair(f[2 * i], f[2 * i + 1]));
    }
    return q;
}

// A row that is written.
template <typename T, int MODE> struct OutRow {
    T *row;
    int32_t shift;           // elements between the boundary at or before the row and the row

    __device__ __forceinline__ explicit OutRow(T *r)
        : row(r), shift(MODE == kAligned ? 0 : static_cast<int32_t>((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(T))) {}
    __device__ __forceinline__ int32_t at(uint32_t v) const { return element_of<T, MODE>(v, shift); }
    // Whether the N elements from e on are all of the row.
    static __device__ __forceinline__ bool whole(int32_t e, uint32_t width) {
        return MODE == kAligned || (e >= 0 && e + (Wide<T>::kCount - 1) * kStep<MODE> < static_cast<int32_t>(width));
    }
    __device__ __forceinline__ void write(int32_t e, uint32_t width, const uint4 &q) const {
        constexpr int N = Wide<T>::kCount;
        if (MODE != kSingle && whole(e, width)) {
            *reinterpret_cast<uint4 *>(row + e) = q;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (static_cast<uint32_t>(e + i * kStep<MODE>) < width) row[e + i * kStep<MODE>] = Wide<T>::element(q, i);
        }
    }
};

// 32 bytes at a 16-byte boundary of an array of at least 64 bytes.
inline const uint4 *safe_in(const void *p) {
    return reinterpret_cast<const uint4 *>((reinterpret_cast<uintptr_t>(p) + 15) & ~static_cast<uintptr_t>(15));
}

// As many threads side by side as the row's vectors need at `per_thread` each,
// a power of two up to the CTA.
inline uint32_t lanes_for(uint32_t vectors, int per_thread) {
    uint32_t log_lanes = 0;
    while ((1 << log_lanes) < kRowThreads && (static_cast<uint64_t>(per_thread) << log_lanes) < vectors) ++log_lanes;
    return log_lanes;
}

inline int launch_status() { return cudaGetLastError() == cudaSuccess ? GSORT_OK : GSORT_ECUDA; }

}  // namespace gsort
