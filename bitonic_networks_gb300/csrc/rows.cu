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
// algorithm's own, and the memory bounds it.  Sums run over j in order, in 32
// bits, rounded once.
//
// Rows move in 16-byte vectors at any alignment (row_access.cuh).
#include <algorithm>

#include "row_access.cuh"

namespace gsort {
namespace {

// CTAs per SM that a kernel's registers leave room for where 16-bit rows start
// anywhere: loads wait for memory, and more of them do with more CTAs (8191 x 6
// rows of 1001: combine 29 us with 4 CTAs of 2 x 2 loads per thread, 37 with 3
// of 4 x 1; backward 55 with 6 CTAs, 58 with 4; since then 26 and 49).  The
// combine spills 20 to 24 bytes under its bound.
constexpr int kShiftedCombine = 4, kShiftedBackward = 6;

template <typename T> struct RowArgs {
    const T *by_token;
    const T *by_row;
    const uint4 *token_safe, *row_safe;   // 32 bytes that can be read in place of others
    T *out;
    const int32_t *positions;
    const int32_t *rows;
    const float *weights;
    float *grad_weights;
    int64_t token_stride, row_stride;
    uint32_t tokens, chosen, capacity, width;
    uint32_t vectors;        // vectors that a written row touches, at most
    uint32_t log_lanes;      // 2^log_lanes threads side by side on a row
    uint32_t chunks;         // a row's pieces of lanes * U vectors
    uint32_t fill_blocks;    // CTAs that fill rows with zeros; the rest move rows
};

template <typename T> __device__ __forceinline__ InRow<T> token_row(const RowArgs<T> &a, uint32_t t) {
    return {a.by_token + static_cast<int64_t>(t) * a.token_stride, t > 0 && t + 1 < a.tokens};
}

template <typename T> __device__ __forceinline__ InRow<T> layout_row(const RowArgs<T> &a, uint32_t p) {
    return {a.by_row + static_cast<int64_t>(p) * a.row_stride, p > 0 && p + 1 < a.capacity};
}

// Zeros the rows that no pair holds: without a pair, or with one whose position
// was taken away since.  Warp w of W looks over rows w, w + W, ...:
// a run of such rows (the end of the layout) is shared among the warps.  These
// CTAs come first, so that it is under way while the others are moved (256
// experts padded to 16, 16384 x 8 rows of 8 KB: 185 us, and 220 when they came
// last with 32 rows in a row to a warp).
template <typename T, int MODE> __device__ __forceinline__ void fill_rows(const RowArgs<T> &a) {
    constexpr uint32_t kWarps = kRowThreads / 32;
    const uint32_t lane = threadIdx.x & 31, warps = a.fill_blocks * kWarps, pairs = a.tokens * a.chosen;
    for (uint32_t base = blockIdx.x * kWarps + (threadIdx.x >> 5); base < a.capacity; base += 32 * warps) {
        const uint32_t r = base + lane * warps;
        const uint32_t n = r < a.capacity ? static_cast<uint32_t>(a.rows[r]) : 0u;
        uint32_t empty = __ballot_sync(kFullMask, r < a.capacity && (n >= pairs || static_cast<uint32_t>(a.positions[n]) != r));
        for (; empty; empty &= empty - 1) {
            const OutRow<T, MODE> o(a.out + static_cast<int64_t>(base + (__ffs(empty) - 1) * warps) * a.width);
            for (uint32_t v = lane; v < a.vectors; v += 32) o.write(o.at(v), a.width, make_uint4(0, 0, 0, 0));
        }
    }
}

// The token and the first vector of this thread: 2^log_lanes threads walk a
// chunk of U vectors each of a token's row side by side.
struct RowPlace {
    uint32_t token, v;
};

template <int U, typename T> __device__ __forceinline__ RowPlace row_place(const RowArgs<T> &a) {
    const uint32_t lanes = 1u << a.log_lanes;
    const uint32_t block = blockIdx.x - a.fill_blocks, group = block / a.chunks, chunk = block % a.chunks;
    return {group * (kRowThreads >> a.log_lanes) + (threadIdx.x >> a.log_lanes), chunk * lanes * U + (threadIdx.x & (lanes - 1))};
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kRowThreads) k_dispatch(const RowArgs<T> a) {
    if (blockIdx.x < a.fill_blocks) {
        fill_rows<T, MODE>(a);
        return;
    }
    const RowPlace at = row_place<1>(a);
    if (at.token >= a.tokens || at.v >= a.vectors) return;
    const InRow<T> in = token_row(a, at.token);
    uint4 q;
    if (MODE == kAligned) q = start_read<T, MODE>(in, element_of<T, MODE>(at.v, 0), a.width, a.token_safe).q;
    const int32_t *pos = a.positions + static_cast<int64_t>(at.token) * a.chosen;
#pragma unroll 4
    for (uint32_t j = 0; j < a.chosen; ++j) {
        const uint32_t p = static_cast<uint32_t>(pos[j]);
        if (p >= a.capacity) continue;
        const OutRow<T, MODE> o(a.out + static_cast<int64_t>(p) * a.width);
        const int32_t to = o.at(at.v);
        // from L1: each row has its own boundaries
        if (MODE != kAligned) q = end_read<T, MODE>(start_read<T, MODE>(in, to, a.width, a.token_safe), in, to, a.width);
        o.write(to, a.width, q);
    }
}

// J slots' rows are loaded together, U vectors of each.
template <typename T, int MODE, int J, int U>
__global__ void __launch_bounds__(kRowThreads, MODE == kShifted ? kShiftedCombine : 1) k_combine(const RowArgs<T> a) {
    constexpr int N = Wide<T>::kCount;
    const RowPlace at = row_place<U>(a);
    if (at.token >= a.tokens) return;
    const uint32_t lanes = 1u << a.log_lanes;
    const int64_t pair0 = static_cast<int64_t>(at.token) * a.chosen;
    const OutRow<T, MODE> out(a.out + static_cast<int64_t>(at.token) * a.width);
    Pair acc[U][N / 2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < N / 2; ++i) acc[u][i] = pair(0.0f, 0.0f);
    for (uint32_t j0 = 0; j0 < a.chosen; j0 += J) {
        Loaded y[J][U];
        InRow<T> row[J];
        float w[J];
        bool there[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t p = j0 + j < a.chosen ? static_cast<uint32_t>(a.positions[pair0 + j0 + j]) : a.capacity;
            there[j] = p < a.capacity;
            w[j] = !there[j] ? 0.0f : a.weights ? a.weights[pair0 + j0 + j] : 1.0f;
            row[j] = layout_row(a, there[j] ? p : 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t v = min(at.v + u * lanes, a.vectors - 1);     // no branch around the loads
                y[j][u] = start_read<T, MODE>(row[j], out.at(v), a.width, a.row_safe);
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t v = at.v + u * lanes;
                if (!there[j] || v >= a.vectors) continue;
                const uint4 q = end_read<T, MODE>(y[j][u], row[j], out.at(v), a.width);
#pragma unroll
                for (int i = 0; i < N / 2; ++i) acc[u][i] = fma2(pair(w[j], w[j]), Wide<T>::pair_of(q, i), acc[u][i]);
            }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t v = at.v + u * lanes;
        if (v >= a.vectors) continue;
        uint4 o;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) Wide<T>::set_pair(o, i, acc[u][i]);
        out.write(out.at(v), a.width, o);
    }
}

// 2^log_lanes threads hold a pair: they write its row of dy and sum its product
// in a fixed order.  Pairs of a token are neighbours, so that its row of dout
// comes from the caches after the first.
template <typename T, int MODE>
__global__ void __launch_bounds__(kRowThreads, MODE == kShifted ? kShiftedBackward : 1) k_combine_backward(const RowArgs<T> a) {
    if (blockIdx.x < a.fill_blocks) {
        fill_rows<T, MODE>(a);
        return;
    }
    constexpr int N = Wide<T>::kCount, U = MODE == kShifted ? 1 : 2;
    __shared__ float s_dot[kRowThreads / 32];
    const uint32_t lanes = 1u << a.log_lanes, warp = threadIdx.x >> 5;
    const uint32_t pr = (blockIdx.x - a.fill_blocks) * (kRowThreads >> a.log_lanes) + (threadIdx.x >> a.log_lanes);
    const uint32_t pairs = a.tokens * a.chosen;
    const uint32_t p = pr < pairs ? static_cast<uint32_t>(a.positions[pr]) : a.capacity;
    Pair dots = pair(0.0f, 0.0f);
    if (p < a.capacity) {
        const float w = a.weights[pr];
        const InRow<T> d_row = token_row(a, pr / a.chosen), y_row = layout_row(a, p);
        const OutRow<T, MODE> out(a.out + static_cast<int64_t>(p) * a.width);
        for (uint32_t v0 = threadIdx.x & (lanes - 1); v0 < a.vectors; v0 += lanes * U) {
            Loaded d[U], y[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t v = min(v0 + u * lanes, a.vectors - 1);       // no branch around the loads
                d[u] = start_read<T, MODE>(d_row, out.at(v), a.width, a.token_safe);
                y[u] = start_read<T, MODE>(y_row, out.at(v), a.width, a.row_safe);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t v = v0 + u * lanes;
                if (v >= a.vectors) continue;
                const int32_t e = out.at(v);
                const uint4 dq = end_read<T, MODE>(d[u], d_row, e, a.width);
                const uint4 yq = end_read<T, MODE>(y[u], y_row, e, a.width);
                const bool whole = MODE == kSingle || out.whole(e, a.width);    // kSingle reads 0 beside the row
                uint4 g;
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    Pair x = Wide<T>::pair_of(dq, i), z = Wide<T>::pair_of(yq, i);
                    if (!whole) {          // what is beside the row is no part of the product
                        if (static_cast<uint32_t>(e + 2 * i) >= a.width) x.f.x = z.f.x = 0.0f;
                        if (static_cast<uint32_t>(e + 2 * i + 1) >= a.width) x.f.y = z.f.y = 0.0f;
                    }
                    dots = fma2(x, z, dots);
                    Wide<T>::set_pair(g, i, mul2(pair(w, w), x));
                }
                out.write(e, a.width, g);
            }
        }
    }
    float dot = dots.f.x + dots.f.y;
    for (uint32_t o = 1; o < min(lanes, 32u); o <<= 1) dot += __shfl_xor_sync(kFullMask, dot, o);
    if (lanes > 32) {
        if ((threadIdx.x & 31) == 0) s_dot[warp] = dot;
        __syncthreads();
        dot = 0.0f;
        for (uint32_t i = 0; i < lanes / 32; ++i) dot += s_dot[(warp & ~(lanes / 32 - 1)) + i];
    }
    if ((threadIdx.x & (lanes - 1)) == 0 && pr < pairs) a.grad_weights[pr] = dot;
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
    a.tokens = static_cast<uint32_t>(L.tokens);
    a.token_stride = L.token_stride;
    a.row_stride = L.row_stride;
    a.chosen = L.chosen;
    a.capacity = static_cast<uint32_t>(L.capacity);
    a.width = static_cast<uint32_t>(L.width);
    a.token_safe = safe_in(L.by_token);
    a.row_safe = safe_in(L.by_row);
    return a;
}

// Calls f(arguments, mode).  SUMS: the rows are summed, not only copied.
template <bool SUMS, typename F> int with_rows(const RowsLaunch &L, F &&f) {
    using std::integral_constant;
    return with_float_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int N = Wide<T>::kCount;
        RowArgs<T> a = row_args<T>(L);
        auto fits = [&](const void *p, int64_t stride) { return p == nullptr || (aligned(p, 16) && stride % N == 0); };
        const bool some = L.tokens > 0 && L.capacity > 0;
        if (some && L.width % N == 0 && fits(L.by_token, L.token_stride) && fits(L.by_row, L.row_stride) && fits(L.out, L.width)) {
            a.vectors = a.width / N;
            return f(a, integral_constant<int, kAligned>{});
        }
        a.vectors = (a.width + 2 * (N - 1)) / N;     // a row of `width` can touch so many
        if constexpr (SUMS && sizeof(T) == 4) {
            if (some) {
                a.vectors = (a.width + 127) / 128 * 32;
                return f(a, integral_constant<int, kSingle>{});
            }
        } else {
            if (some && L.width * sizeof(T) >= 64) return f(a, integral_constant<int, kShifted>{});
        }
        return f(a, integral_constant<int, kElements>{});
    });
}

// CTAs that walk all tokens' rows so.
template <typename T> int64_t split_rows(RowArgs<T> &a, int per_thread) {
    a.log_lanes = lanes_for(a.vectors, per_thread);
    const uint32_t step = per_thread << a.log_lanes, tokens = kRowThreads >> a.log_lanes;
    a.chunks = (a.vectors + step - 1) / step;
    return static_cast<int64_t>((a.tokens + tokens - 1) / tokens) * a.chunks;
}

template <typename T> void set_fill(RowArgs<T> &a) {
    // a row to a warp in a small layout, up to 32 in a large one (8 KB rows of 256 experts
    // padded to 16: 512 pairs 6.9 us, 32 with 32 rows to a warp; 131072 pairs 187, 200 with one)
    const uint32_t rows = std::min(32u, std::max(1u, a.capacity / 4096)) * (kRowThreads / 32);
    a.fill_blocks = (a.capacity + rows - 1) / rows;
}

template <int J, int U, typename T, int MODE> int start_combine(const RowsLaunch &L, RowArgs<T> &a) {
    const int64_t blocks = split_rows(a, U);
    if (blocks > 0x7FFFFFFF) return GSORT_ETOOBIG;
    k_combine<T, MODE, J, U><<<static_cast<uint32_t>(blocks), kRowThreads, 0, L.stream>>>(a);
    return launch_status();
}

}  // namespace

int launch_dispatch(const RowsLaunch &L) {
    return with_rows<false>(L, [&](auto &a, auto m) {
        constexpr int MODE = decltype(m)::value;
        const int64_t blocks = split_rows(a, 1);
        set_fill(a);
        if (blocks + a.fill_blocks > 0x7FFFFFFF) return static_cast<int>(GSORT_ETOOBIG);
        using T = std::decay_t<decltype(*a.out)>;
        k_dispatch<T, MODE><<<a.fill_blocks + static_cast<uint32_t>(blocks), kRowThreads, 0, L.stream>>>(a);
        return launch_status();
    });
}

int launch_combine(const RowsLaunch &L) {
    return with_rows<true>(L, [&](auto &a, auto m) {
        constexpr int MODE = decltype(m)::value;
        using T = std::decay_t<decltype(*a.out)>;
        // four 16-byte loads in flight: 16384 x 8 rows of 8 KB take 200 us so, 255 with eight
        if constexpr (MODE == kShifted || MODE == kSingle) {
            return start_combine<2, 2, T, MODE>(L, a);
        } else {
            if (L.chosen == 1) return start_combine<1, 4, T, MODE>(L, a);
            if (L.chosen == 2) return start_combine<2, 2, T, MODE>(L, a);
            return start_combine<4, 1, T, MODE>(L, a);
        }
    });
}

int launch_combine_backward(const RowsLaunch &L) {
    return with_rows<true>(L, [&](auto &a, auto m) {
        constexpr int MODE = decltype(m)::value;
        using T = std::decay_t<decltype(*a.out)>;
        const int64_t pairs = L.tokens * L.chosen;
        // up to a warp to a pair where pairs fill the device, else up to a CTA (4096 bf16, a
        // warp / a CTA to a pair: 1024 pairs 6.5 / 4.9 us, 2432 9.7 / 11.3, 4928 18.9 / 21.7, 16384
        // 50 / 72; 1001 bf16: 1024 4.7 / 3.5, 4928 9.5 / 8.2, 16384 18.9 / 20.7)
        a.log_lanes = lanes_for(a.vectors, 2);
        if (pairs >= 8 * 4 * L.sm_count) a.log_lanes = std::min(a.log_lanes, 5u);
        const int64_t per = kRowThreads >> a.log_lanes, blocks = (pairs + per - 1) / per;
        set_fill(a);
        if (blocks + a.fill_blocks > 0x7FFFFFFF) return static_cast<int>(GSORT_ETOOBIG);
        k_combine_backward<T, MODE><<<a.fill_blocks + static_cast<uint32_t>(blocks), kRowThreads, 0, L.stream>>>(a);
        return launch_status();
    });
}

}  // namespace gsort
