// group.cu -- stable grouping of (token, slot) pairs by expert: one pass of a
// counting sort with up to 1024 bins, giving each expert's padded segment.
//
// With n the pair's index and e its expert (anything outside [0, E) drops the
// pair), c_e the expert's pairs and A the alignment:
//   offsets[e + 1] = offsets[e] + roundup(c_e, A)
//   positions[n]   = offsets[e] + pairs of e before n   (-1: dropped)
//   rows[positions[n]] = n, every other entry of rows is -1
//
// Up to one tile (4096 pairs): one CTA.  More: a counting kernel, then a
// placing kernel whose CTAs each add up the counts of the CTAs before them
// (a few hundred rows of counts, read from L2), so no CTA waits on another.
// Ranks are warp multisplits over consecutive pairs, and every sum is an integer
// sum: the result does not depend on the order of execution.  The peers of a lane
// are bits that its warp sets in one word for each expert: match_any takes longer
// the more experts a warp meets (4096 pairs of 256 experts: 11.2 us with it, 9.3
// with a vote on every bit of the expert).
#include <algorithm>

#include "model_ops.cuh"

namespace gsort {
namespace {

constexpr int kGroupThreads = 1024;
constexpr int kGroupWarps = kGroupThreads / 32;
constexpr int kGroupItems = 4;                                   // pairs per thread and tile
constexpr uint32_t kGroupTile = kGroupThreads * kGroupItems;
// CTAs of one launch: each reads the counts of all of them, so there are no more than
// run at once, and the workspace's size does not depend on the device (152 SMs here).
constexpr uint32_t kGroupMaxTiles = 148;

struct GroupArgs {
    const int32_t *experts_in;
    uint32_t pairs, span;     // pairs per CTA, a multiple of the tile
    uint32_t experts, align, capacity, tiles;
    int32_t *offsets, *counts, *rows, *positions;
    uint32_t *ws;             // [tiles][experts]
};

__global__ void __launch_bounds__(kGroupThreads) k_group_count(const GroupArgs a) {
    extern __shared__ uint32_t s_hist[];   // [experts]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the placing kernel ranks its pairs meanwhile
    for (uint32_t e = threadIdx.x; e < a.experts; e += kGroupThreads) s_hist[e] = 0;
    __syncthreads();
    const uint32_t begin = blockIdx.x * a.span;
    const uint32_t end = min(a.pairs, begin + a.span);
    for (uint32_t n = begin + threadIdx.x; n < end; n += kGroupThreads) {
        const uint32_t e = static_cast<uint32_t>(a.experts_in[n]);
        if (e < a.experts) atomicAdd(&s_hist[e], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.experts; e += kGroupThreads) a.ws[blockIdx.x * a.experts + e] = s_hist[e];
}

// Shared memory of the placing kernel: u32 total[E], base[E], start[E], scan[33],
// peers[warps][E], then u16 counts[warps][E].
__global__ void __launch_bounds__(kGroupThreads) k_group_place(const GroupArgs a) {
    extern __shared__ uint32_t s_mem[];
    uint32_t *s_total = s_mem, *s_base = s_mem + a.experts, *s_start = s_mem + 2 * a.experts, *s_scan = s_mem + 3 * a.experts;
    uint32_t *s_peer = s_scan + 33;
    uint16_t *s_count = reinterpret_cast<uint16_t *>(s_peer + kGroupWarps * a.experts);
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t E = a.experts;
    const uint32_t begin = blockIdx.x * a.span;
    const uint32_t end = min(a.pairs, begin + a.span);

    for (uint32_t i = tid; i < E * kGroupWarps; i += kGroupThreads) s_peer[i] = 0;

    for (uint32_t tile = begin;; tile += kGroupTile) {
        // ranks of the tile's pairs among their expert's pairs in the warp
        for (uint32_t i = tid; i < E * kGroupWarps / 2; i += kGroupThreads) reinterpret_cast<uint32_t *>(s_count)[i] = 0;
        __syncthreads();
        uint32_t key[kGroupItems], rank[kGroupItems];
        const uint32_t first = tile + warp * (32 * kGroupItems) + lane;
#pragma unroll
        for (int i = 0; i < kGroupItems; ++i) {
            const uint32_t n = first + i * 32;
            key[i] = n < end ? min(static_cast<uint32_t>(a.experts_in[n]), E) : E;   // E: dropped or beyond the end
        }
        uint16_t *count = s_count + warp * E;
        uint32_t *peer = s_peer + warp * E;
#pragma unroll
        for (int i = 0; i < kGroupItems; ++i) {
            // lanes with the same expert: each sets its bit in the warp's word of the expert
            const bool in = key[i] < E;
            if (in) atomicOr(&peer[key[i]], 1u << lane);
            __syncwarp();
            const uint32_t peers = in ? peer[key[i]] : 0u, had = in ? count[key[i]] : 0u;
            const bool first_peer = in && (peers & lanemask_lt()) == 0u;
            rank[i] = had + __popc(peers & lanemask_lt());
            __syncwarp();
            if (first_peer) {
                count[key[i]] = static_cast<uint16_t>(had + __popc(peers));
                peer[key[i]] = 0u;
            }
            __syncwarp();
        }
        __syncthreads();
        // exclusive scan over the warps, expert by expert
        uint32_t tile_total = 0;     // of expert `tid`
        if (tid < E) {
#pragma unroll 8
            for (int w = 0; w < kGroupWarps; ++w) {
                const uint32_t c = s_count[w * E + tid];
                s_count[w * E + tid] = static_cast<uint16_t>(tile_total);
                tile_total += c;
            }
        }
        if (tile == begin) {
            // counts of every expert over all CTAs, and over the CTAs before this one
            if (a.tiles > 1) {
                asm volatile("griddepcontrol.wait;" ::: "memory");     // the counts are complete
                if (tid < E) s_total[tid] = 0, s_base[tid] = 0;
                __syncthreads();
                const uint32_t parts = kGroupThreads / E, part = tid / E, e = tid % E;
                if (part < parts) {
                    uint32_t total = 0, before = 0;
#pragma unroll 16
                    for (uint32_t b = part; b < a.tiles; b += parts) {
                        const uint32_t c = a.ws[b * E + e];
                        total += c;
                        if (b < blockIdx.x) before += c;
                    }
                    if (total) atomicAdd(&s_total[e], total);
                    if (before) atomicAdd(&s_base[e], before);
                }
            } else if (tid < E) {
                s_total[tid] = tile_total;
                s_base[tid] = 0;
            }
            __syncthreads();
            // padded segments: block-wide exclusive scan, one expert per thread
            const uint32_t have = tid < E ? s_total[tid] : 0u;
            const uint32_t padded = (have + a.align - 1) / a.align * a.align;
            const uint32_t incl = warp_inclusive_scan(padded, lane);
            if (lane == 31) s_scan[warp] = incl;
            __syncthreads();
            if (warp == 0) {
                const uint32_t v = s_scan[lane];
                s_scan[lane] = warp_inclusive_scan(v, lane) - v;
            }
            __syncthreads();
            const uint32_t start = s_scan[warp] + incl - padded;
            if (tid < E) {
                s_base[tid] += start;
                if (blockIdx.x == 0) {
                    a.counts[tid] = static_cast<int32_t>(have);
                    a.offsets[tid] = static_cast<int32_t>(start);
                    if (tid == E - 1) a.offsets[E] = static_cast<int32_t>(start + padded);
                }
                s_start[tid] = start;
                if (tid == E - 1) s_scan[32] = start + padded;
            }
            __syncthreads();
            // padding: of the experts that fall to this CTA, a thread each, or a warp
            // where it can be long; and the layout's end
            if (a.align <= 32) {
                if (tid < E && tid % a.tiles == blockIdx.x)
                    for (uint32_t p = start + have; p < start + padded; ++p) a.rows[p] = -1;
            } else {
                for (uint32_t e = blockIdx.x + warp * a.tiles; e < E; e += a.tiles * kGroupWarps) {
                    const uint32_t end_e = e + 1 < E ? s_start[e + 1] : s_scan[32];
                    for (uint32_t p = s_start[e] + s_total[e] + lane; p < end_e; p += 32) a.rows[p] = -1;
                }
            }
            for (uint32_t p = s_scan[32] + blockIdx.x * kGroupThreads + tid; p < a.capacity; p += a.tiles * kGroupThreads) a.rows[p] = -1;
        } else {
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kGroupItems; ++i) {
            const uint32_t n = first + i * 32;
            if (n < end) {
                int32_t p = -1;
                if (key[i] < E) {
                    const uint32_t to = s_base[key[i]] + count[key[i]] + rank[i];
                    if (to < a.capacity) {     // always, unless the experts change meanwhile
                        p = static_cast<int32_t>(to);
                        a.rows[to] = static_cast<int32_t>(n);
                    }
                }
                a.positions[n] = p;
            }
        }
        if (tile + kGroupTile >= end) break;   // the same for the whole CTA
        __syncthreads();
        if (tid < E) s_base[tid] += tile_total;
    }
}

size_t place_smem(uint32_t experts) { return (3 * experts + 33) * 4 + static_cast<size_t>(kGroupWarps) * experts * 6; }

uint32_t group_tiles(uint32_t pairs) {
    return std::max(1u, std::min(kGroupMaxTiles, (pairs + kGroupTile - 1) / kGroupTile));
}

}  // namespace

size_t group_workspace_bytes(uint32_t pairs, int experts) {
    const uint32_t tiles = group_tiles(pairs);
    return tiles > 1 ? static_cast<size_t>(tiles) * experts * 4 : 0;
}

int launch_group(const GroupLaunch &L) {
    GroupArgs a{};
    a.experts_in = L.experts_in;
    a.pairs = L.pairs;
    a.experts = L.experts;
    a.align = L.align;
    a.capacity = L.capacity;
    a.offsets = L.offsets;
    a.counts = L.counts;
    a.rows = L.rows;
    a.positions = L.positions;
    a.ws = L.ws;
    const uint32_t most = group_tiles(L.pairs);
    const uint32_t per = (L.pairs + most - 1) / most;
    a.span = std::max(kGroupTile, (per + kGroupTile - 1) / kGroupTile * kGroupTile);
    a.tiles = std::max(1u, (L.pairs + a.span - 1) / a.span);
    // the limit is the kernel's largest need: it is set once, for every number of experts
    if (set_smem_limit(reinterpret_cast<const void *>(&k_group_place), place_smem(GSORT_ROUTE_MAX_EXPERTS)) != cudaSuccess)
        return GSORT_ECUDA;
    const size_t smem = place_smem(a.experts);
    if (a.tiles > 1) {
        k_group_count<<<a.tiles, kGroupThreads, a.experts * 4, L.stream>>>(a);
        if (cudaGetLastError() != cudaSuccess) return GSORT_ECUDA;
    }
    // The placing kernel may start while the counting kernel runs: up to its wait
    // it only reads the experts.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.tiles);
    cfg.blockDim = dim3(kGroupThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.tiles > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_group_place, a) == cudaSuccess ? GSORT_OK : GSORT_ECUDA;
}

}  // namespace gsort
