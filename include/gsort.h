/*
 * gsort.h -- C ABI of libgsort.so: GB300 (sm_103a) stable LSD radix sort,
 * stream compaction, segmented bitonic sort, and the selection and grouping
 * operators of language models (expert routing, token log probabilities).
 *
 * Sources of the operations (reference pages, by title and section):
 *   [PMPP10]  "Parallel Patterns: Sorting on the GPU" (textbook chapter 10):
 *             10.2 Bitonic Sort, 10.3 Radix Sort, 10.6 Key-Value sorting,
 *             10.7 stable vs unstable sorting, section 8 exercises.
 *   [CUDA3]   "CUDA 算子笔记 3" (CUDA operator notes 3): Stream Compaction
 *             (three kernels; decoupled look-back), Radix Sort (CPU LSD
 *             sort; processing several bits at once: histogram of every
 *             pass, scan of the bins, one-pass scatter with look-back).
 *   [WGPU41]  "WebGPU Unleashed 4.1 Radix Sort": key/id pair buffers,
 *             stable per-digit reordering.
 *   [GPUSORT] "gpu排序" (GPU sort): bitonic sort of <=1024 keys per block,
 *             padded with 0xFFFFFFFF.
 *
 * Conventions shared by every call:
 *   - Pointers named d_* are DEVICE pointers on the current CUDA device.
 *     The caller owns every buffer, including the workspace; the library
 *     never allocates or frees memory and keeps no state between calls.
 *   - Every call is asynchronous on `stream` (0 = legacy default stream).
 *     Argument errors and launch errors are returned at once.  Errors that
 *     only the device can see (a look-back wait that gave up) are recorded
 *     in the workspace and returned by gsort_check().
 *   - 32-bit data must be 4-byte aligned (else GSORT_EALIGN).  Buffers that
 *     are also 16-byte aligned take 128-bit vector paths; others take a
 *     scalar path with identical results.
 *   - n counts elements.  0 <= n <= GSORT_MAX_N (larger: GSORT_ETOOBIG);
 *     n == 0 is a no-op returning GSORT_OK.  The cap comes from the 30-bit
 *     count field of the look-back state words.
 *   - Workspaces must be 256-byte aligned (torch and cudaMalloc allocations
 *     are).  Their contents on entry do not matter.  Two calls that share a
 *     workspace must not run concurrently.
 */
#ifndef GSORT_H
#define GSORT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same definition as the CUDA runtime's, so either header may come first. */
typedef struct CUstream_st *cudaStream_t;

typedef enum gsort_status {
    GSORT_OK = 0,
    GSORT_EINVAL = -1,      /* bad argument: NULL, bad range, overlapping buffers */
    GSORT_EALIGN = -2,      /* a pointer is not 4-byte (data) or 256-byte (workspace) aligned */
    GSORT_EWORKSPACE = -3,  /* workspace missing or smaller than the *_workspace_bytes() answer */
    GSORT_ETOOBIG = -4,     /* n above the entry point's maximum (GSORT_MAX_N, or the smaller limit it states) */
    GSORT_ECUDA = -5,       /* a CUDA runtime call or kernel launch failed */
    GSORT_ETIMEOUT = -6     /* a device-side look-back wait gave up (see gsort_check) */
} gsort_status;

typedef enum gsort_key_kind {
    GSORT_KEY_U32 = 0,      /* unsigned 32-bit integers */
    GSORT_KEY_F32 = 1,      /* IEEE-754 binary32, ordered as totalOrder for non-NaN */
    GSORT_KEY_I32 = 2,      /* two's-complement 32-bit integers */
    GSORT_KEY_U64 = 3,      /* unsigned 64-bit integers */
    GSORT_KEY_F64 = 4,      /* IEEE-754 binary64, ordered as totalOrder for non-NaN */
    GSORT_KEY_I64 = 5       /* two's-complement 64-bit integers */
} gsort_key_kind;

/* Flags of gsort_radix_sort(). */
#define GSORT_DESCENDING 1  /* largest key first; equal keys keep their input order */

#define GSORT_MAX_N ((int64_t)((1 << 30) - 1))

/* Human-readable name of a status code (static string). */
const char *gsort_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
int gsort_version(void);

/* ------------------------------------------------------------------------
 * Radix sort  ([PMPP10] 10.3, 10.6, 10.7; [CUDA3] Radix Sort, several bits
 * at once; [WGPU41])
 *
 * Stable LSD radix sort with 8-bit digits, least significant digit first.
 * One upfront pass reads the keys once and builds the 256-bin histogram of
 * every digit; each digit pass then scatters every element to
 *   (keys with a smaller digit) + (keys with this digit in earlier tiles)
 *   + (its stable rank among this digit's keys in its own tile),
 * where the middle term comes from a decoupled look-back over per-(tile,
 * digit) counts.  Equal keys keep their input order; values move with keys.
 *
 * Keys only, sorted by every bit of the key: equal keys are identical, so a
 * pass needs the input order only between keys that differ in the bits
 * below its digit.  There the first pass places keys in any order within
 * their bin (atomic bin cursors instead of the look-back), and a warp whose
 * keys agree below the digit ranks them by shared atomics instead of the
 * multisplit.  The output is the same (a sorted key sequence is unique);
 * the intermediate order may differ from run to run.
 *
 * Float keys (GSORT_KEY_F32): the bit pattern is mapped to an unsigned
 * integer that orders every non-NaN value as IEEE totalOrder (-inf < ... <
 * -0 < +0 < ... < +inf); the output holds the original bit patterns.
 * ([PMPP10] section 8, exercise 7 poses the question; this is the reading
 * taken.)  NaNs are not promised an order; with this map +NaN sorts after
 * +inf and -NaN before -inf.
 * ---------------------------------------------------------------------- */

/* Workspace bytes for sorting n elements (with_values != 0: pairs).
 * Holds a status word, counters, the digit histograms, two look-back
 * state regions and one ping-pong buffer per sorted array. */
size_t gsort_radix_workspace_bytes(int64_t n, int with_values);

/* Sort n 32-bit keys (kind GSORT_KEY_U32, F32 or I32) ascending by all 32
 * bits.  d_keys_in is not modified unless it equals d_keys_out (in place is
 * allowed).  Partially overlapping buffers: GSORT_EINVAL. */
int gsort_radix_keys(const void *d_keys_in, void *d_keys_out, int64_t n,
                     int kind, void *d_ws, size_t ws_bytes, cudaStream_t stream);

/* Stable sort of (key, value) pairs by key bits [begin_bit, end_bit)
 * (0 <= begin_bit <= end_bit <= 32) for the 32-bit kinds U32, F32 and I32
 * (other kinds: GSORT_EINVAL; gsort_radix_sort takes every kind).  Bits
 * outside the range do not take part in the order but are carried.
 * begin_bit == end_bit copies.  For F32 and I32 the range applies to the
 * mapped key (use 0..32).
 * d_vals_in and d_vals_out are both NULL (keys only) or both non-NULL.
 * In-place (in == out) is allowed for keys and for values. */
int gsort_radix_pairs(const void *d_keys_in, void *d_keys_out,
                      const uint32_t *d_vals_in, uint32_t *d_vals_out, int64_t n,
                      int kind, int begin_bit, int end_bit,
                      void *d_ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * General radix sort: every key kind, ascending or descending.
 * ([PMPP10] section 8, exercises 2 (64-bit keys: 8 passes of radix 256),
 * 6 (descending order) and 7 (float keys); signed keys flip the sign bit,
 * the same idea for two's complement.)
 *
 * Stable sort of n keys of `kind` (4- or 8-byte words, see gsort_key_kind),
 * with optional 32-bit values, by the bits [begin_bit, end_bit) of the
 * mapped key: the key's bit pattern taken through the order map of its kind
 * (identity for unsigned, sign bit flipped for signed, the totalOrder map for
 * floats), complemented when flags has GSORT_DESCENDING.  0 <= begin_bit <=
 * end_bit <= 8 * key bytes; 0..32 or 0..64 sorts by the whole key.  Equal
 * (masked) keys keep their input order in both directions.  Output keys
 * hold the original bit patterns.
 *
 * Keys must be aligned to their size (else GSORT_EALIGN), values to 4 bytes.
 * In place, aliasing and NULL rules as for gsort_radix_pairs.  flags other
 * than 0 and GSORT_DESCENDING: GSORT_EINVAL.  The workspace comes from
 * gsort_radix_sort_workspace_bytes() with the same kind; for 32-bit kinds it
 * equals gsort_radix_workspace_bytes().
 * ---------------------------------------------------------------------- */
size_t gsort_radix_sort_workspace_bytes(int64_t n, int kind, int with_values);

int gsort_radix_sort(const void *d_keys_in, void *d_keys_out,
                     const uint32_t *d_vals_in, uint32_t *d_vals_out, int64_t n,
                     int kind, int flags, int begin_bit, int end_bit,
                     void *d_ws, size_t ws_bytes, cudaStream_t stream);

/* The upfront histogram step on its own: d_hist_out receives
 * passes * 256 uint32 counts, passes = ceil((end_bit - begin_bit) / 8);
 * entry [p * 256 + d] counts the keys whose p-th 8-bit digit (from
 * begin_bit, last digit narrowed to end_bit) of the mapped key (ascending
 * order map of `kind`, any kind; end_bit <= 8 * key bytes) is d.  Needs no
 * workspace. */
int gsort_digit_histograms(const void *d_keys, int64_t n, int kind,
                           int begin_bit, int end_bit, uint32_t *d_hist_out,
                           cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Stream compaction  ([CUDA3] Stream Compaction: predicate, exclusive scan,
 * scatter; the single-pass decoupled look-back version)
 *
 * Writes every d_in[i] > 0 (IEEE: NaN, +0 and -0 are dropped, positive
 * subnormals kept) to d_out[0..m) in input order and +0.0 to d_out[m..n).
 * If d_num_kept is not NULL, *d_num_kept = m (device int64) on completion.
 * d_in and d_out must not overlap.
 * ---------------------------------------------------------------------- */
size_t gsort_compact_workspace_bytes(int64_t n);

int gsort_compact_positive(const float *d_in, float *d_out, int64_t n,
                           int64_t *d_num_kept, void *d_ws, size_t ws_bytes,
                           cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Allocation-free compaction.  The reference pages have no counterpart: this
 * call exists for callers that cannot provide a workspace, because they run
 * where device allocation is forbidden or too costly (the execute step of a
 * plugin whose host framework owns all device memory, a real-time loop that
 * cannot afford cudaMalloc's device-wide synchronisation and latency, a
 * handler that runs while the caller's allocator is busy).
 *
 * Same result as gsort_compact_positive, for 0 <= n <=
 * GSORT_COMPACT_NOALLOC_MAX_N (larger: GSORT_ETOOBIG).  The caller still
 * passes the input, the output and the optional kept count.  The scratch is
 * one static device array inside the library (about 4 MiB), which every GPU
 * that loads the library keeps until the process exits; this call allocates
 * nothing.  The first call on a device looks up that array's device address
 * (make that first call before any stream capture); later calls reuse it.
 * All calls share the array: calls whose work overlaps on the GPU (for
 * example on two streams at once) race and corrupt each other's results, so
 * serialise them.  A device-side look-back timeout, which does not occur in
 * normal operation, leaves the output undefined and is not reported here.
 * ---------------------------------------------------------------------- */
#define GSORT_COMPACT_NOALLOC_MAX_N ((int64_t)1 << 28)

int gsort_compact_positive_noalloc(const float *d_in, float *d_out, int64_t n,
                                   int64_t *d_num_kept, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Segmented bitonic sort  ([GPUSORT] sort of <=1024 elements in one block;
 * [PMPP10] 10.2)
 *
 * Sorts each of num_segments consecutive segments of segment_len uint32
 * keys ascending, in place, with the bitonic network held in registers
 * (one warp per segment).  1 <= segment_len <= 1024; lengths that are not a
 * power of two are padded internally with 0xFFFFFFFF.  num_segments >= 0.
 * Not stable (keys only, so the result is still unique).
 * ---------------------------------------------------------------------- */
int gsort_segmented_bitonic(uint32_t *d_keys, int64_t num_segments,
                            int segment_len, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Stable 2-way split (partition)  ([CUDA3] "Radix Sort": predicate,
 * exclusive scan, scatter of one side before the other; "Stream
 * Compaction" keeps only one side)
 *
 * Writes every element whose predicate holds, in input order, to
 * d_out[0..m) and every other element, in input order, to d_out[m..n);
 * values (optional, 32-bit) move with their elements; *d_num_true = m
 * (device int64, may be NULL).  d_in/d_vals_in must not overlap the outputs.
 * Predicates on the 32-bit word x of element i:
 *   GSORT_PRED_FLAGS       d_flags[i] != 0 (uint8 array of n entries)
 *   GSORT_PRED_BIT_SET     bit `param` of x is 1 (param < 32)
 *   GSORT_PRED_BIT_CLEAR   bit `param` of x is 0
 *   GSORT_PRED_LESS        x < param in the sort order of `kind` (U32, I32,
 *                          F32: IEEE totalOrder, so -0.0 < +0.0 and NaNs
 *                          fall outside +-inf, as in the radix sort)
 *   GSORT_PRED_POSITIVE    IEEE x > 0 for float bits (the compaction
 *                          predicate; NaN, +0 and -0 are false)
 * Traffic: one counting read, then one read and one write per element.
 * ---------------------------------------------------------------------- */
#define GSORT_PRED_FLAGS 0
#define GSORT_PRED_BIT_SET 1
#define GSORT_PRED_BIT_CLEAR 2
#define GSORT_PRED_LESS 3
#define GSORT_PRED_POSITIVE 4

size_t gsort_partition_workspace_bytes(int64_t n);

int gsort_partition(const uint32_t *d_in, uint32_t *d_out, const uint32_t *d_vals_in,
                    uint32_t *d_vals_out, int64_t n, int pred, int kind, uint32_t param,
                    const uint8_t *d_flags, int64_t *d_num_true, void *d_ws, size_t ws_bytes,
                    cudaStream_t stream);

/* ------------------------------------------------------------------------
 * 1-bit split radix sort  ([CUDA3] "Radix Sort": one predicate / scan /
 * scatter pass per bit, zeros before ones)
 *
 * Stable ascending sort of unsigned 32-bit keys (and 32-bit values) by the
 * bits [begin_bit, end_bit), one split pass per bit (up to 32): the pages'
 * bitwise LSD sort.  The zero count of every bit comes from one upfront
 * histogram read.  Same result as gsort_radix_pairs with GSORT_KEY_U32, at
 * about 8x its traffic; it exists as the pages' method and as a check of
 * the split primitive.  In place and aliasing rules as for
 * gsort_radix_pairs.
 * ---------------------------------------------------------------------- */
size_t gsort_split_sort_workspace_bytes(int64_t n, int with_values);

int gsort_split_sort(const uint32_t *d_keys_in, uint32_t *d_keys_out,
                     const uint32_t *d_vals_in, uint32_t *d_vals_out, int64_t n,
                     int begin_bit, int end_bit, void *d_ws, size_t ws_bytes,
                     cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Variable-length segmented sort  ([PMPP10] 10.5, strategy 2: radix sort
 * for the coarse order with bitonic networks for the small pieces;
 * [GPUSORT]: pieces of <= 1024 keys go to a bitonic sort)
 *
 * d_offsets holds num_segments + 1 uint32 entries with d_offsets[0] == 0,
 * d_offsets[s] <= d_offsets[s + 1] and d_offsets[num_segments] == n; segment
 * s is keys [d_offsets[s], d_offsets[s + 1]).  Each segment is sorted
 * stably by the whole key of `kind` (32-bit kinds: GSORT_KEY_U32, F32, I32;
 * others: GSORT_EINVAL), ascending, or descending with GSORT_DESCENDING;
 * equal keys keep their input order and values (optional, 32-bit) move
 * with their keys.  Segments of 2..1024 keys are sorted by one warp each
 * (register bitonic network; with values it sorts (key, position) pairs,
 * which makes it stable); longer segments by a radix sort whose tiles never
 * cross a segment boundary.  Empty segments are allowed.
 *
 * Offsets are read on the device: offsets that break the rules above make
 * the call record GSORT_EINVAL in the workspace (returned by gsort_check)
 * and leave the output unspecified; no memory outside the given arrays is
 * touched.  n == 0 is a no-op (the offsets are not read); num_segments == 0
 * requires n == 0.  In place (in == out, for keys and for values) is
 * allowed; other overlaps: GSORT_EINVAL.  The workspace comes from
 * gsort_segmented_sort_workspace_bytes(): 4.25 bytes per key for keys
 * only (8.25 with values) when every segment is long, growing with the
 * number of segments up to about 12.3 (16.3) bytes per key.
 * ---------------------------------------------------------------------- */
size_t gsort_segmented_sort_workspace_bytes(int64_t n, int64_t num_segments, int with_values);

int gsort_segmented_sort(const void *d_keys_in, void *d_keys_out,
                         const uint32_t *d_vals_in, uint32_t *d_vals_out, int64_t n,
                         const uint32_t *d_offsets, int64_t num_segments,
                         int kind, int flags, void *d_ws, size_t ws_bytes,
                         cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Language-model operators: the selection, grouping and row moves around a
 * layer of experts, and the selection over a model's output.
 *
 * Element types of activations and logits; arithmetic and sums are in 32
 * bits whatever the type, rounded once when stored.  Exponentials that enter
 * a sum over a row, or a 16-bit gradient, carry a relative error of up to 2^-22 +
 * (max - x) 2^-23; those of weights, choices and float32 gradients are within
 * 2^-21 of e^(x - max), the difference rounded to 32 bits.  Pointers are aligned to
 * their element (else GSORT_EALIGN); rows and bases that are also 16-byte
 * aligned move as 16-byte vectors.  Strides count elements, from one row to
 * the next; elements of a row are consecutive.  A count of zero rows is a
 * no-op returning GSORT_OK.  Outputs must not overlap inputs or each other
 * (GSORT_EINVAL), except where a call allows it.  Indices that the device
 * reads (experts, positions, targets) are checked there: one outside its
 * range takes no part, as each call states, and touches no memory.
 * ---------------------------------------------------------------------- */
typedef enum gsort_float {
    GSORT_F32 = 0,
    GSORT_BF16 = 1,
    GSORT_F16 = 2
} gsort_float;

/* Routing of tokens to experts.  Per token, with logits x of `experts`
 * experts (1..GSORT_ROUTE_MAX_EXPERTS):
 *   candidates  experts whose logit is above -inf (masked and NaN are none)
 *   score s     GSORT_SCORE_SOFTMAX: softmax over the candidates;
 *               GSORT_SCORE_SIGMOID: 1 / (1 + exp(-x))
 *   choice c    x if d_bias is NULL (s grows with x), else s + d_bias[e]; an
 *               expert whose choice value is -inf or NaN is no candidate
 *   groups      groups > 1 (a divisor of experts, at most 32): consecutive
 *               experts form groups of equal size; a group's value is
 *               GSORT_GROUP_MAX: its largest c, or GSORT_GROUP_TOP2: the sum
 *               of its two largest s (+ bias); experts outside the
 *               groups_kept best groups are no candidates
 *   chosen      the `chosen` (1..GSORT_ROUTE_MAX_CHOSEN, at most experts)
 *               largest c in descending order; ties, here and between groups,
 *               go to the lower index
 *   weight      scale * s, or with renormalise != 0 scale * s / (sum of the
 *               chosen s); a sigmoid of a logit below -745 counts as 0
 * d_weights and d_experts are [tokens][chosen]; where a token has fewer
 * candidates, the rest are expert -1 with weight 0. */
#define GSORT_SCORE_SOFTMAX 0
#define GSORT_SCORE_SIGMOID 1
#define GSORT_GROUP_MAX 0
#define GSORT_GROUP_TOP2 1
#define GSORT_ROUTE_MAX_EXPERTS 1024
#define GSORT_ROUTE_MAX_CHOSEN 32

int gsort_route_experts(const void *d_logits, int dtype, int64_t tokens, int experts,
                        int64_t row_stride, const float *d_bias, int score, int groups,
                        int groups_kept, int group_score, int chosen, int renormalise, float scale,
                        float *d_weights, int32_t *d_experts, cudaStream_t stream);

/* Gradient of the weights by the logits, for the chosen experts given: the
 * choice, the groups and the bias have none.  d_grad_logits is contiguous
 * [tokens][experts] of the logits' type and is written whole.  A token's
 * experts are distinct (or outside the range: no part). */
int gsort_route_experts_backward(const float *d_grad_weights, const void *d_logits, int dtype,
                                 int64_t tokens, int experts, int64_t row_stride,
                                 const int32_t *d_experts, int chosen, int score, int renormalise,
                                 float scale, void *d_grad_logits, cudaStream_t stream);

/* Stable grouping of (token, slot) pairs by expert.  With pair n's expert
 * e = d_experts[n] (outside 0..experts-1: the pair is dropped) and c_e pairs
 * of expert e:
 *   d_counts[e] = c_e                                       experts entries
 *   d_offsets[0] = 0, d_offsets[e + 1] = d_offsets[e] + c_e rounded up to a
 *                 multiple of align                          experts + 1 entries
 *   d_positions[n] = d_offsets[e] + pairs of e before n; -1: dropped
 *   d_rows[d_positions[n]] = n, every other entry -1        capacity entries
 * capacity = gsort_group_capacity(), the most rows that any experts can need
 * (0 where an argument is out of range or the result exceeds GSORT_MAX_N).
 * The workspace comes from gsort_group_workspace_bytes() and may be NULL where
 * that is 0. */
int64_t gsort_group_capacity(int64_t pairs, int experts, int align);
size_t gsort_group_workspace_bytes(int64_t pairs, int experts);

int gsort_group_by_expert(const int32_t *d_experts, int64_t pairs, int experts, int align,
                          int32_t *d_offsets, int32_t *d_counts, int32_t *d_rows, int64_t capacity,
                          int32_t *d_positions, void *d_ws, size_t ws_bytes, cudaStream_t stream);

/* Rows to the experts and back.  `width` elements to a row, `chosen` slots to
 * a token, positions and rows as gsort_group_by_expert gives them.  Positions
 * may be taken away afterwards: a pair whose position is outside
 * 0..capacity-1 takes no part, and the row that d_rows has for it counts as held
 * by no pair.  Outputs are contiguous and written whole.
 *   dispatch          d_out[positions[t][j]] = d_x[t]; rows that no pair
 *                     holds are zero
 *   combine           d_out[t] = sum over j of weights[t][j] *
 *                     d_y[positions[t][j]]; d_weights NULL: ones.  With ones
 *                     it is dispatch's gradient.
 *   combine_backward  d_grad_y[positions[t][j]] = weights[t][j] *
 *                     d_grad_out[t], rows that no pair holds are zero;
 *                     d_grad_weights[t][j] = sum of d_grad_out[t] *
 *                     d_y[positions[t][j]] (0 without a position) */
int gsort_dispatch_rows(const void *d_x, int dtype, int64_t tokens, int64_t width, int64_t row_stride,
                        const int32_t *d_positions, int chosen, const int32_t *d_rows,
                        int64_t capacity, void *d_out, cudaStream_t stream);

int gsort_combine_rows(const void *d_y, int dtype, int64_t capacity, int64_t width, int64_t row_stride,
                       const float *d_weights, const int32_t *d_positions, int64_t tokens, int chosen,
                       void *d_out, cudaStream_t stream);

int gsort_combine_rows_backward(const void *d_grad_out, int dtype, int64_t tokens, int64_t width,
                                int64_t grad_stride, const void *d_y, int64_t capacity,
                                int64_t row_stride, const float *d_weights,
                                const int32_t *d_positions, int chosen, const int32_t *d_rows,
                                void *d_grad_y, float *d_grad_weights, cudaStream_t stream);

/* Log probabilities of given tokens.  Per row of `vocab` logits x (1 ..
 * GSORT_MAX_N; -inf: masked):
 *   d_logprobs[r]      log softmax(x) at d_targets[r] (4- or 8-byte signed
 *                      integers, target_bytes); 0 for a negative target, NaN
 *                      for one beyond the vocabulary, -inf for a masked one;
 *                      both pointers NULL: not wanted
 *   d_entropy[r]       - sum of p log p (NULL: not wanted)
 *   d_stats[r][2]      max x and sum of exp(x - max x): the log of the sum of
 *                      exponentials is max + log(sum)
 *   d_top_logprobs[r][top], d_top_ids[r][top]   the `top` (0 ..
 *                      GSORT_LOGPROBS_MAX_TOP) largest logits' log
 *                      probabilities and indices, descending, ties to the
 *                      lower index; -inf and -1 where a row has fewer logits
 *                      above -inf
 * A row that is masked whole has log probabilities -inf and entropy 0.  A row
 * with NaN or +inf has NaN results (NaN is no alternative). */
#define GSORT_LOGPROBS_MAX_TOP 32

int gsort_token_logprobs(const void *d_logits, int dtype, int64_t rows, int64_t vocab,
                         int64_t row_stride, const void *d_targets, int target_bytes, int top,
                         float *d_logprobs, float *d_entropy, float *d_stats, float *d_top_logprobs,
                         int32_t *d_top_ids, cudaStream_t stream);

/* Gradient by the logits of sum over rows of grad_logprobs[r] * logprobs[r] +
 * grad_entropy[r] * entropy[r] (either gradient may be NULL: zeros), from the
 * forward call's entropy and stats.  d_grad_logits has rows grad_stride apart;
 * it may be the logits themselves (same pointer and stride).  A row without a
 * target takes no part through its log probability; a row that is masked whole
 * gets zeros. */
int gsort_token_logprobs_backward(const float *d_grad_logprobs, const float *d_grad_entropy,
                                  const void *d_logits, int dtype, int64_t rows, int64_t vocab,
                                  int64_t row_stride, const void *d_targets, int target_bytes,
                                  const float *d_entropy, const float *d_stats, void *d_grad_logits,
                                  int64_t grad_stride, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Device-side status: synchronises `stream`, then returns GSORT_OK or the
 * error a kernel recorded in this workspace during the last call that used
 * it (GSORT_ETIMEOUT), or GSORT_ECUDA if the stream reports an error.
 * ---------------------------------------------------------------------- */
int gsort_check(const void *d_ws, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Extended calls: the same operations with options for tracing, tuning and
 * testing.  A NULL options pointer means the defaults.
 * ---------------------------------------------------------------------- */
typedef struct gsort_options {
    /* Polls of one look-back wait before the kernel records GSORT_ETIMEOUT
     * and returns (0 = default, about a second of back-off). */
    uint32_t spin_limit;
    /* Testing only: the tile with this id never publishes its counts, so
     * waits behind it run out.  -1 = none. */
    int64_t stall_tile;
    /* Optional array of cudaEvent_t handles recorded on `stream` around the
     * launches: radix: [0] start, [1] after init, [2] after histogram,
     * [3 + p] after digit pass p; compaction: [0] start, [1] after init,
     * [2] and [3] after the scan/scatter kernel (which also writes the
     * zero tail).  Extra
     * entries are left alone; missing ones are skipped. */
    void **events;
    int num_events;
    /* Launch configuration of the digit passes of 32-bit keys (0 = default;
     * see gsort_radix_variant_name()); 64-bit keys have one configuration
     * and accept only 0. */
    int variant;
} gsort_options;

int gsort_radix_pairs_ex(const void *d_keys_in, void *d_keys_out,
                         const uint32_t *d_vals_in, uint32_t *d_vals_out, int64_t n,
                         int kind, int begin_bit, int end_bit,
                         void *d_ws, size_t ws_bytes, cudaStream_t stream,
                         const gsort_options *options);

int gsort_radix_sort_ex(const void *d_keys_in, void *d_keys_out,
                        const uint32_t *d_vals_in, uint32_t *d_vals_out, int64_t n,
                        int kind, int flags, int begin_bit, int end_bit,
                        void *d_ws, size_t ws_bytes, cudaStream_t stream,
                        const gsort_options *options);

/* Events for the segmented sort: [0] start, [1] after the classification,
 * [3] after the large segments' histograms, [4 + p] after digit pass p of
 * the large segments, [2] at the end, once the small segments are sorted too
 * (their networks run on streams of the library's own beside the large
 * segments' kernels; `stream` waits for them before [2]). */
int gsort_segmented_sort_ex(const void *d_keys_in, void *d_keys_out,
                            const uint32_t *d_vals_in, uint32_t *d_vals_out, int64_t n,
                            const uint32_t *d_offsets, int64_t num_segments,
                            int kind, int flags, void *d_ws, size_t ws_bytes,
                            cudaStream_t stream, const gsort_options *options);

int gsort_compact_positive_ex(const float *d_in, float *d_out, int64_t n,
                              int64_t *d_num_kept, void *d_ws, size_t ws_bytes,
                              cudaStream_t stream, const gsort_options *options);

/* Number of digit-pass launch configurations, and the name of one
 * ("warps x items per thread, ranking method"); NULL if out of range. */
int gsort_radix_num_variants(void);
const char *gsort_radix_variant_name(int variant);

/* Kernel launches one call makes with the default variant (for launch
 * accounting): radix: 2 for 32-bit keys and n <= 2^18 (one cooperative
 * kernel runs every pass), else 2 + passes (+1 copy-back when sorting in
 * place with an odd pass count; +1 histogram clear for 64-bit keys, see
 * gsort_radix_sort_launch_count); compaction: 2; segmented: 1 (0 when
 * there is nothing to do). */
int gsort_radix_launch_count(int64_t n, int begin_bit, int end_bit, int in_place);
int gsort_radix_sort_launch_count(int64_t n, int kind, int begin_bit, int end_bit, int in_place);

#ifdef __cplusplus
}
#endif

#endif /* GSORT_H */
