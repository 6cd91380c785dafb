/*
 * ep.h -- C ABI of the MI355X (gfx950) expert-parallel layout / dispatch /
 * combine library (libep.so).
 *
 * The operations follow these pages:
 *   [P1] "DeepEP Buffer Class API for Expert Parallel Communication:
 *        Architecture and Usage": "Configuration and Layout Helpers"
 *        (get_dispatch_layout), "Dispatch Operation", "Combine Operation",
 *        "IB-GDA Kernels" (low_latency_dispatch / low_latency_combine),
 *        "Explicit Resource Cleanup" (destroy) and the FAQ on the handle.
 *   [P3] DeepEP-Lib "Core Implementation" (C++ runtime): "Memory Alignment
 *        and Validation" (int4-multiple rows, buffer alignment).
 *   [P4] "How DeepEP Optimizes Handle Reuse for Repeated Dispatches": "What
 *        the Handle Contains", "Fast Path Dispatch with Handle Reuse",
 *        "Performance Contract and Constraints".
 *   [P5] "Chapter 10, V2: buffers beyond EP", section 10.2 (load-balance
 *        operations over redundant experts).
 *
 * The R destination ranks are logical partitions of this GPU's memory: a
 * "segment" is a contiguous range of rows of one caller buffer.  Nothing here
 * talks to another GPU.
 *
 * Conventions for every entry point
 *   - Memory: every array argument is a DEVICE pointer owned by the caller,
 *     except the ones documented as host pointers.  The library never frees
 *     caller memory.  The handle is the only library-owned memory.
 *   - Streams: `stream` is a hipStream_t (NULL = the legacy default stream).
 *     All device work is enqueued on it, in order; no call synchronizes the
 *     host unless its documentation says so.
 *   - Layouts are dense row-major.  bf16 tensors are 16-bit words.  topk_idx
 *     is int64 with -1 for a masked slot; weights are fp32.
 *   - Expert e belongs to rank e / (E/R) as local expert e % (E/R).
 *   - Alignment ([P3]): token-row pointers (x, recv_x, y, out, bias0, bias1,
 *     packed_x, packed_y, load-balance tensors) must be 16-byte aligned, and
 *     hidden*2 must be a multiple of 16 (rows are whole int4 vectors); int64
 *     arrays 8-byte, others 4-byte aligned.  Violations return EP_ERR_ALIGN
 *     before any work is enqueued.
 *   - Expert ids outside [-1, E) are invalid input.  The kernels ignore such
 *     slots (treat them as masked) so that no access leaves its buffer.
 *   - Errors: every int-returning call returns an ep_status.  On any error no
 *     work has been enqueued and no output pointer argument was written,
 *     except as noted.  Host-side errors never throw across the ABI.
 *   - Environment (read by the library, never required):
 *       EP_LOG=1     one line per kernel launch on stderr with its launch geometry;
 *       EP_TRACE=1   a roctx range around every entry point (rocprofv3 marker trace);
 *       EP_CHECK=1   the handle-reuse table check of ep_dispatch;
 *       EP_TUNE_DISPATCH / EP_TUNE_COMBINE   initial launch-shape overrides (ep_set_tuning).
 *   - Concurrency: calls may run on different streams concurrently as long
 *     as they do not write the same caller memory.  One handle may be read by
 *     several calls at once; it must not be freed while they are in flight
 *     on other streams than its last one (the freed memory is reused only by
 *     work on the handle's last stream).
 */
#ifndef EP_H
#define EP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void *ep_stream_t; /* a hipStream_t */

typedef enum ep_status {
    EP_OK = 0,
    EP_ERR_INVALID = 1,  /* bad dimension, NULL where required, forbidden argument mix */
    EP_ERR_ALIGN = 2,    /* pointer or row-size alignment rule broken */
    EP_ERR_CAPACITY = 3, /* caller buffer has fewer rows than the result needs */
    EP_ERR_HANDLE = 4,   /* handle does not match the dims, or NULL handle */
    EP_ERR_HIP = 5,      /* a HIP runtime call failed (see ep_last_hip_error) */
    EP_ERR_NOMEM = 6,    /* device or host allocation failed */
    EP_ERR_TOO_LARGE = 7 /* larger than the call takes (ep_get_dispatch_layout_noalloc, ep_ll_moe) */
} ep_status;

/* Problem sizes.  Limits: 0 <= num_tokens <= 2^24; hidden > 0, hidden % 8 == 0,
 * hidden <= 2^20; 1 <= num_topk <= 64; 1 <= num_ranks <= 512;
 * num_experts % num_ranks == 0, num_experts <= 8192; num_channels >= 1,
 * num_channels <= 4096. */
typedef struct ep_dims {
    int32_t num_tokens;   /* T */
    int32_t hidden;       /* H, bf16 elements per token row */
    int32_t num_topk;     /* K */
    int32_t num_experts;  /* E */
    int32_t num_ranks;    /* R */
    int32_t num_channels; /* C: channels are ceil(T/C)-token contiguous ranges */
} ep_dims;

/* Opaque, library-owned dispatch layout ("handle" of [P4] "What the Handle
 * Contains"): rank_prefix_matrix, channel_prefix_matrix,
 * recv_channel_prefix_matrix, recv_src_idx, is_token_in_rank, send_head, the
 * per-rank and per-expert counts, the dims, and per-token destination-row
 * lists.  Immutable once created; freed by ep_handle_free. */
typedef struct ep_handle ep_handle;

/* Caller-owned device outputs of the layout.  Any field may be NULL (not
 * wanted).  Shapes:
 *   num_tokens_per_rank        int32 [R]    tokens that go to rank r
 *   num_tokens_per_expert      int32 [E]    (token, slot) pairs naming e
 *   is_token_in_rank           uint8 [T][R] 1 iff t goes to r
 *   rank_prefix_matrix         int32 [R]    inclusive prefix of num_tokens_per_rank;
 *                                           segment r starts at row [r-1] (0 for r = 0),
 *                                           N = [R-1] rows in total
 *   channel_prefix_matrix      int32 [R][C] tokens of rank r before the end of channel c
 *   recv_channel_prefix_matrix int32 [R][C] tokens of rank r before the start of channel c
 *   send_head                  int32 [T][R] row of t inside segment r, -1 if none
 *   recv_src_idx               int32 [recv_src_cap] source token of packed row i, i < N
 */
typedef struct ep_layout_out {
    int32_t *num_tokens_per_rank;
    int32_t *num_tokens_per_expert;
    uint8_t *is_token_in_rank;
    int32_t *rank_prefix_matrix;
    int32_t *channel_prefix_matrix;
    int32_t *recv_channel_prefix_matrix;
    int32_t *send_head;
    int32_t *recv_src_idx;
    int64_t recv_src_cap; /* rows available in recv_src_idx */
} ep_layout_out;

/* Largest possible row count N of a dispatch: T * min(K, R). */
int64_t ep_max_recv_rows(const ep_dims *dims);

/*
 * [P1] "Configuration and Layout Helpers": compute the token-to-rank layout
 * of topk_idx [T][K] on the GPU, before any token data moves.
 *
 * out (nullable): fields that are non-NULL receive copies of the layout.  If
 *   out->recv_src_idx is non-NULL and recv_src_cap < ep_max_recv_rows(), the
 *   call waits for N (the layout's count kernel stores it into pinned host
 *   memory, which the host polls; the positions may still be being written
 *   when it returns) and returns EP_ERR_CAPACITY if N > recv_src_cap;
 *   then no output in `out` is written and no handle is returned (*handle_out
 *   is left unchanged; the layout's memory returns to the pool).
 * handle_out (nullable): receives a new handle holding the layout.  Such a
 *   handle may be given to one ep_dispatch together with the same topk_idx
 *   (the "pre-computed layout" of [P1] "Dispatch Operation").
 * rank_mask [R] int32 (nullable; [P1] "Dynamic Rank Masking", nonzero =
 *   masked): every slot whose expert lives on a masked rank is treated as a
 *   masked slot, so a masked rank gets no tokens and its experts count 0.
 *   The mask is read on the device when the layout kernels run.
 * No host synchronization unless noted above.
 */
int ep_get_dispatch_layout(const ep_dims *dims, const int64_t *topk_idx, const int32_t *rank_mask,
                           ep_layout_out *out, ep_handle **handle_out, ep_stream_t stream);

/*
 * ep_get_dispatch_layout for callers that cannot allocate (code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation): the
 * same layout, written into `out`, with no handle, no hipMalloc / hipFree /
 * host allocation and no host synchronization.  The layout kernels write the
 * caller's buffers directly; their scratch (and any output field left NULL)
 * lives in one static device array of EP_NOALLOC_SCRATCH_BYTES per GPU, held
 * until the process ends.  Every call on a GPU shares that GPU's array:
 * calls that overlap on one GPU (other streams, other threads) race and give
 * undefined results; calls in one stream's order are fine.  Nothing in the
 * array needs to start at zero.
 *   out: required.  Fields as for ep_get_dispatch_layout; recv_src_idx, when
 *     non-NULL, needs recv_src_cap >= ep_max_recv_rows() (EP_ERR_CAPACITY
 *     otherwise: N is not read back).  send_head must be 16-byte aligned and
 *     is_token_in_rank 4-byte aligned (EP_ERR_ALIGN), since the kernels store
 *     them 4 ranks at a time.
 *   The layout always takes the count and position kernels (the one-launch
 *   layout of the "layout" tuning knob is not used here).
 * A problem whose scratch would exceed EP_NOALLOC_SCRATCH_BYTES returns
 * EP_ERR_TOO_LARGE before anything is enqueued.
 */
#define EP_NOALLOC_SCRATCH_BYTES (32u << 20)
int ep_get_dispatch_layout_noalloc(const ep_dims *dims, const int64_t *topk_idx,
                                   const int32_t *rank_mask, ep_layout_out *out,
                                   ep_stream_t stream);

/*
 * [P1] "Dispatch Operation" and [P4] "Fast Path Dispatch with Handle Reuse":
 * pack token rows x [T][H] (bf16) into R contiguous per-rank segments of
 * recv_x [recv_cap][H] in token order: row S[r] + send_head[t][r] receives
 * x[t] for every rank r that t goes to.
 *
 *   *handle == NULL       fresh dispatch: topk_idx is required; the layout is
 *                         computed and a new handle is stored in *handle.
 *   handle from ep_get_dispatch_layout and not yet used by a dispatch:
 *                         the layout is reused; topk_idx / topk_weights may
 *                         be given and must be the table the layout came from.
 *   handle returned by an earlier dispatch (cached fast path):
 *                         topk_idx and topk_weights must be NULL
 *                         (EP_ERR_INVALID otherwise); only rows are packed.
 *
 * recv_topk_idx [recv_cap][K] int64 (nullable, needs topk_idx): slot k of
 *   packed row (t, r) holds e - r*(E/R) when slot k of t is valid and its
 *   expert e lives on r, else -1.
 * recv_topk_weights [recv_cap][K] fp32 (nullable, needs topk_weights): the
 *   slot's weight in the same case, else 0.
 * recv_x (nullable): NULL skips the row copy (layout / size query only).
 * recv_cap: rows available in recv_x / recv_topk_*.  If it is below N the
 *   call returns EP_ERR_CAPACITY.  When recv_cap >= ep_max_recv_rows() no
 *   host synchronization is needed to check it.
 * num_recv (HOST pointer, nullable): receives N; asking for it waits once
 *   per handle (later calls use the cached value).  On a fresh dispatch the
 *   layout's count kernel stores N into pinned host memory, which the host
 *   polls (no copy is enqueued, and the call does not wait for the position
 *   kernel); on a handle made earlier N is copied there once and polled.
 * On any error of a fresh dispatch the new handle is released again and
 *   *handle is left NULL (the layout may already be enqueued; its memory
 *   returns to the pool in stream order).
 * Debug check ([P4] "Performance Contract and Constraints": a layout is only
 *   valid for the table it came from): with EP_CHECK=1 in the environment,
 *   ep_get_dispatch_layout stores a 64-bit hash of topk_idx in the handle,
 *   and a dispatch given that handle together with a topk_idx hashes it and
 *   reads both hashes back (one stream synchronization); a different table
 *   returns EP_ERR_INVALID before anything is packed.
 * rank_mask [R] int32 (nullable): as for ep_get_dispatch_layout; used only
 *   by a fresh dispatch (the layout it computes).  A handle already holds
 *   its layout, so a non-NULL rank_mask with *handle != NULL returns
 *   EP_ERR_INVALID.
 * dims must equal the handle's dims except hidden, which may differ.
 */
int ep_dispatch(const ep_dims *dims, const void *x, const int64_t *topk_idx,
                const float *topk_weights, const int32_t *rank_mask, ep_handle **handle,
                void *recv_x, int64_t *recv_topk_idx, float *recv_topk_weights,
                int64_t recv_cap, int64_t *num_recv, ep_stream_t stream);

/*
 * [P1] "Combine Operation": addition-based reduction of the packed rows
 * y [y_rows][hidden] (bf16, same segment layout as the dispatch that made
 * handle) back to token order:
 *   out[t] = bf16_rne( sum over ranks r ascending that t went to of
 *                      fp32(y[S[r] + send_head[t][r]])
 *                      + fp32(bias0[t]) + fp32(bias1[t]) ),
 *   fp32 accumulation starting at +0, in that order; a token that went
 *   nowhere gets the bias sum (+0 without bias).
 * bias0, bias1 [T][hidden] bf16 (each nullable): the optional bias terms of
 *   the same section, added after the rank sum, before the one rounding.
 * recv_topk_weights [y_rows][K] fp32 (nullable) and combined_topk_weights
 * [T][K] fp32 (nullable, needs the former): the same ascending-rank fp32 sum
 * of the per-row weights (the reduced weights combine returns).
 * rank_mask [R] int32 (nullable; [P1] "Dynamic Rank Masking"): ranks masked
 *   now (nonzero) are left out of both sums, as if t had not gone there;
 *   the order of the remaining terms is unchanged.
 * y_rows below N returns EP_ERR_CAPACITY (checked without synchronizing
 * when y_rows >= ep_max_recv_rows(), else N is read once per handle).
 */
int ep_combine(ep_handle *handle, int32_t hidden, const void *y, int64_t y_rows,
               const float *recv_topk_weights, const void *bias0, const void *bias1,
               const int32_t *rank_mask, void *out, float *combined_topk_weights,
               ep_stream_t stream);

/*
 * [P1] "IB-GDA Kernels", low_latency_dispatch: stream every valid (token,
 * slot) pair straight into its expert's receive area.  With epr = E/R:
 *   packed_x  [epr][R][num_slots][H] bf16: cell (le, r, s) gets x[t] for the
 *             pair (t, k) naming expert r*epr + le whose slot is s
 *   packed_count [epr][R] int32: pairs routed to each expert
 *   src_info  [epr][R][num_slots] int32: source token of each used cell, -1
 *             for unused cells
 *   topk_slot [T][K] int32: slot s of pair (t, k), -1 when masked or dropped
 * Slots follow (token, slot) order.  Requires T <= num_slots
 * (EP_ERR_CAPACITY); pairs past num_slots (possible only when a token names
 * one expert twice) are dropped and still counted.  Unused packed_x cells
 * are not written.  packed_x may be NULL (metadata only).  No host sync.
 * rank_mask [R] int32 (nullable; [P1] "Dynamic Rank Masking"): nonzero
 *   marks a masked rank, whose experts receive nothing (count 0, no slots;
 *   their pairs get topk_slot -1), as if those slots were masked.
 */
int ep_ll_dispatch(const ep_dims *dims, int32_t num_slots, const void *x,
                   const int64_t *topk_idx, const int32_t *rank_mask, void *packed_x,
                   int32_t *packed_count, int32_t *src_info, int32_t *topk_slot,
                   ep_stream_t stream);

/*
 * ep_ll_dispatch with an FP8 payload ([P1] "IB-GDA Kernels": FP8 with
 * use_fp8, which the pages' code example sets on the dispatch).  Slots,
 * counts, src_info and topk_slot are exactly those of ep_ll_dispatch.
 * Every sent row is cut into 128-element blocks; per block
 *   amax = max(max |x|, 1e-4), q = e4m3(x * (448 / amax)), scale = amax / 448
 * in fp32, e4m3 being OCP FP8 E4M3 ("e4m3fn") with round to nearest even,
 * saturating at +-448.  x ~ q * scale.
 *   packed_q     [E/R][R][num_slots][H]     uint8 codes (8-byte aligned)
 *   packed_scale [E/R][R][num_slots][H/128] fp32
 * Requires hidden % 128 == 0 (EP_ERR_ALIGN).  Unused cells are not written.
 */
int ep_ll_dispatch_fp8(const ep_dims *dims, int32_t num_slots, const void *x,
                       const int64_t *topk_idx, const int32_t *rank_mask, void *packed_q,
                       float *packed_scale, int32_t *packed_count, int32_t *src_info,
                       int32_t *topk_slot, ep_stream_t stream);

/*
 * [P1] "IB-GDA Kernels", low_latency_combine: for every token,
 *   out[t] = bf16_rne(acc),  acc = fma(topk_weights[t][k], fp32(cell(t, k)), acc)
 * over k ascending, valid non-dropped slots only, from acc = +0, where cell
 * (t, k) is the packed_y row [le][r][topk_slot[t][k]] of the slot's expert.
 * packed_y has packed_x's layout; topk_slot comes from ep_ll_dispatch.
 * rank_mask [R] (nullable): pairs whose expert sits on a rank masked now
 * contribute nothing, whatever the dispatch did.  No host sync.
 */
int ep_ll_combine(const ep_dims *dims, int32_t num_slots, const void *packed_y,
                  const int64_t *topk_idx, const float *topk_weights,
                  const int32_t *topk_slot, const int32_t *rank_mask, void *out,
                  ep_stream_t stream);

/*
 * ep_ll_combine with an FP8 payload, the layout ep_ll_dispatch_fp8 writes
 * ([P1] "IB-GDA Kernels", FP8 with use_fp8; reading: the scales are applied
 * in the combine).  For every element of a cell:
 *   v = e4m3_decode(code) * scale[block]      (exact decode, one fp32 multiply)
 * then exactly the weighted sum of ep_ll_combine:
 *   out[t] = bf16_rne(acc),  acc = fma(topk_weights[t][k], v(cell(t, k)), acc)
 * over k ascending, valid non-dropped slots, from acc = +0.
 *   packed_q     [epr][R][num_slots][H] e4m3 codes (bytes), 8-byte aligned
 *   packed_scale [epr][R][num_slots][H/128] fp32
 * hidden must be a multiple of 128 (EP_ERR_ALIGN).  A NaN code gives NaN
 * terms.  rank_mask as for ep_ll_combine.  No host sync.
 */
int ep_ll_combine_fp8(const ep_dims *dims, int32_t num_slots, const void *packed_q,
                      const float *packed_scale, const int64_t *topk_idx,
                      const float *topk_weights, const int32_t *topk_slot,
                      const int32_t *rank_mask, void *out, ep_stream_t stream);

/* [P1] "Dynamic Rank Masking" on a caller-owned device mask rank_mask[R]
 * (0 active, 1 masked), stream-ordered like the other calls:
 *   ep_mask_update  set rank `rank` to masked (nonzero) or active (0)
 *   ep_mask_clean   set every rank active
 *   ep_mask_query   copy the mask to host_out[R] (HOST pointer); this call
 *                   synchronizes the stream. */
int ep_mask_update(int32_t *rank_mask, int32_t num_ranks, int32_t rank, int32_t masked,
                   ep_stream_t stream);
int ep_mask_clean(int32_t *rank_mask, int32_t num_ranks, ep_stream_t stream);
int ep_mask_query(const int32_t *rank_mask, int32_t num_ranks, int32_t *host_out,
                  ep_stream_t stream);

/*
 * Load balancing over redundant expert replicas ([P5] 10.2): replica j is a
 * copy of expert mapping[j] (mapping: int64 [num_replicas], device; entries
 * outside [0, num_experts) are ignored).  Tensors are bf16, one row of
 * elems_per_expert elements per expert / replica (elems % 8 == 0, 16-byte
 * aligned rows).
 *   ep_lb_prefetch_weights: redundant[j] = expert[mapping[j]] (bit copy).
 *   ep_lb_reduce_grads: for every expert e with replicas,
 *     expert[e] = bf16_rne(fp32(expert[e]) + sum over j ascending with
 *                          mapping[j] == e of fp32(redundant[j])),
 *     in place; experts without replicas are untouched.
 * num_replicas <= 65535.  No host sync.
 */
int ep_lb_prefetch_weights(const void *expert_weights, void *redundant_weights,
                           const int64_t *mapping, int32_t num_replicas, int32_t num_experts,
                           int64_t elems_per_expert, ep_stream_t stream);
int ep_lb_reduce_grads(const void *redundant_grads, void *expert_grads, const int64_t *mapping,
                       int32_t num_replicas, int32_t num_experts, int64_t elems_per_expert,
                       ep_stream_t stream);

/*
 * Root-mean-square norm of token rows, in front of the routing:
 *   s = fp32(x) + fp32(residual),  rstd = 1 / sqrt(mean(s^2) + eps),  y = s * rstd * weight
 *   residual_out = bf16_rne(s),  out = bf16_rne(y)
 *   out_q, out_scale: y in the FP8 format of ep_ll_dispatch_fp8 (e4m3 codes, one
 *     fp32 scale per 128 elements), quantised from the fp32 y.
 * x, residual, residual_out, out [num_tokens][hidden] bf16, weight [hidden] bf16,
 * out_q [num_tokens][hidden] (8-byte aligned), out_scale [num_tokens][hidden/128],
 * rstd [num_tokens] fp32.  residual, out, out_q and rstd are nullable (out or
 * out_q is required); residual_out needs residual and may be the same memory as
 * residual or x.  out_q needs hidden % 128 == 0 (EP_ERR_ALIGN) and out_scale.
 * eps must be finite and not negative.  No host sync.
 */
int ep_rms_norm(int32_t num_tokens, int32_t hidden, float eps, const void *x,
                const void *residual, const void *weight, void *residual_out, void *out,
                void *out_q, float *out_scale, float *rstd, ep_stream_t stream);

/*
 * Gradients of ep_rms_norm at the normed rows h (its residual_out, or x
 * without a residual) and the rstd it returned:
 *   a = dout * weight,  xh = h * rstd
 *   dx = bf16_rne(rstd * (a - xh * mean(a * xh)) + dresidual)
 *   dweight = sum over tokens of dout * xh   (fp32, in a fixed order)
 * dx is the gradient of x and of residual alike; dresidual (nullable) is the
 * gradient that arrived at residual_out.  dweight [hidden] fp32 is overwritten
 * (zeros without tokens).  workspace: ep_rms_norm_backward_workspace() bytes,
 * 16-byte aligned, the caller's (EP_ERR_CAPACITY if workspace_bytes is less).
 */
size_t ep_rms_norm_backward_workspace(int32_t num_tokens, int32_t hidden);
int ep_rms_norm_backward(int32_t num_tokens, int32_t hidden, const void *dout, const void *h,
                         const void *weight, const float *rstd, const void *dresidual, void *dx,
                         float *dweight, void *workspace, size_t workspace_bytes,
                         ep_stream_t stream);

/*
 * Product of FP8 rows with an FP8 weight, one fp32 scale per 128 inner
 * elements of a row and per 128 x 128 block of the weight:
 *   out[m][n] = bf16_rne( sum_b a_scale[m][b] * w_scale[n / 128][b]
 *                         * sum_{k in block b} a[m][k] * w[n][k] )
 * The scaled blocks are summed in fp32.  Inside a block the FP8 matrix instruction
 * adds the products of each eight neighbouring k (8 i .. 8 i + 7) after aligning them
 * to the largest of the eight, 2^E, and drops their bits below 2^(E - 13): each of the
 * other seven can lose up to 2^-13 of the largest.  The eights are summed in fp32.
 * a_q [m][k] and w_q [n][k] e4m3 codes, 16-byte aligned; a_scale [m][k/128],
 * w_scale [ceil(n/128)][k/128]; out [m][n] bf16.  k % 128 == 0 and n % 8 == 0
 * (EP_ERR_ALIGN), k and n at most 2^20.  No host sync.
 */
int ep_fp8_product(int32_t m, int32_t n, int32_t k, const void *a_q, const float *a_scale,
                   const void *w_q, const float *w_scale, void *out, ep_stream_t stream);

/*
 * The experts' gated feed-forward on low-latency cells (packed_x and
 * packed_count as ep_ll_dispatch left them).  For a used cell with row x of
 * expert e, and I = inter:
 *   g = x Wg^T,  u = x Wu^T,  act = g * sigmoid(g) * u,  out = act W2^T
 * w13 [E][2 I][H] bf16 holds expert e's Wg rows, then its Wu rows; w2 [E][H][I]
 * bf16; E is indexed by the expert id (r * E/R + le for cell block [le][r]).
 * act [E/R][R][num_slots][I] bf16 is workspace; the activation is rounded to
 * bf16 between the products (fp32 sums in both).  out has packed_x's layout;
 * unused cells are neither read nor written.  Counts above num_slots are taken
 * as num_slots.  num_tokens and num_topk bound the used cells: the counts must
 * add up to at most num_tokens * num_topk (experts past that are left out).
 * inter % 8 == 0 (EP_ERR_ALIGN).  No host sync.
 */
int ep_ll_expert_ffn(const ep_dims *dims, int32_t num_slots, int32_t inter, const void *packed_x,
                     const int32_t *packed_count, const void *w13, const void *w2, void *act,
                     void *out, ep_stream_t stream);

/*
 * ep_ll_expert_ffn on the cells of ep_ll_dispatch_fp8 with FP8 weights (one
 * scale per 128 x 128 block: w13_scale [E][2 I/128][H/128], w2_scale
 * [E][H/128][I/128]).  Between the products the activation is quantised, from
 * its fp32 value, in the same format: act_q [E/R][R][num_slots][I] codes and
 * act_scale [..][I/128] are workspace.  The down product sums as ep_fp8_product does.
 * The gate and up products of few activations (num_tokens * num_topk * inter below
 * 2^17) are fp32 sums of exact products; those of more may be either, as their
 * kernels go by the batch's shape.  So an activation near a rounding border of its
 * code can get the neighbouring code in a batch of another size; in every batch it is
 * the code of a value within that sum's bound of the exact one.  out is bf16.
 * hidden % 128 == 0 and inter % 128 == 0 (EP_ERR_ALIGN).
 */
int ep_ll_expert_ffn_fp8(const ep_dims *dims, int32_t num_slots, int32_t inter,
                         const void *packed_q, const float *packed_scale,
                         const int32_t *packed_count, const void *w13_q, const float *w13_scale,
                         const void *w2_q, const float *w2_scale, void *act_q, float *act_scale,
                         void *out, ep_stream_t stream);

/*
 * Dispatched rows grouped by expert.  A pair is a valid slot of a row:
 * recv_topk_idx[row][k] in [0, E/R), row in segment r as rank_prefix (the
 * layout's rank_prefix_matrix) has it; its expert is r * E/R + the id.  Rows at
 * or past rank_prefix[R-1] hold no pairs, whatever their ids.  Pairs are sorted
 * by (expert, row, slot).
 *   recv_topk_idx  int64 [num_rows][K]
 *   expert_offsets int32 [E + 1]   expert e's pairs are [e], ..., [e + 1] - 1
 *   pair_row       int32 [pair_cap] row of the pair; the sign bit is set when it
 *                                   is the only pair of its row
 *   pair_slot      int32 [pair_cap] row * K + slot
 *   row_pair       int32 [num_rows][K] the slot's pair, -1 if none
 *   counts         int32 [E] workspace (the pairs of each expert)
 * pair_cap must be at least min(num_tokens, num_rows) * K (EP_ERR_CAPACITY): a
 * dispatch gives each of its num_tokens * K slots to one row.  Pairs past it
 * are left out.  num_rows * K and pair_cap at most 2^31 - 1.  No host sync.
 */
int ep_expert_rows(const ep_dims *dims, const int32_t *rank_prefix, const int64_t *recv_topk_idx,
                   int64_t num_rows, int64_t pair_cap, int32_t *counts, int32_t *expert_offsets,
                   int32_t *pair_row, int32_t *pair_slot, int32_t *row_pair, ep_stream_t stream);

/* What ep_expert_rows wrote, for the calls below. */
typedef struct ep_expert_groups {
    int64_t num_rows;
    int64_t pair_cap;
    const int32_t *expert_offsets;
    const int32_t *pair_row;
    const int32_t *pair_slot;
    const int32_t *row_pair;
} ep_expert_groups;

/*
 * The experts between ep_dispatch and ep_combine: for every row of x
 * [num_rows][hidden] (bf16, packed rows)
 *   y[row] = bf16_rne( sum over its pairs, slot ascending, of
 *                      topk_weights[row][slot] * (act W2^T) ),  act as above,
 * a row without pairs giving +0.  topk_weights fp32 [num_rows][K], w13 and w2
 * as for ep_ll_expert_ffn.  Workspaces: act [pair_cap][inter] bf16, terms
 * [pair_cap][hidden] fp32 (16-byte aligned).  gate_up [pair_cap][2 inter] fp32
 * (nullable) receives g and u, which the backward pass needs.  Of dims, the
 * tokens and channels are not used.  inter % 8 == 0 (EP_ERR_ALIGN).
 */
int ep_expert_ffn(const ep_dims *dims, int32_t inter, const ep_expert_groups *groups,
                  const void *x, const float *topk_weights, const void *w13, const void *w2,
                  void *act, float *gate_up, float *terms, void *y, ep_stream_t stream);

/*
 * Gradients of ep_expert_ffn given dy [num_rows][hidden] bf16:
 *   dx [num_rows][hidden] bf16 (+0 for rows without pairs), dtopk_weights
 *   [num_rows][K] fp32 (0 for slots without a pair), dw13 [E][2 inter][hidden]
 *   and dw2 [E][hidden][inter] bf16 (zeros for experts without pairs), each
 *   overwritten.  All sums are fp32 in a fixed order.
 * Workspaces: dgate_up [pair_cap][2 inter] bf16, act [pair_cap][inter] bf16,
 * terms [pair_cap][hidden] fp32, parts [pair_cap][ceil(inter / 256)] fp32.
 */
int ep_expert_ffn_backward(const ep_dims *dims, int32_t inter, const ep_expert_groups *groups,
                           const void *dy, const void *x, const float *topk_weights,
                           const void *w13, const void *w2, const float *gate_up, void *dgate_up,
                           void *act, float *terms, float *parts, void *dx, float *dtopk_weights,
                           void *dw13, void *dw2, ep_stream_t stream);

/*
 * The router: the experts of each token and their weights, from its logits l[e].
 *   s = softmax(l) over all E experts, or sigmoid(l)
 *   key[e] = s[e] + bias[e]; without a bias key[e] = l[e] (s grows with l)
 *   with groups of E / num_groups neighbouring experts, the topk_groups groups of the
 *   largest scores stay: a group's score is its largest key, with a bias the sum of
 *   its two largest (of its largest alone where there is no second)
 *   topk_idx[t]: the K largest keys left, largest first; equal keys (and groups) go to the lowest index
 *   weight of a chosen expert: scale * s, or with normalize
 *     softmax: scale * the softmax over the chosen logits alone
 *     sigmoid: scale * s / (the chosen ones' sum + 1e-20)
 * An expert whose logit is -inf or NaN, or whose rank is masked, is not chosen.  Slots for which
 * nothing is left get -1 and weight 0.  The choice is that of exact keys: gaps within fp32 rounding are
 * decided in 64 bits.  Weights are fp32.  Scores are not changed by the mask.  A row of
 * -inf alone has scores 0.  A softmax row with +inf or NaN has NaN for scores: with a bias it has no keys
 * and nothing is chosen, without one its weights are NaN, but normalised ones, which are of the chosen logits
 * alone, only where +inf is among those.  A NaN logit makes all of its row's part of the score sums NaN.
 */
#define EP_SCORE_SOFTMAX 0
#define EP_SCORE_SIGMOID 1
typedef struct ep_router {
    int32_t score;       /* EP_SCORE_SOFTMAX or EP_SCORE_SIGMOID */
    int32_t num_groups;  /* 1 to 64, divides E; 1: no groups */
    int32_t topk_groups; /* 1 to num_groups */
    int32_t normalize;   /* nonzero: weights are divided by the chosen ones' sum */
    float scale;         /* finite */
} ep_router;

/*
 * Routes logits [num_tokens][E], fp32 or (logits_bf16 nonzero) bf16.  Of dims, the hidden
 * size and channels are not used.  bias fp32 [E] and rank_mask int32 [R] are nullable.
 *   topk_idx     int64 [num_tokens][K], topk_weights fp32 [num_tokens][K]
 *   score_sums   fp32 [E], nullable: sum over tokens of p, p = s for softmax and s / sum(s)
 *                for sigmoid scores (in a fixed order): with the tokens' counts, what a balancing
 *                loss is made of.  It needs workspace, ep_route_workspace() bytes
 *                (EP_ERR_CAPACITY if workspace_bytes is less).
 * No host sync.
 */
size_t ep_route_workspace(const ep_dims *dims);
int ep_route(const ep_dims *dims, const ep_router *router, const void *logits, int32_t logits_bf16,
             const float *bias, const int32_t *rank_mask, int64_t *topk_idx, float *topk_weights,
             float *score_sums, void *workspace, size_t workspace_bytes, ep_stream_t stream);

/*
 * Gradient of ep_route: dlogits [num_tokens][E], of the logits' type, overwritten, given the gradients
 * of topk_weights [num_tokens][K] fp32 and (nullable) of score_sums [E] fp32.  topk_idx is what
 * ep_route wrote (ids outside [0, E) are taken as -1); the choice itself has no gradient.
 * The weights' sums are those of ep_route.  No host sync.
 */
int ep_route_backward(const ep_dims *dims, const ep_router *router, const float *dtopk_weights,
                      const void *logits, int32_t logits_bf16, const int64_t *topk_idx,
                      const float *dscore_sums, void *dlogits, ep_stream_t stream);

/*
 * A whole mixture-of-experts layer for a few tokens: router, experts and combine in one call, no rows
 * packed in between.
 *   logits[t][e] = fp32(x[t] . w_router[e]), summed in 64 bits, in one order for every num_tokens
 *   topk_idx, topk_weights as ep_route gives them for these logits
 *   y[t] = bf16_rne( residual[t] + sum over its experts, fp32, of weight * (act W2^T) ), act as for
 *          ep_ll_expert_ffn, kept to 2^-16 of itself between the products beside bf16 weights and
 *          rounded to bf16 beside FP8 ones (an infinite W2 gives infinities or NaN)
 * x, residual (nullable), y [num_tokens][hidden] bf16; y may be the same memory as residual, not as x.
 * w_router [E][hidden] bf16, or fp32 with w_router_fp32 nonzero.  bias [E], rank_mask [R] nullable.
 * w13 [E][2 inter][hidden], w2 [E][hidden][inter]: bf16, or with w13_scale and w2_scale (both or neither)
 * FP8 codes and scales as for ep_ll_expert_ffn_fp8.  Beside FP8 weights too, x and
 * act are bf16: every product is exact and summed in fp32, the scales applied once per 128 of K.
 * A token's experts and weights do not depend on the batch it comes in; y's rounding can, as the batch decides how
 * its sums are split.
 * num_tokens <= 64 and E <= 512 (EP_ERR_TOO_LARGE); hidden % 8 == 0 and inter % 8 == 0, with FP8
 * % 128 (EP_ERR_ALIGN).  workspace: ep_ll_moe_workspace() bytes, 256-byte aligned
 * (EP_ERR_CAPACITY if workspace_bytes is less).  No host sync.
 */
size_t ep_ll_moe_workspace(const ep_dims *dims, int32_t inter);
int ep_ll_moe(const ep_dims *dims, int32_t inter, const ep_router *router, const void *x, const void *w_router,
              int32_t w_router_fp32, const float *bias, const int32_t *rank_mask, const void *w13,
              const float *w13_scale, const void *w2, const float *w2_scale, const void *residual,
              int64_t *topk_idx, float *topk_weights, void *y, void *workspace, size_t workspace_bytes,
              ep_stream_t stream);

/*
 * Low-rank adapters of many requests beside a shared projection (ep_fp8_product's, or any other): token t
 * uses adapter a = adapter_ids[t], none if that is outside [0, num_adapters).
 *   h[t] = scales[a] * (x[t] down_a^T),  out[t] = bf16_rne( base[t] + h[t] up_a^T )
 * with fp32 sums and h kept to 2^-16 of itself (an infinite up gives infinities or NaN); a token without an adapter gets base[t] (zeros without a base).
 *   x [T][in] bf16, adapter_ids int64 [T], down [L][rank][in], up [L][out][rank] bf16, scales fp32 [L]
 *   base [T][out] bf16, nullable; out [T][out] may be the same memory as base
 *   hidden [2][T][rank] bf16, nullable: h, which the backward pass takes, as the sum of its bf16 value
 *     and of what that rounding lost (zeros without an adapter)
 * The same call gives the same bits every time; a token's result can differ in its rounding with T and L, which
 * decide how the sums over in are split.  Past 256 tokens or 127 adapters the tokens are sorted by adapter first, in
 * a time that grows with T * L (8 us for 8192 tokens on 16 adapters, 15 on 1024, 0.2 ms for 131072 on 1024, 1.2 ms on 8192).
 * in, out and rank % 8 == 0 (EP_ERR_ALIGN), rank <= 128, L <= 8192.  workspace: ep_adapter_workspace(dims, 0)
 * bytes, 256-byte aligned (EP_ERR_CAPACITY if workspace_bytes is less; 0, so that it may be null, for a few
 * tokens).  No host sync.
 */
typedef struct ep_adapter_dims {
    int32_t num_tokens;   /* T */
    int32_t in_features;  /* x's width */
    int32_t out_features; /* out's width */
    int32_t rank;
    int32_t num_adapters; /* L */
} ep_adapter_dims;
size_t ep_adapter_workspace(const ep_adapter_dims *dims, int32_t backward);
int ep_adapter_product(const ep_adapter_dims *dims, const void *x, const int64_t *adapter_ids, const void *down,
                       const void *up, const float *scales, const void *base, void *out, void *hidden,
                       void *workspace, size_t workspace_bytes, ep_stream_t stream);

/*
 * Gradients of ep_adapter_product given dy [T][out] bf16 (base's gradient is dy itself; scales are constants):
 *   dh[t] = scales[a] * (dy[t] up_a),  dx[t] = bf16_rne( dx_base[t] + dh[t] down_a )
 *   ddown_a = bf16_rne( sum_t dh[t]^T x[t] ),  dup_a = bf16_rne( sum_t dy[t]^T h[t] ),  in a fixed order,
 * h and dh there to 2^-16 of themselves (an infinite dy or x gives infinities or NaN)
 * dx_base [T][in] (nullable) is the projection's own gradient of x; dx may be the same memory.  ddown and
 * dup are overwritten whole (zeros for adapters without tokens).  hidden is ep_adapter_product's.
 * num_adapters * (ceil(in / 64) + ceil(out / 64)) <= 2^27 (EP_ERR_INVALID past it: weights and gradients of
 * 275 GB and more).
 * workspace: ep_adapter_workspace(dims, 1) bytes.  No host sync.
 */
int ep_adapter_product_backward(const ep_adapter_dims *dims, const void *dy, const void *x,
                                const int64_t *adapter_ids, const void *down, const void *up,
                                const float *scales, const void *hidden, const void *dx_base, void *dx,
                                void *ddown, void *dup, void *workspace, size_t workspace_bytes,
                                ep_stream_t stream);

/* Copy the handle's layout into caller buffers (fields may be NULL); same
 * shapes and capacity rule as ep_get_dispatch_layout. */
int ep_handle_copy_layout(ep_handle *handle, ep_layout_out *out, ep_stream_t stream);

/* N of the handle.  The first time, waits for the handle's last stream to
 * reach the copy of N into pinned host memory (work enqueued after it may
 * still be running when the call returns); later calls use the cached value. */
int ep_handle_num_recv(ep_handle *handle, int64_t *num_recv);

/* The handle's dims (host copy). */
int ep_handle_dims(const ep_handle *handle, ep_dims *dims);

/* Device bytes the handle holds (the print_memory_usage of the pages' V2.5
 * buffer base class). */
size_t ep_handle_nbytes(const ep_handle *handle);

/* [P1] "Explicit Resource Cleanup": release a handle.  NULL is a no-op.  The
 * memory returns to the library's per-device pool, tagged with the handle's
 * last stream; only a later handle made on that same stream reuses it, so
 * stream order puts every use of the memory before its reuse.  Nothing is
 * enqueued.
 * The pool is capped per device: at most EP_POOL_CAP_MB MiB (environment,
 * read once; default 256) and 64 arenas.  A free that takes the pool past
 * either limit synchronizes the device once (the only case in which this
 * call waits), returns the oldest arenas to HIP until the pool holds at most
 * half the byte cap and 32 arenas, and makes the arenas it keeps reusable by
 * handles on any stream (they are idle after that synchronization). */
void ep_handle_free(ep_handle *handle);

/* Release every pooled device allocation of the calling thread's current
 * device (synchronizes the device first).  Returns an ep_status. */
int ep_pool_trim(void);

/* The calling thread's current device's pool: bytes and arenas it keeps for
 * reuse, and its byte cap (each pointer nullable; HOST pointers).  Returns an
 * ep_status. */
int ep_pool_stats(size_t *kept_bytes, int32_t *kept_arenas, size_t *cap_bytes);

/* Launch-shape override for the pack ("dispatch") or the reduce ("combine")
 * kernels, process-wide, for every later call.  Results never depend on it.
 * a = lanes per group G, b = 16-byte vectors per lane VPT, c = a code for
 * the rest: dispatch X*10000 + S*1000 + NTL*100 + NTS*10 + P/256, combine
 * X*10000 + S*1000 + U*100 + NTL*10 + P/256, where X = 1 for the
 * destination-major (scatter) pack (the default) and the gather-form reduce
 * (G threads per workgroup, one vector each),
 * S = lane groups per token (row slices), NTS/NTL = nontemporal
 * stores/loads, U = rows in flight and P = persistent block count (0 = one
 * lane group per token slice).  ep_tuning_list enumerates the compiled-in
 * shapes.  a = b = c = -1 restores the default choice; a shape
 * that is not compiled in returns EP_ERR_INVALID.  The env vars
 * EP_TUNE_DISPATCH="G,VPT,c" and EP_TUNE_COMBINE="G,VPT,c" set the initial
 * override.
 * op "ll" picks the low-latency dispatch kernels (b = c = 0): a = 0 automatic
 * (one launch when T*K <= 4096, else a per-expert slot scan followed by a
 * token-major row copy), 1 slot scan + copy always, 2 one launch whenever
 * T*K <= 4096.  Both give identical results.
 * op "layout" picks the layout kernels (b = c = 0), for handles made
 * afterwards: a = 0 automatic (= 1), 1 the count and position kernels (a
 * scan kernel between them past 16384 tokens), 2 one launch whenever it fits
 * (up to 8192 tokens; measured slower than two launches on gfx950, kept for
 * callers that count launches).  Identical results. */
int ep_set_tuning(const char *op, int a, int b, int c);

/* Enumerate the compiled-in shapes of `op`: writes shape `index` (if in
 * range) to a, b, c and returns how many there are (-1 for an unknown op). */
int ep_tuning_list(const char *op, int index, int *a, int *b, int *c);

/* Static text of a status code. */
const char *ep_status_str(int status);

/* Text of the last HIP error seen by this thread (empty if none). */
const char *ep_last_hip_error(void);

/* ABI version: (major << 16) | minor.  2.0: rank_mask arguments of
 * ep_get_dispatch_layout, ep_dispatch and ep_combine; 2.1: ep_ll_combine_fp8;
 * 2.2: ep_pool_stats and the capped pool; 2.3: ep_get_dispatch_layout_noalloc
 * and EP_ERR_TOO_LARGE; 2.4: the destination-major dispatch and gather-form
 * combine tuning shapes (code X*10000).  The expert operations (ep_rms_norm to
 * ep_expert_ffn_backward), the router (ep_route*), ep_ll_moe and the adapters (ep_adapter_*)
 * were added without a new number: look the symbol up. */
int ep_version(void);

#ifdef __cplusplus
}
#endif

#endif /* EP_H */
