// ep_internal.h -- declarations shared by the gfx950 kernels and the host
// runtime of libep.so.  Not part of the public ABI (that is include/ep.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ep.h"

namespace ep {

// 16-byte vector: the unit of every token-row load and store (rows are whole
// int4 vectors, as the runtime's alignment rule requires).
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWave = 64;          // CDNA wavefront width
constexpr int kMaxRanks = 512;     // NW <= 8 64-bit rank-mask words
constexpr int kMaxTopk = 64;
constexpr int kMaxExperts = 8192;  // per-block expert histogram lives in LDS
constexpr int kMaxChannels = 4096;
constexpr int kMaxLLSlots = 4096;  // slots per low-latency expert cell list
constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int kMaxHidden = 1 << 20;

// Device pointers of one layout (all inside a handle's arena).  The first
// kLayoutCtrBytes of every arena hold the one-launch layout's counters,
// zeroed when the arena is allocated and only ever increased after that.
constexpr int kArenaFields = 17;
constexpr size_t kLayoutCtrBytes = 256;
struct LayoutBufs {
    uint64_t *layout_ctr;                // [4] tickets, count units done, count blocks done, wait-timeout flag
    int32_t *num_tokens_per_rank;        // [R]
    int32_t *num_tokens_per_expert;      // [E]
    uint8_t *is_token_in_rank;           // [T][R]
    int32_t *rank_prefix_matrix;         // [R]
    int32_t *channel_prefix_matrix;      // [R][C]
    int32_t *recv_channel_prefix_matrix; // [R][C]
    int32_t *send_head;                  // [T][R]
    int32_t *recv_src_idx;               // [T*Kmax]
    int32_t *dst_row;                    // [T][Kmax] packed rows of t, ascending rank, -1 padded
    int32_t *dst_rank;                   // [T][Kmax] their ranks
    uint64_t *wave_mask;                 // [nW][R] ballot of "token hits r" per 64-token wave
    int32_t *wave_base;                  // [nW][R] hits of r in earlier waves of the same block
    int32_t *blk_count;                  // [nB][R] block totals (exclusive bases after a scan kernel)
    int32_t *blk_ecount;                 // [nB][E] per-block expert counts
    int64_t *num_recv;                   // [1] N
    uint64_t *topk_hash;                 // [2] hash of the layout's topk_idx, and of a later one
};

struct LayoutShape {
    int T, K, E, R, C, epr, kmax, nW, nB;
    bool fused;  // one-launch layout (count blocks of 256 tokens), else two kernels (512)
};

// allow_fused: the one-launch layout may be chosen (it needs the arena's
// counter bookkeeping, so only handle arenas allow it).
LayoutShape layout_shape(const ep_dims &d, bool allow_fused = true);
// Byte offsets of every LayoutBufs field inside one arena; returns the total.
size_t layout_arena_bytes(const LayoutShape &s, size_t off[kArenaFields]);
LayoutBufs layout_bufs_at(void *base, const size_t off[kArenaFields]);

// EP_LOG=1 in the environment: one line per kernel launch on stderr with its
// launch geometry (read at every call).
bool log_enabled();
void log_launch(const char *fmt, ...) __attribute__((format(printf, 1, 2)));

// How far an arena's one-launch layout counters have advanced: the tickets
// and done marks of every layout launched in it so far (host-side, kept with
// the arena; stream order makes each launch start where the last one ended).
struct LayoutCounters {
    uint64_t tickets = 0;
    uint64_t done = 0;
    uint64_t counted = 0;  // count blocks that summed into the early N
};

// rank_mask [R] int32 (nullable): nonzero ranks are masked.  num_recv_host
// (nullable): pinned, coherent host memory that also receives N, exactly
// once, so that a caller waiting for N can poll it instead of copying it
// back.  On the two-kernel path the count kernel's last block stores it, as
// soon as the counts are known and before the positions are.
hipError_t launch_layout(const LayoutShape &s, const int64_t *topk_idx, const int32_t *rank_mask,
                         const LayoutBufs &b, int64_t *num_recv_host, LayoutCounters &lc,
                         hipStream_t stream);

hipError_t launch_dispatch(const LayoutShape &s, int hidden, const void *x, const LayoutBufs &b,
                           const int64_t *topk_idx, const float *topk_weights, void *recv_x,
                           int64_t *recv_topk_idx, float *recv_topk_weights, hipStream_t stream);

hipError_t launch_combine(const LayoutShape &s, int hidden, const void *y, const LayoutBufs &b,
                          const float *recv_topk_weights, const void *bias0, const void *bias1,
                          const int32_t *rank_mask, void *out, float *combined_topk_weights,
                          hipStream_t stream);

// packed_q (nullable) selects the FP8 variant: codes [cells][H] bytes and
// packed_scale [cells][H/128]; packed_x is then unused.
hipError_t launch_ll_dispatch(const ep_dims &d, int num_slots, const void *x,
                              const int64_t *topk_idx, const int32_t *rank_mask, void *packed_x,
                              void *packed_q, float *packed_scale, int32_t *packed_count,
                              int32_t *src_info, int32_t *topk_slot, hipStream_t stream);

hipError_t launch_ll_combine(const ep_dims &d, int num_slots, const void *packed_y,
                             const int64_t *topk_idx, const float *topk_weights,
                             const int32_t *topk_slot, const int32_t *rank_mask, void *out,
                             hipStream_t stream);
// packed_q: e4m3 codes [cells][H] bytes, packed_scale [cells][H/128].
hipError_t launch_ll_combine_fp8(const ep_dims &d, int num_slots, const void *packed_q,
                                 const float *packed_scale, const int64_t *topk_idx,
                                 const float *topk_weights, const int32_t *topk_slot,
                                 const int32_t *rank_mask, void *out, hipStream_t stream);

// Order-independent 64-bit hash of n top-k ids into *out (debug check).
hipError_t launch_topk_hash(const int64_t *topk_idx, int64_t n, uint64_t *out, hipStream_t stream);

hipError_t launch_mask_set(int32_t *mask, int num_ranks, int rank, int value, hipStream_t stream);

hipError_t launch_lb_reduce_grads(const void *redundant_grads, void *expert_grads,
                                  const int64_t *mapping, int num_replicas, int num_experts,
                                  int64_t elems, hipStream_t stream);

hipError_t launch_lb_prefetch_weights(const void *expert_weights, void *redundant_weights,
                                      const int64_t *mapping, int num_replicas, int num_experts,
                                      int64_t elems, hipStream_t stream);

// ---------------------------------------------------------------- experts

// Rows grouped by expert (ep_expert_rows): pairs sorted by (expert, row, slot).
// pair_row's sign bit marks the only pair of its row.
struct ExpertFfn {
    int experts, hidden, inter, topk;
    int64_t rows;   // token rows
    int64_t pairs;  // capacity of the pair arrays
    const int32_t *offsets, *pair_row, *pair_slot, *row_pair;
    const float *weights;  // [rows][topk]
};

hipError_t launch_expert_rows(int E, int epr, int K, int64_t rows, const int32_t *prefix,
                              const int64_t *ids, int64_t cap, int32_t *counts, int32_t *offsets,
                              int32_t *pair_row, int32_t *pair_slot, int32_t *row_pair,
                              hipStream_t stream);

// Column tiles of the routing weight's partial gradients.
int expert_ffn_tiles(int inter);

hipError_t launch_expert_ffn(const ExpertFfn &f, const void *x, const void *w13, const void *w2,
                             void *act, float *gate_up, float *terms, void *y, hipStream_t stream);

hipError_t launch_expert_ffn_backward(const ExpertFfn &f, const void *dy, const void *x, const void *w13,
                                      const void *w2, const float *gate_up, void *dgu, void *wact,
                                      float *parts, float *terms, void *dx, float *dweight, void *dw13,
                                      void *dw2, hipStream_t stream);

hipError_t launch_ll_expert_ffn(int E, int R, int slots, int H, int I, int64_t max_pairs,
                                const int32_t *counts, const void *packed, const void *w13,
                                const void *w2, void *act, void *out, hipStream_t stream);

// FP8 operands: e4m3 codes, and fp32 scales [row][K/128] of the token rows and
// [ceil(N/128)][K/128] of a weight.
hipError_t launch_fp8_product(int64_t M, int N, int K, const void *a_q, const float *a_scale,
                              const void *w_q, const float *w_scale, void *out, hipStream_t stream);

hipError_t launch_ll_expert_ffn_fp8(int E, int R, int slots, int H, int I, int64_t max_pairs,
                                    const int32_t *counts, const void *packed_q,
                                    const float *packed_scale, const void *w13_q,
                                    const float *w13_scale, const void *w2_q, const float *w2_scale,
                                    void *act_q, float *act_scale, void *out, hipStream_t stream);

hipError_t launch_rms_norm(int64_t T, int H, float eps, const void *x, const void *residual,
                           const void *weight, void *residual_out, void *out, void *out_q,
                           float *out_scale, float *rstd, hipStream_t stream);

// Rows of fp32 partial sums of dweight that the backward pass writes.
int rms_norm_parts(int64_t T);

hipError_t launch_rms_norm_backward(int64_t T, int H, const void *dout, const void *h,
                                    const void *weight, const float *rstd, const void *dresidual,
                                    void *dx, float *dweight, float *parts, hipStream_t stream);

// out[c] = the sum of parts[0 .. n - 1][c], in a fixed order.
hipError_t launch_sum_parts(const float *parts, int n, int width, float *out, hipStream_t stream);

// ----------------------------------------------------------------- router

struct RouteRule;  // route.h

// Rows of fp32 partial score sums that the router writes.
int route_parts(int64_t T, int experts);

hipError_t launch_route(const RouteRule &rule, int64_t T, const void *logits, bool bf16, int64_t *topk_idx,
                        float *weights, float *score_sums, float *parts, hipStream_t stream);

hipError_t launch_route_backward(const RouteRule &rule, int64_t T, const float *dweights, const void *logits, bool bf16,
                                 const int64_t *topk_idx, const float *dsums, void *dlogits, hipStream_t stream);

// ------------------------------------------------------------ whole layer

constexpr int kMoeTokens = 64;    // a bit each in an expert's mask
constexpr int kMoeExperts = 512;  // what the router holds in one wave

struct MoeCall {
    int T, H, I;
    const void *x, *w_router, *w13, *w2, *residual;  // residual nullable
    bool router_f32;
    const float *w13_scale, *w2_scale;               // FP8 weights, else null
    int64_t *topk_idx;
    float *topk_weights;
    void *y, *workspace;
};
size_t moe_workspace(int T, int E, int K, int I);
hipError_t launch_moe(const RouteRule &rule, const MoeCall &call, hipStream_t stream);

// --------------------------------------------------------------- adapters

constexpr int kMaxRank = 128;
constexpr int kMaxAdapters = 8192;
constexpr int64_t kMaxGradBlocks = int64_t(1) << 27;  // of 64 columns of an adapter: at rank 8 weights and gradients of 275 GB

struct AdapterShape {
    int T, K, N, r, L;
    const int64_t *ids;   // [T]
    const float *scales;  // [L]
};
size_t adapter_workspace(const AdapterShape &s, bool back);
hipError_t launch_adapter(const AdapterShape &s, const void *x, const void *down, const void *up, const void *base, void *out,
                          void *hidden, void *workspace, hipStream_t stream);
hipError_t launch_adapter_backward(const AdapterShape &s, const void *dy, const void *x, const void *down, const void *up,
                                   const void *hidden, const void *dx_base, void *dx, void *ddown, void *dup, void *workspace,
                                   hipStream_t stream);

// A block for each row.  A dimension of a launch holds fewer than 2^32 threads,
// so rows past 2^20 go into y; the kernel drops the excess.
constexpr int64_t kRowGrid = int64_t(1) << 20;
inline dim3 row_grid(int64_t rows)
{
    return rows <= kRowGrid ? dim3(unsigned(rows))
                            : dim3(unsigned(kRowGrid), unsigned((rows + kRowGrid - 1) / kRowGrid));
}
// Blocks of one launch of a 512-thread kernel (the same limit).
constexpr int64_t kMaxTileBlocks = int64_t(1) << 22;

// Compute units of the current device, in whole rounds of its XCDs: the blocks of
// a launch whose blocks each fill one and work through tiles.
int compute_units();

// Row tile of the tile kernels.  A 256-row tile reads a group's weight once for
// up to 256 rows and shortens its last tile to what is there.  64-row tiles
// where a group has no more rows on average (their third LDS stage hides more
// of the weight's latency; 64 experts of 51 rows, 352 x 256: 11.1 against 15.0 us),
// or where the larger ones, which take 2.5 times as long, leave half of the card
// idle (FP8, K = 2048: 1500 x 4096, 96 tiles, 30.7 against 35.0 us; 3000 x 4096, 208
// tiles, 46.2 against 38.1).
inline int tile_rows(int64_t rows, int64_t groups, int64_t column_tiles)
{
    groups = groups > 0 ? groups : 1;
    return rows / groups > 64 && (rows / 256 + groups) * column_tiles * 2 > compute_units() ? 256 : 64;
}

// Row tiles of one launch: every group can end in a part tile, and no more tiles than
// rows exist.
inline int64_t row_tiles(int64_t rows, int64_t groups, int height)
{
    return rows / height + (groups < rows ? groups : rows);
}
// The most tiles that the rule above can give.  Where it takes 64 rows because 256
// would leave the card idle there are less than four times the card's compute units;
// kLeast stands for those.
inline int64_t tiles_at_most(int64_t rows, int64_t groups, int64_t column_tiles)
{
    constexpr int64_t kLeast = 1 << 16;
    groups = groups > 0 ? groups : 1;
    const int64_t n = (rows / (rows / groups > 64 ? 256 : 64) + groups) * column_tiles;
    return n > kLeast ? n : kLeast;
}

// Shared with the entry points outside ep_api.hip.
int api_hip_error(hipError_t e);
void api_trace_push(const char *name);
void api_trace_pop();

// Launch-shape overrides (never change results).  (-1, ...) restores the
// default choice.  Return false for a shape that is not compiled in.
bool set_dispatch_tuning(int g, int vpt, int code);
bool set_combine_tuning(int g, int vpt, int u);
// Low-latency dispatch variant: 0 automatic (one launch for T*K <= 4096,
// else slot scan + token-major copy), 1 slot scan + copy always, 2 one
// launch whenever T*K allows.
bool set_ll_tuning(int mode);
// Layout: 0 automatic (the count and position kernels), 1 those kernels
// always, 2 one launch whenever it fits (up to 8192 tokens).  Read when a
// handle is made.
bool set_layout_tuning(int mode);
int dispatch_tuning_count();
void dispatch_tuning_at(int i, int *g, int *vpt, int *code);
int combine_tuning_count();
void combine_tuning_at(int i, int *g, int *vpt, int *u);

// ---------------------------------------------------------------- device helpers

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// fp32 -> bf16 round to nearest, ties to even: add just under half of the
// dropped 16-bit fraction, plus one when the kept lsb is odd, then truncate.
// A mantissa carry correctly bumps the exponent.  NaN is kept quiet.
__device__ __forceinline__ uint32_t bf16_rne(float f)
{
    uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u)
        return (u >> 16) | 0x40u;
    return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    return bf16_rne(lo) | (bf16_rne(hi) << 16);
}

// The same rounding in one instruction (a NaN may come out with other payload
// bits): for results of arithmetic, where the copies' bit rule does not apply.
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi)
{
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}

__device__ __forceinline__ uint64_t wave_ballot(bool p) { return __ballot(p); }

__device__ __forceinline__ uint64_t lanemask_lt()
{
    const unsigned lane = __lane_id();
    return lane == 0 ? 0ull : (~0ull >> (64 - lane));
}

}  // namespace ep
