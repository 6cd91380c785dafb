// gemm.h -- the matrix-core tile loop that the expert products share (bf16 and
// FP8 block-scaled), for gfx950.  Device code; included by experts.hip and
// fp8.hip.
//
// A tile computes D[n, m] = sum_k P[n, k] Q[m, k]: P is the operand whose
// index runs along the output's rows of memory (a weight's output column),
// Q the operand whose index picks the output row (a token).  P is the
// matrix instruction's first operand, so a lane ends with four consecutive n
// of one m and stores them as one vector.
//
// Each operand lies in memory in one of two ways:
//   Row  k is contiguous (a token row, a weight [n][k]).
//   Col  the operand's own index is contiguous and k picks the row (a weight
//        used transposed, or both operands of a weight gradient).  Its
//        fragments come out of LDS through the transposing read.
//
// Both are staged by the loads that write LDS directly, 16 bytes a lane, in
// K steps of 128 bytes (64 bf16 or 128 FP8 values).  LDS is written in lane
// order, so the bank swizzle is applied to the global address instead.
#pragma once

#include "ep_internal.h"

namespace ep {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

typedef __attribute__((address_space(3))) char lds_char;

// 16 zero bytes: what a lane reads in place of a value past the end of K, so
// that a tail adds exact zeros whatever lies behind a row (a NaN included).
static __device__ __attribute__((aligned(16))) const unsigned int kZero16[4] = {0, 0, 0, 0};

// 16 (or 4) bytes a lane from src to dst + 16 (4) * lane, dst the same for the
// whole wave.  In assembly because the compiler, which cannot tell the LDS
// stages apart, makes every later LDS read wait for the loads in flight: that
// is the overlap the stages are for.  The instruction has no destination
// register; landed() is its wait, always before the barrier that publishes a stage.
// M0 is set inside the block, and nothing else in these kernels uses it.
__device__ __forceinline__ uint32_t lds_at(const lds_char *p)
{
    return uint32_t(__builtin_amdgcn_readfirstlane(int(uint32_t(reinterpret_cast<uintptr_t>(p)))));
}
__device__ __forceinline__ void load_lds16(const char *src, lds_char *dst)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(src), "s"(lds_at(dst))
                 : "memory");
}
__device__ __forceinline__ void load_lds4(const char *src, lds_char *dst)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
                 :
                 : "v"(src), "s"(lds_at(dst))
                 : "memory");
}
// Every load of this wave but the last N has landed.
template <int N>
__device__ __forceinline__ void landed()
{
    static_assert(N >= 0 && N < 64, "vmcnt has six bits");
    asm volatile("s_waitcnt vmcnt(%0)" : : "i"(N) : "memory");
}

constexpr int kStepBytes = 128;  // K bytes of one stage

// Row-contiguous operand, ROWS rows staged by NT threads.  LDS row r holds its
// eight 16-byte chunks at position c ^ ((r >> 1) & 7): sixteen consecutive
// rows read at one chunk then fall on sixteen different 16-byte bank groups.
template <int ROWS, int NT>
struct RowStage {
    static constexpr int J = ROWS * 8 / NT;
    static constexpr int kBytes = ROWS * kStepBytes;
    const char *ptr[J];
    int cb[J];  // byte of the chunk inside the K step

    // row_ptr(r): the address of LDS row r at k = 0 (any valid row for rows
    // past the end: their results are never stored).
    template <class F>
    __device__ __forceinline__ void init(int tid, F row_ptr)
    {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int q = j * NT + tid;
            const int r = q >> 3;
            cb[j] = ((q & 7) ^ ((r >> 1) & 7)) * 16;
            ptr[j] = row_ptr(r) + cb[j];
        }
    }
    // Stage K bytes [kb, kb + 128); kbytes: all K bytes of the operand.
    __device__ __forceinline__ void issue(lds_char *base, int wave, int64_t kb, int64_t kbytes)
    {
        const bool whole = kb + kStepBytes <= kbytes;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const char *p = ptr[j] + kb;
            if (!whole && kb + cb[j] >= kbytes)
                p = reinterpret_cast<const char *>(kZero16);
            load_lds16(p, base + (j * NT + wave * kWave) * 16);
        }
    }
    // Chunk ch (0..7) of LDS row r.
    static __device__ __forceinline__ const lds_char *at(const lds_char *base, int r, int ch)
    {
        return base + r * kStepBytes + ((ch ^ ((r >> 1) & 7)) << 4);
    }
};

// Operand with its own index contiguous: 64 k rows of COLS bf16.  Chunk c of
// k row r lies at c ^ 2 g(r), g(r) = (r & 3) | ((r >> 3) & 1) << 2: the
// sixteen 32-byte runs that one transposing read touches then spread over
// eight bank groups, which is all of them.
template <int COLS, int NT>
struct ColStage {
    static constexpr int CH = COLS / 8;  // 16-byte chunks of a k row
    static constexpr int J = 64 * CH / NT;
    static constexpr int kBytes = 64 * COLS * 2;
    int k[J];   // k row inside the step
    int cb[J];  // byte of the (clamped) column inside a row of memory

    static __device__ __forceinline__ int g2(int r) { return ((r & 3) | (((r >> 3) & 1) << 2)) << 1; }

    // n0: first column of the tile, n: columns of the operand (a multiple of 8)
    __device__ __forceinline__ void init(int tid, int n0, int n)
    {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int q = j * NT + tid;
            k[j] = q / CH;
            int c = n0 + ((q % CH) ^ g2(k[j])) * 8;
            c = c < n ? c : n - 8;
            cb[j] = c * 2;
        }
    }
    // row_ptr(j, k): address of memory row k (k < kn), for this thread's j-th chunk
    template <class F>
    __device__ __forceinline__ void issue(lds_char *base, int wave, int k0, int kn, F row_ptr)
    {
        const bool whole = k0 + 64 <= kn;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const char *p;
            if (whole || k0 + k[j] < kn)
                p = row_ptr(j, k0 + k[j]) + cb[j];
            else
                p = reinterpret_cast<const char *>(kZero16);
            load_lds16(p, base + (j * NT + wave * kWave) * 16);
        }
    }
    // Fragment of 16 columns from c0 and the 32 k values of half ks: lane l
    // gets column c0 + l % 16, k = ks * 32 + (l / 16) * 8 .. + 7.
    static __device__ __forceinline__ bf16x8 frag(const lds_char *base, int c0, int ks, int lane)
    {
        const int i = lane & 15, b = lane >> 4;
        const int kr = ks * 32 + b * 8 + (i >> 2);  // and + 4 for the second read
        const int ch = (c0 >> 3) + ((i >> 1) & 1);
        const lds_char *p0 = base + kr * (COLS * 2) + ((ch ^ g2(kr)) << 4) + ((i & 1) << 3);
        const lds_char *p1 = p0 + 4 * (COLS * 2);
        s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4 *)p0);
        s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4 *)p1);
        s16x8 r = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf16x8, r);
    }
};

constexpr int NT = 512;  // threads of a tile block: 8 waves, 2 (tokens) x 4 (columns)
constexpr int BN = 256;  // columns of a tile
constexpr int kNoLimit = 0x7fffffff;
constexpr int32_t kRowMask = 0x7fffffff;  // pair_row without its "only pair of the row" bit

// kGated: the weight holds gate rows, then up rows, and a tile takes as many of
// each; kBack: the gate's backward.
enum class Form { kPlain, kGated, kBack };

__device__ __forceinline__ float sigmoidf(float v) { return 1.0f / (1.0f + expf(-v)); }

__device__ __forceinline__ uint2 pack4(f32x4 v)
{
    return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

struct TileArgs {
    const char *q;            // rows of tokens
    const int32_t *q_rows;    // their places (nullable: in group order)
    int64_t ldq;              // bytes of a row
    const char *p;            // weights
    int64_t p_expert;         // bytes of an expert's weight
    int64_t ldp;              // bytes of a weight row
    int N, K;                 // columns (I for the gated form) and inner length
    unsigned mt, nt;          // grid of row and column tiles
};

// ------------------------------------------------------------------ tiles
//
// Groups of rows (one expert's rows each), as the device sees them: either
// contiguous ranges given by offsets[G + 1], or the low-latency cells, slots
// rows each of which the first counts[g] are used.
struct Groups {
    const int32_t *offsets;  // contiguous ranges, or
    const int32_t *counts;   // cell blocks (null: every slot is used)
    int32_t slots;           // rows of a cell block
    int32_t num;             // G
    int32_t ranks, epr;      // cell block g holds expert (g % ranks) * epr + g / ranks
    int32_t min_rows;        // groups of fewer rows are left to another kernel
    int32_t max_rows;        // and so are groups of more
};

__device__ __forceinline__ int group_rows(const Groups &G, int g)
{
    int c;
    if (G.offsets != nullptr)
        c = G.offsets[g + 1] - G.offsets[g];
    else {
        c = G.counts != nullptr ? G.counts[g] : G.slots;
        c = c < G.slots ? c : G.slots;
    }
    return c >= G.min_rows && c <= G.max_rows ? c : 0;
}
__device__ __forceinline__ int64_t group_start(const Groups &G, int g)
{
    return G.offsets != nullptr ? int64_t(G.offsets[g]) : int64_t(g) * G.slots;
}
__device__ __forceinline__ int group_expert(const Groups &G, int g)
{
    return G.offsets != nullptr ? g : (g % G.ranks) * G.epr + g / G.ranks;
}

struct Tile {
    int group;
    int m0;    // first row of the tile inside its group
    int rows;  // rows of the group
};

// The tile-th row tile over all groups (each cut into ceil(rows / BM)), or
// group = -1 past the last.  Every thread of the block takes part; s: NT/64 + 1
// ints of LDS.
template <int BM, int NT>
__device__ __forceinline__ Tile find_tile(const Groups &G, int tile, int *s)
{
    constexpr int W = NT / kWave;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __shared__ int found[3];
    if (threadIdx.x == 0)
        found[0] = -1;
    int base = 0;
    for (int g0 = 0; g0 < G.num; g0 += NT) {
        const int g = g0 + threadIdx.x;
        const int rows = g < G.num ? group_rows(G, g) : 0;
        const int t = (rows + BM - 1) / BM;
        int pre = t;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int o = __shfl_up(pre, d);
            pre += lane >= d ? o : 0;
        }
        if (lane == 63)
            s[wave] = pre;
        __syncthreads();
        int before = base, total = base;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int v = s[w];
            before += w < wave ? v : 0;
            total += v;
        }
        const int first = before + pre - t;
        if (tile >= first && tile < first + t) {
            found[0] = g;
            found[1] = (tile - first) * BM;
            found[2] = rows;
        }
        __syncthreads();
        base = total;
        if (tile < base)
            break;
    }
    return Tile{found[0], found[1], found[2]};
}

// Block id -> (row tile, column tile).  Consecutive blocks go round the eight
// XCDs, so each XCD is given a contiguous run of the tile order; in it, bands
// of kBand row tiles are crossed column by column, which keeps both operands
// of the blocks that run together in the XCD's own L2.
constexpr int kXcds = 8;
constexpr int kBand = 4;
__device__ __forceinline__ void tile_of_block(unsigned b, unsigned mt, unsigned nt, unsigned &m,
                                              unsigned &n)
{
    const unsigned total = mt * nt;
    const unsigned per = total / kXcds, extra = total % kXcds;
    const unsigned x = b % kXcds, i = b / kXcds;
    const unsigned id = x * per + (x < extra ? x : extra) + i;
    const unsigned band = id / (kBand * nt), r = id % (kBand * nt);
    const unsigned left = mt - band * kBand;
    const unsigned h = left < kBand ? left : kBand;
    n = r / h;
    m = band * kBand + r % h;
}

__device__ __forceinline__ f32x4 mfma_bf16(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Rows in the order of the groups themselves (low-latency cells).
struct RowOut {
    static constexpr bool kBlockWide = false;
    uint16_t *out;
    template <int MT, int NW>
    __device__ __forceinline__ void store(const Tile &t, int64_t start, int m0, int n0, int N,
                                          const f32x4 (&acc)[MT][NW], int lane) const
    {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = m0 + mt * 16 + (lane & 15);
            if (m >= t.rows)
                continue;
#pragma unroll
            for (int nt = 0; nt < NW; ++nt) {
                const int n = n0 + nt * 16 + (lane >> 4) * 4;
                if (n < N)
                    *reinterpret_cast<uint2 *>(out + (start + m) * N + n) = pack4(acc[mt][nt]);
            }
        }
    }
};

}  // namespace ep
