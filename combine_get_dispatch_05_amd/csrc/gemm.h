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
//
// The eight waves of a block are two groups of four, one wave of each on every
// SIMD, and take turns (turns_on_ring, turns_on_pair): while one group's wave keeps the matrix
// core busy, the other reads its next fragments from LDS and sends off loads.
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

// A value that is the same in every lane, told to the compiler.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const char *uniform(const char *p)
{
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = uint32_t(uniform(int(uint32_t(v)))), hi = uint32_t(uniform(int(uint32_t(v >> 32))));
    return reinterpret_cast<const char *>(uint64_t(lo) | uint64_t(hi) << 32);
}

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
// The same from base + off, base the same for the whole wave.
__device__ __forceinline__ void load_lds16(const char *base, uint32_t off, lds_char *dst)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(off), "s"(uniform(base)), "s"(lds_at(dst))
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

// Ties a value to its place among the barriers: matrix instructions touch no
// memory, so only what they read keeps them from being moved across one.
template <class T>
__device__ __forceinline__ void hold(T &v)
{
    asm volatile("" : "+v"(v));
}

// A copy whose uses are computed where they stand: what only a last, partial stage
// needs would otherwise be kept in registers through the whole loop.
__device__ __forceinline__ int here(int v)
{
    hold(v);
    return v;
}

constexpr int32_t kRowMask = 0x7fffffff;  // pair_row without its "only pair of the row" bit

constexpr int kStepBytes = 128;  // K bytes of one stage

// Row-contiguous operand, ROWS rows staged by NT threads.  LDS row r holds its
// eight 16-byte chunks at position c ^ ((r >> 1) & 7): sixteen consecutive
// rows read at one chunk then fall on sixteen different 16-byte bank groups.
template <int ROWS, int NT>
struct RowStage {
    static constexpr int J = ROWS * 8 / NT;
    static constexpr int kBytes = ROWS * kStepBytes;
    const char *ptr[J];
    // byte of the thread's j-th chunk inside the K step
    static __device__ __forceinline__ int byte_of(int tid, int j)
    {
        const int q = j * NT + tid;
        return ((q & 7) ^ ((q >> 4) & 7)) * 16;
    }

    // row_ptr(j, r): the address of LDS row r (this thread's j-th) at k = 0 (any valid row for rows
    // past the end: their results are never stored).
    template <class F>
    __device__ __forceinline__ void init(int tid, F row_ptr)
    {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            ptr[j] = row_ptr(j, (j * NT + tid) >> 3) + byte_of(tid, j);
        }
    }
    // Stage K bytes [kb, kb + 128); kbytes: all K bytes of the operand (a whole
    // number of steps where TAIL is false).
    // J0, JS: this thread's chunks J0, J0 + JS, ...
    template <bool TAIL, int J0 = 0, int JS = 1>
    __device__ __forceinline__ void issue(lds_char *base, int tid, int wave, int64_t kb, int64_t kbytes)
    {
        if (!TAIL || kb + kStepBytes <= kbytes) {
#pragma unroll
            for (int j = J0; j < J; j += JS)
                load_lds16(ptr[j] + kb, base + (j * NT + wave * kWave) * 16);
        } else {
            tid = here(tid);
#pragma unroll
            for (int j = J0; j < J; j += JS)
                load_lds16(kb + byte_of(tid, j) >= kbytes ? reinterpret_cast<const char *>(kZero16) : ptr[j] + kb,
                           base + (j * NT + wave * kWave) * 16);
        }
    }
    // Chunk ch (0..7) of LDS row r.
    static __device__ __forceinline__ const lds_char *at(const lds_char *base, int r, int ch)
    {
        return base + r * kStepBytes + ((ch ^ ((r >> 1) & 7)) << 4);
    }
    // bf16 fragment of 16 rows from r0 and the 32 k values of half ks: lane l
    // gets row r0 + l % 16, k = ks * 32 + (l / 16) * 8 .. + 7.
    static __device__ __forceinline__ bf16x8 frag(const lds_char *base, int r0, int ks, int lane)
    {
        return *(const __attribute__((address_space(3))) bf16x8 *)at(base, r0 + (lane & 15),
                                                                     ks * 4 + (lane >> 4));
    }
};

// The same for rows that lie within 4 GB of one address: 32-bit offsets, half the
// registers, and no address arithmetic in the loop.
template <int ROWS, int NT>
struct NearRowStage {
    static constexpr int J = ROWS * 8 / NT;
    static constexpr int kBytes = ROWS * kStepBytes;
    const char *base;  // uniform
    uint32_t off[J];
    // row_off(j, r): offset of LDS row r from base_
    template <class F>
    __device__ __forceinline__ void init(int tid, const char *base_, F row_off)
    {
        base = uniform(base_);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int q = j * NT + tid;
            const int r = q >> 3;
            off[j] = row_off(j, r) + RowStage<ROWS, NT>::byte_of(tid, j);
        }
    }
    template <bool TAIL, int J0 = 0, int JS = 1>
    __device__ __forceinline__ void issue(lds_char *lds, int tid, int wave, int64_t kb, int64_t kbytes)
    {
        if (!TAIL || kb + kStepBytes <= kbytes) {
#pragma unroll
            for (int j = J0; j < J; j += JS)
                load_lds16(base + kb, off[j], lds + (j * NT + wave * kWave) * 16);
        } else {
            tid = here(tid);
#pragma unroll
            for (int j = J0; j < J; j += JS) {
                const bool past = kb + RowStage<ROWS, NT>::byte_of(tid, j) >= kbytes;
                load_lds16(past ? reinterpret_cast<const char *>(kZero16) : base + kb + off[j],
                           lds + (j * NT + wave * kWave) * 16);
            }
        }
    }
    static __device__ __forceinline__ bf16x8 frag(const lds_char *lds, int r0, int ks, int lane)
    {
        return RowStage<ROWS, NT>::frag(lds, r0, ks, lane);
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
    int cb[J];  // byte of this thread's (clamped) column inside a row of memory

    static __device__ __forceinline__ int g2(int r) { return ((r & 3) | (((r >> 3) & 1) << 2)) << 1; }
    static __device__ __forceinline__ int k_of(int tid, int j) { return (j * NT + tid) / CH; }

    // n0: first column of the tile, n: columns of the operand (a multiple of 8)
    __device__ __forceinline__ void init(int tid, int n0, int n)
    {
        static_assert(CH >= 16, "the swizzle reaches over sixteen chunks");
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int q = j * NT + tid;
            int c = n0 + ((q % CH) ^ g2(q / CH)) * 8;
            c = c < n ? c : n - 8;
            cb[j] = c * 2;
        }
    }
    // Rows k0 .. k0 + 63 of memory, those past kn as zeros; row 0 at base, ld
    // bytes apart.  J0, JN: this thread's chunks J0 .. J0 + JN - 1 (the first half
    // of them is the first half of the rows).
    template <int J0 = 0, int JN = J>
    __device__ __forceinline__ void issue(lds_char *lds, int tid, int wave, const char *base, int64_t ld,
                                          int k0, int kn)
    {
        const char *first = uniform(base + k0 * ld);
        if (k0 + 64 <= kn) {
#pragma unroll
            for (int j = J0; j < J0 + JN; ++j)
                load_lds16(first, uint32_t(k_of(tid, j)) * uint32_t(ld) + cb[j],
                           lds + (j * NT + wave * kWave) * 16);
        } else {
            tid = here(tid);
#pragma unroll
            for (int j = J0; j < J0 + JN; ++j) {
                const int k = k_of(tid, j);
                load_lds16(k0 + k < kn ? first + k * ld + cb[j] : reinterpret_cast<const char *>(kZero16),
                           lds + (j * NT + wave * kWave) * 16);
            }
        }
    }
    // The same with row[j] the memory row of this thread's j-th chunk, as pair_row has it.
    template <int J0 = 0, int JN = J>
    __device__ __forceinline__ void issue(lds_char *lds, int tid, int wave, const char *base, int64_t ld,
                                          int k0, int kn, const int (&row)[J])
    {
        if (k0 + 64 <= kn) {
#pragma unroll
            for (int j = J0; j < J0 + JN; ++j)
                load_lds16(base + (row[j] & kRowMask) * ld + cb[j], lds + (j * NT + wave * kWave) * 16);
        } else {
            tid = here(tid);
#pragma unroll
            for (int j = J0; j < J0 + JN; ++j)
                load_lds16(k0 + k_of(tid, j) < kn ? base + (row[j] & kRowMask) * ld + cb[j]
                                                  : reinterpret_cast<const char *>(kZero16),
                           lds + (j * NT + wave * kWave) * 16);
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

// kGated: the weight holds gate rows, then up rows, and a tile takes as many of
// each; kBack: the gate's backward.
enum class Form { kPlain, kGated, kBack };

// 1 / (1 + e^-v), good to a few units in the last place.  e^-v = 2^t (1 + r ln 2)
// with t = -v / ln 2 rounded and r what the rounding lost; one Newton step on the
// hardware reciprocal.  Past 87 the steps are taken at 87, where it is 1, so that
// they stay finite; below -87 it would no longer be a normal number, and is 0.  A NaN
// gives some number: each use multiplies by v as well.  (The library's exponential and
// division took 13 us of a 254 us tile.)
__device__ __forceinline__ float sigmoidf(float v)
{
    constexpr float kLog2e = 1.44269504f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.69314718f;
    const float c = __builtin_amdgcn_fmed3f(v, -87.0f, 87.0f);
    const float t = -c * kLog2e;
    const float r = fmaf(-c, kLog2e, -t) - c * kLog2eLow;
    const float e = __builtin_amdgcn_exp2f(t);
    const float d = 1.0f + fmaf(e, r * kLn2, e);
    const float q = __builtin_amdgcn_rcpf(d);
    return v < -87.0f ? 0.0f : fmaf(q, fmaf(-d, q, 1.0f), q);
}

__device__ __forceinline__ uint2 pack4(f32x4 v)
{
    return make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
}

// The bf16 stores of a wave's NW 16 x 16 tiles of one row tile: a lane holds four
// columns of each tile, 8 bytes; swapping with the neighbouring 16 lanes gives
// it eight of one tile, so that four lanes write 64 bytes of a row together.
// row: this lane's row of the output (its column 0); n0: the first column.
template <int NW>
__device__ __forceinline__ void store_bf16_row(uint16_t *row, int n0, int N, const f32x4 (&v)[NW], int lane)
{
    const int g = lane >> 4;
    if constexpr (NW % 2 == 0) {
#pragma unroll
        for (int i = 0; i < NW; i += 2) {
            const uint2 a = pack4(v[i]), b = pack4(v[i + 1]);
            const auto x = __builtin_amdgcn_permlane16_swap(a.x, b.x, false, false);
            const auto y = __builtin_amdgcn_permlane16_swap(a.y, b.y, false, false);
            const int n = n0 + (i + (g & 1)) * 16 + (g >> 1) * 8;
            if (row != nullptr && n < N)
                *reinterpret_cast<u32x4 *>(row + n) = u32x4{x[0], y[0], x[1], y[1]};
        }
    } else {
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const int n = n0 + i * 16 + g * 4;
            if (row != nullptr && n < N)
                *reinterpret_cast<uint2 *>(row + n) = pack4(v[i]);
        }
    }
}

struct TileArgs {
    const char *q;            // rows of tokens
    const int32_t *q_rows;    // their places (nullable: in group order)
    int64_t ldq;              // bytes of a row
    const char *p;            // weights
    int64_t p_expert;         // bytes of an expert's weight
    int64_t ldp;              // bytes of a weight row
    int N, K;                 // columns (I for the gated form) and inner length
    unsigned nt;              // column tiles
    unsigned blocks;          // no tile from this block on
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
    return G.offsets != nullptr ? int64_t(uniform(G.offsets[g])) : int64_t(g) * G.slots;
}
__device__ __forceinline__ int group_expert(const Groups &G, int g)
{
    return G.offsets != nullptr ? g : (g % G.ranks) * G.epr + g / G.ranks;
}

// Inclusive sum over the wave, in the registers: inside each 16 lanes, then the
// rows' last lanes passed on.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v)
{
    v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x111, 0xF, 0xF, true));
    v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x112, 0xF, 0xF, true));
    v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x114, 0xF, 0xF, true));
    v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x118, 0xF, 0xF, true));
    v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x142, 0xA, 0xF, false));
    v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x143, 0xC, 0xF, false));
    return v;
}

struct Tile {
    int group;
    int m0;    // first row of the tile inside its group
    int rows;  // rows of the group
    int n;     // column tile
};

// The order of mt x nt tiles: bands of kBand row tiles, crossed column by column,
// which keeps both operands of the blocks that run together in an L2.
constexpr int kXcds = 8;
constexpr int kBand = 4;
__device__ __forceinline__ void tile_in_bands(unsigned id, unsigned mt, unsigned nt, unsigned &m,
                                              unsigned &n)
{
    const unsigned band = id / (kBand * nt), r = id % (kBand * nt);
    const unsigned left = mt - band * kBand;
    const unsigned h = left < kBand ? left : kBand;
    n = r / h;
    m = band * kBand + r % h;
}

// The i-th of XCD x's contiguous share of n items, or -1 past its last.
__device__ __forceinline__ int64_t share_of_xcd(unsigned n, unsigned x, unsigned i)
{
    const unsigned per = n / kXcds, extra = n % kXcds;
    if (i >= per + (x < extra))
        return -1;
    return int64_t(x) * per + (x < extra ? x : extra) + i;
}

// The tile of block b, over all groups (each cut into row tiles of BM) and nt
// column tiles; group = -1 past the last.  Consecutive blocks go round the
// eight XCDs, so each XCD has a contiguous run of the order.  First come the
// tiles of more than BM / 2 rows, in bands, then the groups' shorter last tiles,
// which cost at most half: in the order of the groups they would leave some blocks
// with a round more of whole tiles than others (experts of about 1024 rows: 9
// rounds of blocks for 8.5 rounds of work).  The order is laid over the tiles
// that there are, not over the grid.  Every thread of the block takes part; calls
// need no barrier between them.
template <int BM, int NT>
__device__ __forceinline__ Tile find_tile(const Groups &G, unsigned b, unsigned nt)
{
    constexpr int W = NT / kWave;
    __shared__ uint64_t s[W];
    __shared__ int found[3];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // low half: whole tiles, high half: the part tile
    auto tiles_of = [&](int g, int &rows) -> uint64_t {
        rows = g < G.num ? group_rows(G, g) : 0;
        const unsigned rest = unsigned(rows) % BM;
        return uint64_t(unsigned(rows) / BM + (rest > BM / 2)) | uint64_t(rest > 0 && rest <= BM / 2) << 32;
    };
    auto scan = [&](uint64_t t, uint64_t &total) {  // exclusive sum of t over the block
        const uint64_t pre = uint64_t(wave_scan(uint32_t(t))) | uint64_t(wave_scan(uint32_t(t >> 32))) << 32;
        __syncthreads();
        if (lane == 63)
            s[wave] = pre;
        // behind the scan's first barrier, which no wave passes before all have read what
        // an earlier call found, and before its second, which the match below comes after
        if (threadIdx.x == 0)
            found[0] = -1;
        __syncthreads();
        uint64_t before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint64_t v = s[w];
            before += w < wave ? v : 0;
            total += v;
        }
        return before + pre - t;
    };
    int rows = 0;
    uint64_t total = 0;
    uint64_t t = tiles_of(threadIdx.x, rows);
    uint64_t first = scan(t, total);
    uint64_t all = total;
    for (int g0 = NT; g0 < G.num; g0 += NT) {  // more groups than threads: the sum first
        int r;
        uint64_t n;
        scan(tiles_of(g0 + threadIdx.x, r), n);
        all += n;
    }
    const unsigned whole = uniform(int(uint32_t(all))), part = uniform(int(uint32_t(all >> 32)));
    unsigned tm = 0, tn = 0;
    const unsigned x = b % kXcds, i = b / kXcds;
    int64_t id = share_of_xcd(whole * nt, x, i);
    const bool is_whole = id >= 0;
    if (is_whole) {
        tile_in_bands(unsigned(id), whole, nt, tm, tn);
    } else {
        // this XCD's whole tiles are i's first ones
        const unsigned mine = whole * nt / kXcds + (x < whole * nt % kXcds);
        id = share_of_xcd(part * nt, x, i - mine);
        if (id < 0)
            return Tile{-1, 0, 0, 0};
        tile_in_bands(unsigned(id), part, nt, tm, tn);
    }
    uint64_t base = 0;
    for (int g0 = 0;;) {
        const unsigned at = is_whole ? uint32_t(base + first) : uint32_t((base + first) >> 32);
        const unsigned n = is_whole ? uint32_t(t) : uint32_t(t >> 32);
        if (tm >= at && tm < at + n) {
            found[0] = g0 + threadIdx.x;
            found[1] = is_whole ? int(tm - at) * BM : rows / BM * BM;
            found[2] = rows;
        }
        base += total;
        g0 += NT;
        if (tm < (is_whole ? uint32_t(base) : uint32_t(base >> 32)) || g0 >= G.num)
            break;
        t = tiles_of(g0 + threadIdx.x, rows);
        first = scan(t, total);
    }
    __syncthreads();
    return Tile{uniform(found[0]), uniform(found[1]), uniform(found[2]), int(tn)};
}

__device__ __forceinline__ f32x4 mfma_bf16(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// A barrier that is only that: no wait for loads in flight, and nothing the
// compiler may move across.
__device__ __forceinline__ void turn()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" : : : "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// The K loop.  A stage is worked off in PH phases, each of them a read half
// (read(s, ph): LDS reads, and loads of later stages) and a compute half
// (compute(s, ph): matrix instructions only), with a barrier after each; the
// second group runs one half behind the first, so one group reads while the
// other computes.  (8192 x 4096 x 7168 bf16, 256 x 256 tiles: 1454 TFLOP/s,
// against 1153 with both groups in step and one barrier a stage.)
//
// Two rules hold everywhere.  A wait for a stage's loads stands in the read half
// of the last phase before it, so the barrier after it publishes the stage to
// both groups.  And LDS that a phase's reads were the last to use is loaded again
// in the next phase's read half at the earliest: the second group's reads of the
// phase before ended, with their wait, before the barrier that opens that half.
__device__ __forceinline__ void end_of_reads()
{
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    turn();
}

// With ST >= 3 stages: stage s + ST - 1 goes where stage s - 1 was, from phase 0
// on.  issue(part, s): parts 0 and 1 are P's halves, 2 and 3 Q's; LOADS a stage.
template <int ST, class Issue>
__device__ __forceinline__ void open_ring(int steps, Issue issue)
{
#pragma unroll
    for (int s = 0; s < ST - 1; ++s)
        if (s < steps) {
#pragma unroll
            for (int part = 0; part < 4; ++part)
                issue(part, s);
        }
}
template <int PH, int ST, int LOADS, class Issue, class Read, class Compute>
__device__ __forceinline__ void turns_on_ring(int steps, int group, Issue issue, Read read, Compute compute)
{
    constexpr int kLater = LOADS * (ST - 2);
    if (steps >= ST - 1)
        landed<kLater>();
    else
        landed<0>();
    turn();
    if (group == 1)
        turn();
    for (int s = 0; s < steps; ++s) {
#pragma unroll
        for (int ph = 0; ph < PH; ++ph) {
            read(s, ph);
            if (ph == 0 && s + ST - 1 < steps) {
#pragma unroll
                for (int part = 0; part < 4; ++part)
                    issue(part, s + ST - 1);
            }
            if (ph == PH - 1) {
                if (s + ST - 1 < steps)
                    landed<kLater>();
                else
                    landed<0>();
            }
            end_of_reads();
            compute(s, ph);
            turn();
        }
    }
    if (group == 0)
        turn();
}

// With two stages, loaded a quarter a phase (a block's 64 KB take the L1 data
// path half of a stage's time, so they are spread over all of it), each as its
// last readers finish.  P's fragments are all read in the first half of the
// phases and kept, so with four phases the halves of P of stage s + 2 are sent
// off in phases 2 and 3 of stage s and the halves of Q of stage s + 1 in phases
// 0 and 1 of stage s: P, the weight, which comes from memory, four and five
// phases before its wait, Q three and two.
// issue(part, s): parts 0 and 1 are P's halves, 2 and 3 Q's; LP: P's loads.
template <class Issue>
__device__ __forceinline__ void open_pair(int steps, Issue issue)
{
    issue(0, 0);
    issue(1, 0);
    issue(2, 0);
    issue(3, 0);
    if (steps > 1) {
        issue(0, 1);
        issue(1, 1);
    }
}
template <int PH, int LP, class Issue, class Read, class Compute>
__device__ __forceinline__ void turns_on_pair(int steps, int group, Issue issue, Read read, Compute compute)
{
    if (steps > 1)
        landed<LP>();
    else
        landed<0>();
    turn();
    if (group == 1)
        turn();
    for (int s = 0; s < steps; ++s) {
        const bool more = s + 2 < steps;
#pragma unroll
        for (int ph = 0; ph < PH; ++ph) {
            read(s, ph);
            if (ph == 0 && s + 1 < steps) {
                if (PH == 1 && s > 0) {
                    issue(0, s + 1);
                    issue(1, s + 1);
                }
                issue(2, s + 1);
            }
            if (ph == (PH > 1) && s + 1 < steps)
                issue(3, s + 1);
            if (PH > 1 && more) {
                if (ph == (PH == 4 ? 2 : PH - 1))
                    issue(0, s + 2);
                if (ph == PH - 1)
                    issue(1, s + 2);
            }
            if (ph == PH - 1) {
                if (PH > 1 && more)
                    landed<LP>();
                else
                    landed<0>();
            }
            end_of_reads();
            compute(s, ph);
            turn();
        }
    }
    if (group == 0)
        turn();
}

// A tile's rows are computed at the least of these heights that holds them.
template <int N>
struct Rows {
    static constexpr int value = N;
};
template <int BM, class F>
__device__ __forceinline__ void at_height(int rows, F f)
{
    if (BM == 64 || rows <= 64)
        return f(Rows<64>{});
    if (rows <= 128)
        return f(Rows<(BM > 64 ? 128 : 64)>{});
    if (rows <= 192)
        return f(Rows<(BM > 64 ? 192 : 64)>{});
    f(Rows<BM>{});
}

// The phases of a bf16 stage for a wave of MT x 4 16 x 16 tiles: with MT = 8 a
// half of the rows and a half ks of the stage's K, with fewer a ks, with MT = 2
// the whole stage.  P's fragments are all read in the first half of the phases.
template <int MT, class FragP, class FragQ>
struct Bf16Phases {
    static constexpr int kPhases = MT == 8 ? 4 : MT > 2 ? 2 : 1;
    static constexpr int MQ = MT == 8 ? 4 : MT;  // row tiles of a phase
    f32x4 (&acc)[MT][4];
    FragP frag_p;  // (stage, column tile, ks)
    FragQ frag_q;  // (stage, row tile, ks)
    bf16x8 p[2][4], q[kPhases == 1 ? 2 : 1][MQ];
    static __device__ __forceinline__ int ks_of(int ph) { return kPhases == 4 ? ph & 1 : ph; }
    static __device__ __forceinline__ int mh_of(int ph) { return kPhases == 4 ? ph >> 1 : 0; }
    __device__ __forceinline__ void read(int s, int ph)
    {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
            if (kPhases == 4 ? ph == ks : ph == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    p[ks][i] = frag_p(s, i, ks);
            }
#pragma unroll
        for (int k = 0; k < (kPhases == 1 ? 2 : 1); ++k)
#pragma unroll
            for (int m = 0; m < MQ; ++m)
                q[k][m] = frag_q(s, mh_of(ph) * 4 + m, kPhases == 1 ? k : ks_of(ph));
    }
    __device__ __forceinline__ void compute(int ph)
    {
#pragma unroll
        for (int k = 0; k < (kPhases == 1 ? 2 : 1); ++k)
#pragma unroll
            for (int m = 0; m < MQ; ++m)
                hold(q[k][m]);
#pragma unroll
        for (int k = 0; k < (kPhases == 1 ? 2 : 1); ++k)
#pragma unroll
            for (int m = 0; m < MQ; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int a = mh_of(ph) * 4 + m;
                    acc[a][i] = mfma_bf16(p[kPhases == 1 ? k : ks_of(ph)][i], q[k][m], acc[a][i]);
                }
    }
};

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
            store_bf16_row<NW>(m < t.rows ? out + (start + m) * N : nullptr, n0, N, acc[mt], lane);
        }
    }
};

// Blocks that reach every tile: an XCD's run of whole tiles and its run of part
// tiles can each be one longer than an eighth.
inline int64_t blocks_for_tiles(int64_t tiles) { return (tiles / kXcds + 2) * kXcds; }


}  // namespace ep
