// few_rows.h -- the products of groups that hold few rows (a decode batch, one
// token): the weight is read once and its bytes are the whole cost, so it
// goes from memory straight into the matrix instruction's registers, a wave
// owning its own weight rows, and only the partial sums of waves that share an
// output cross LDS.  bf16 or FP8 operands.
#pragma once

#include "gemm.h"

namespace ep {

struct FewArgs {
    const char *q;         // token rows, in group order
    const float *q_scale;  // FP8: [row][K / 128]
    int64_t ldq;           // bytes of a token row
    const char *p;         // weights
    const float *p_scale;  // FP8: [expert][rows of blocks][K / 128]
    int64_t p_expert;      // bytes of an expert's weight
    int64_t p_scales;      // scales of an expert's weight
    int64_t ldp;           // bytes of a weight row
    int N;                 // columns (I for the gated form)
    int kbytes;            // bytes of the inner dimension
    unsigned nt;           // column tiles
    int active;            // groups that can hold rows, where fewer than all
};

// The j-th group that holds rows, or -1.  Every thread of the block takes part.
template <int NTH>
__device__ __forceinline__ int find_group(const Groups &G, int j)
{
    constexpr int W = NTH / kWave;
    __shared__ int s[W], found;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (threadIdx.x == 0)
        found = -1;
    for (int g0 = 0, base = 0; g0 < G.num && j >= base; g0 += NTH) {
        const int g = g0 + threadIdx.x;
        const bool alive = g < G.num && group_rows(G, g) > 0;
        const uint64_t m = wave_ballot(alive);
        __syncthreads();
        if (lane == 0)
            s[wave] = __popcll(m);
        __syncthreads();
        int before = base;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int v = s[w];
            before += w < wave ? v : 0;
            base += v;
        }
        if (alive && before + __popcll(m & lanemask_lt()) == j)
            found = g;
    }
    __syncthreads();
    return uniform(found);
}

// 32 bytes of a row for one K step: bytes [16 g, 16 g + 16) and 64 further on,
// g = lane / 16.  Both operands use the same places, so their order inside the
// step does not matter.
struct Frag {
    i32x4 lo, hi;
};
__device__ __forceinline__ Frag load_frag(const char *p, int kb, int kbytes)
{
    Frag f;
    const i32x4 z = {};
    f.lo = kb < kbytes ? *reinterpret_cast<const i32x4 *>(p) : z;
    f.hi = kb + 64 < kbytes ? *reinterpret_cast<const i32x4 *>(p + 64) : z;
    return f;
}

// One scale block of K.  The instruction adds the products of each eight
// neighbouring k after aligning them to the largest, 2^E, and drops what lies
// below 2^(E - 13); the eights are added in fp32.  That is 2e-5 of the summed
// magnitudes, far below a bf16 result's rounding, for twice the rate of bf16.
__device__ __forceinline__ f32x4 mfma_step_fp8(const Frag &a, const Frag &b)
{
    const i32x8 x = __builtin_shufflevector(a.lo, a.hi, 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 y = __builtin_shufflevector(b.lo, b.hi, 0, 1, 2, 3, 4, 5, 6, 7);
    const f32x4 z = {};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, z, 0, 0, 0, 0x7f7f7f7f, 0,
                                                            0x7f7f7f7f);
}

// The gated form's FP8 fragments are widened to bf16, exactly, and multiplied in
// full fp32 sums: there the alignment would show, on a few rows, where it moves
// an activation across a rounding border of its own 8-bit code, and the memory,
// not the matrix cores, sets the time.
struct Wide {
    bf16x8 v[4];
};
__device__ __forceinline__ Wide widen(const Frag &f)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    Wide w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = i < 2 ? f.lo[2 * i + h] : f.hi[2 * (i - 2) + h];
            const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false);
            const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true);
            w.v[i][4 * h] = lo[0];
            w.v[i][4 * h + 1] = lo[1];
            w.v[i][4 * h + 2] = hi[0];
            w.v[i][4 * h + 3] = hi[1];
        }
    }
    return w;
}
__device__ __forceinline__ f32x4 mfma_step_bf16(const Frag &a, const Frag &b, f32x4 c)
{
    c = mfma_bf16(__builtin_bit_cast(bf16x8, a.lo), __builtin_bit_cast(bf16x8, b.lo), c);
    return mfma_bf16(__builtin_bit_cast(bf16x8, a.hi), __builtin_bit_cast(bf16x8, b.hi), c);
}

// One block: kCols columns of one group, and of its rows every gridDim.y-th run of
// 16 MT.  WN x WK waves: WN share out the columns, WK the K steps.  A wave holds NW
// 16-column tiles (half gate, half up in the gated form) and MT 16-row tiles.
template <bool FP8, int WN, int WK, int NW, int MT, Form F, class Epi>
__global__ __launch_bounds__(WN *WK *kWave, WN == 1 && MT == 1 ? 4 : 2) void few_rows_kernel(FewArgs a, Groups G, Epi epi)
{
    constexpr int kCols = WN * (F == Form::kGated ? NW / 2 : NW) * 16;  // of a block
    constexpr int kWaveCols = kCols / WN;
    __shared__ f32x4 sums[WK > 1 ? (WK - 1) * WN * MT * NW * kWave : 1];
    int g = blockIdx.x / a.nt;
    const int tn = int(blockIdx.x % a.nt);
    if (a.active < G.num) {
        g = find_group<WN * WK * kWave>(G, g);
        if (g < 0)
            return;
    }
    const int rows = uniform(group_rows(G, g));
    const int first = int(blockIdx.y) * 16 * MT, stride = int(gridDim.y) * 16 * MT;
    if (first >= rows)
        return;
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int wn = wave % WN, wk = wave / WN;
    const int64_t start = group_start(G, g);
    const int e = group_expert(G, g);
    const char *pw = a.p + int64_t(e) * a.p_expert;
    const int n0 = tn * kCols + wn * kWaveCols;
    const int kl = (lane >> 4) * 16;
    const char *pp[NW];
    const float *ps[2] = {nullptr, nullptr};
    const int kblocks = a.kbytes >> 7;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const bool up = F == Form::kGated && i >= NW / 2;
        int n = n0 + (up ? i - NW / 2 : i) * 16 + (lane & 15);
        n = (n < a.N ? n : a.N - 1) + (up ? a.N : 0);
        pp[i] = pw + int64_t(n) * a.ldp + kl;
    }
    if constexpr (FP8) {
        const int nb = n0 < a.N ? n0 : a.N - 1;
        ps[0] = a.p_scale + e * a.p_scales + int64_t(nb >> 7) * kblocks;
        ps[1] = F == Form::kGated ? ps[0] + int64_t(a.N >> 7) * kblocks : ps[0];
    }
    const int steps = (a.kbytes + kStepBytes - 1) / kStepBytes;
    const int s0 = steps * wk / WK, s1 = steps * (wk + 1) / WK;
    for (int m0 = first; m0 < rows; m0 += stride) {
        const char *qp[MT];
        const float *qs[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            int m = m0 + i * 16 + (lane & 15);
            m = m < rows ? m : rows - 1;
            qp[i] = a.q + (start + m) * a.ldq + kl;
            qs[i] = FP8 ? a.q_scale + (start + m) * kblocks : nullptr;
        }
        f32x4 acc[MT][NW] = {};
        struct Step {
            Frag p[NW], q[MT];
            float sp[2], sq[MT];
        };
        auto load = [&](Step &t, int s) {
            const int64_t kb = int64_t(s) * kStepBytes;
            const int left = a.kbytes - int(kb);
#pragma unroll
            for (int i = 0; i < NW; ++i)
                t.p[i] = load_frag(pp[i] + kb, kl, left);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                t.q[i] = load_frag(qp[i] + kb, kl, left);
            if constexpr (FP8) {
                t.sp[0] = ps[0][s];
                t.sp[1] = F == Form::kGated ? ps[1][s] : t.sp[0];
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    t.sq[i] = qs[i][s];
            }
        };
        auto use = [&](const Step &t) {
            if constexpr (FP8 && F == Form::kGated) {
                Wide q[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    q[m] = widen(t.q[m]);
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    const Wide p = widen(t.p[i]);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        f32x4 part = {};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            part = mfma_bf16(p.v[k], q[m].v[k], part);
                        acc[m][i] += part * (t.sq[m] * t.sp[i >= NW / 2]);
                    }
                    __builtin_amdgcn_sched_barrier(0);  // one tile at a time: more would not fit the registers
                }
            } else if constexpr (FP8) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < NW; ++i)
                        acc[m][i] += mfma_step_fp8(t.p[i], t.q[m]) * (t.sq[m] * t.sp[0]);
            } else {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < NW; ++i)
                        acc[m][i] = mfma_step_bf16(t.p[i], t.q[m], acc[m][i]);
            }
        };
        // U steps are in flight while U are used: as many as the registers hold
        constexpr int U = NW + MT == 2 ? 2 : 1;
        Step cur[U], nxt[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u < s1)
                load(cur[u], s0 + u);
        for (int s = s0; s < s1; s += U) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s + U + u < s1)
                    load(nxt[u], s + U + u);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s + u < s1)
                    use(cur[u]);
#pragma unroll
            for (int u = 0; u < U; ++u)
                cur[u] = nxt[u];
        }
        if constexpr (WK > 1) {
            if (wk > 0) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < NW; ++i)
                        sums[((((wk - 1) * WN + wn) * MT + m) * NW + i) * kWave + lane] = acc[m][i];
            }
            __syncthreads();
            if (wk == 0) {
#pragma unroll 1
                for (int w = 0; w < WK - 1; ++w)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < NW; ++i)
                            acc[m][i] += sums[(((w * WN + wn) * MT + m) * NW + i) * kWave + lane];
            }
        }
        const Tile t{g, m0, rows, tn};
        if constexpr (Epi::kBlockWide)
            epi.template store_block<MT, NW, WN, 16 * MT>(t, start, wk == 0, wn, 0, n0, a.N, acc, lane);
        else if (wk == 0)
            epi.store(t, start, m0, n0, a.N, acc, lane);
        if (m0 + stride < rows)
            __syncthreads();  // the sums are read before the next rows' are written
    }
}

// --------------------------------------------------------------- launches

// Rows up to which a group takes this kernel: it reads the weight again (from L2)
// for every 16 MT rows.
constexpr int kFewRows = 64;

template <bool FP8, int WN, int WK, int NW, int MT, Form F, class Epi>
hipError_t launch_few_shape(FewArgs a, const Groups &G, int row_blocks, const Epi &epi, const char *what,
                            hipStream_t stream)
{
    constexpr int cols = WN * (F == Form::kGated ? NW / 2 : NW) * 16;
    a.nt = unsigned((a.N + cols - 1) / cols);
    const int64_t blocks = int64_t(a.nt) * a.active;
    if (blocks > kMaxTileBlocks || row_blocks > 65535)
        return hipErrorInvalidValue;
    if (log_enabled())
        log_launch("%s: groups<=%d of %d N=%d K bytes=%d few rows %d cols=%d waves=%dx%d blocks=%lld x %d", what,
                   a.active, G.num, a.N, a.kbytes, MT * 16, cols, WN, WK, (long long)blocks, row_blocks);
    hipLaunchKernelGGL((few_rows_kernel<FP8, WN, WK, NW, MT, F, Epi>), dim3(unsigned(blocks), row_blocks),
                       dim3(WN * WK * kWave), 0, stream, a, G, epi);
    return hipGetLastError();
}

// avg: rows of an active group on average.  Blocks of 256 columns (128 gated)
// where that makes one for every compute unit, else of 16, all eight waves
// sharing out K: one token's eight experts of 768 x 2048 in 48 blocks took
// %WIDE% us, in 384 %NARROW%.
template <bool FP8, Form F, class Epi>
hipError_t launch_few(FewArgs a, const Groups &G, int64_t avg, int row_blocks, const Epi &epi, const char *what,
                      hipStream_t stream)
{
    if constexpr (!Epi::kBlockWide) {
        const int wide = F == Form::kGated ? 128 : 256;
        if (int64_t((a.N + wide - 1) / wide) * a.active * row_blocks < compute_units()) {
            constexpr int NW = F == Form::kGated ? 2 : 1;
            return avg <= 16 ? launch_few_shape<FP8, 1, 8, NW, 1, F>(a, G, row_blocks, epi, what, stream)
                             : launch_few_shape<FP8, 1, 8, NW, 4, F>(a, G, row_blocks, epi, what, stream);
        }
    }
    return avg <= 8 ? launch_few_shape<FP8, 4, 2, 4, 1, F>(a, G, row_blocks, epi, what, stream)
                    : launch_few_shape<FP8, 4, 2, 4, 2, F>(a, G, row_blocks, epi, what, stream);
}

// The low-latency cells: groups of few rows by launch_few, the others by
// tiles(G, most): both walk the groups on the device, which alone knows their
// rows; most bounds the groups left for the tiles.
template <bool FP8, Form F, class Epi, class Tiles>
hipError_t launch_cells(FewArgs a, Groups G, int64_t max_pairs, const Epi &epi, const char *what,
                        hipStream_t stream, Tiles tiles)
{
    a.active = int(max_pairs < G.num ? max_pairs : G.num);
    const int64_t avg = max_pairs / a.active;
    if (avg <= kFewRows / 2) {
        Groups few = G;
        few.max_rows = kFewRows;
        hipError_t e = launch_few<FP8, F>(a, few, avg, 1, epi, what, stream);
        if (e != hipSuccess || G.slots <= kFewRows || max_pairs <= kFewRows)
            return e;
        G.min_rows = kFewRows + 1;
    }
    const int64_t most = max_pairs / G.min_rows;
    return tiles(G, most < G.num ? most : G.num);
}

}  // namespace ep
