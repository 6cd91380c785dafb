// few_rows.h -- the products of groups that hold few rows (a decode batch, one
// token): the weight is read once and its bytes are the whole cost.  Where there
// are columns enough for every compute unit, it goes from memory straight into the
// matrix instruction's registers, a wave owning its own weight rows
// (few_rows_kernel); where there are not, the waves of a block share out K
// (split_kernel).  bf16 or FP8 operands.
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

// The j-th group that holds rows, or -1.  Every thread of the block takes part;
// s: LDS of one int a wave and one more, free again afterwards.
template <int NTH>
__device__ __forceinline__ int find_group(const Groups &G, int j, int *s)
{
    constexpr int W = NTH / kWave;
    int &found = s[W];
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
    const int g = found;
    __syncthreads();
    return uniform(g);
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
__device__ __forceinline__ f32x4 mfma_step_wide(const Wide &a, const Wide &b)
{
    f32x4 c = {};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        c = mfma_bf16(a.v[k], b.v[k], c);
    return c;
}
__device__ __forceinline__ f32x4 mfma_step_bf16(const Frag &a, const Frag &b, f32x4 c)
{
    c = mfma_bf16(__builtin_bit_cast(bf16x8, a.lo), __builtin_bit_cast(bf16x8, b.lo), c);
    return mfma_bf16(__builtin_bit_cast(bf16x8, a.hi), __builtin_bit_cast(bf16x8, b.hi), c);
}

// HBM bounds it: 128 tokens on 256 FP8 experts of 2048 x 7168, 11.1 GB, take 1.27 ms
// gated and 0.64 down, 5.8 TB/s (a copy, which also writes, reaches 5.4).
// One block: kCols columns of one group, and of its rows every gridDim.y-th run of
// 16 MT.  WN x WK waves: WN share out the columns, WK the K steps.  A wave holds NW
// 16-column tiles (half gate, half up in the gated form) and MT 16-row tiles.
template <bool FP8, int WN, int WK, int NW, int MT, Form F, class Epi>
__global__ __launch_bounds__(WN *WK *kWave, 2) void few_rows_kernel(FewArgs a, Groups G, Epi epi)
{
    constexpr int kCols = WN * (F == Form::kGated ? NW / 2 : NW) * 16;  // of a block
    constexpr int kWaveCols = kCols / WN;
    __shared__ f32x4 sums[WK > 1 ? (WK - 1) * WN * MT * NW * kWave : 1];
    int g = blockIdx.x / a.nt;
    const int tn = int(blockIdx.x % a.nt);
    if (a.active < G.num) {
        g = find_group<WN * WK * kWave>(G, g, reinterpret_cast<int *>(sums));
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
                    for (int m = 0; m < MT; ++m)
                        acc[m][i] += mfma_step_wide(p, q[m]) * (t.sq[m] * t.sp[i >= NW / 2]);
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
        Step cur, nxt;  // one step in flight while one is used
        if (s0 < s1)
            load(cur, s0);
        for (int s = s0; s < s1; ++s) {
            if (s + 1 < s1)
                load(nxt, s + 1);
            use(cur);
            cur = nxt;
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

// Products whose blocks leave compute units idle: 16 MT rows by 64 columns (32
// gate and their 32 up) a block, K shared out over the eight waves.  A wave stages
// its own K steps in LDS of its own, whole 128-byte lines a row, and nobody else
// reads them, so the loop has no barrier: as soon as a step is in registers the
// next is sent off behind its matrix instructions.  The waves' sums meet at the end.
// Gated FP8 rows, whose codes need the largest of 128 activations: 128 gate and
// their 128 up columns a block, and four waves, which then fill the LDS.
constexpr int kSplitCols = 64;
template <bool BLOCK_WIDE>
struct SplitShape {
    static constexpr int kWaves = BLOCK_WIDE ? 4 : NT / kWave;
    static constexpr int kCols = BLOCK_WIDE ? BN : kSplitCols;  // of the weight
    static constexpr int kThreads = kWaves * kWave;
};

// 16 rows from r0 of a staged K step.
__device__ __forceinline__ Frag staged_frag(const lds_char *base, int r0, int lane)
{
    using At = RowStage<16, kWave>;  // (where a chunk lies does not depend on the rows staged)
    typedef const __attribute__((address_space(3))) i32x4 lds_i32x4;
    Frag f;
    f.lo = *(lds_i32x4 *)At::at(base, r0 + (lane & 15), lane >> 4);
    f.hi = *(lds_i32x4 *)At::at(base, r0 + (lane & 15), 4 + (lane >> 4));
    return f;
}

template <bool FP8, int MT, Form F, class Epi>
__global__ __launch_bounds__(SplitShape<Epi::kBlockWide>::kThreads, Epi::kBlockWide ? 1 : MT == 1 ? 4 : 2) void
split_kernel(FewArgs a, Groups G, Epi epi)
{
    using Shape = SplitShape<Epi::kBlockWide>;
    constexpr int W = Shape::kWaves, NW = Shape::kCols / 16;
    constexpr int kCols = F == Form::kGated ? Shape::kCols / 2 : Shape::kCols;
    constexpr bool kWiden = FP8 && F == Form::kGated;
    using PR = NearRowStage<Shape::kCols / 2, kWave>;
    using QR = NearRowStage<16 * MT, kWave>;
    constexpr int kQ = 2 * PR::kBytes, kOwn = kQ + QR::kBytes;
    static_assert(kOwn >= MT * NW * kWave * 16, "a wave's sums take the place of its last step");
    __shared__ __attribute__((aligned(128))) char smem[W * kOwn];
    int g = blockIdx.x / a.nt;
    const int n0 = int(blockIdx.x % a.nt) * kCols;
    if (a.active < G.num) {
        g = find_group<Shape::kThreads>(G, g, reinterpret_cast<int *>(smem));
        if (g < 0)
            return;
    }
    const int rows = uniform(group_rows(G, g));
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    lds_char *own = (lds_char *)smem + wave * kOwn;
    const int64_t start = group_start(G, g);
    const int e = group_expert(G, g);
    const int steps = (a.kbytes + kStepBytes - 1) / kStepBytes;
    const int s0 = steps * wave / W, s1 = steps * (wave + 1) / W;
    PR pr[2];  // gate and up columns, or the two halves
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c0 = F == Form::kGated ? n0 : n0 + h * (Shape::kCols / 2);
        const int c = c0 < a.N ? c0 : a.N - 1;
        const int64_t row = c + (F == Form::kGated ? h * int64_t(a.N) : 0);
        pr[h].init(lane, a.p + int64_t(e) * a.p_expert + row * a.ldp, [&](int, int r) {
            return uint32_t(c + r < a.N ? r : a.N - 1 - c) * uint32_t(a.ldp);
        });
    }
    const float *ps = FP8 ? a.p_scale + e * a.p_scales + int64_t(n0 >> 7) * steps : nullptr;
    const float *ps_up = kWiden ? ps + int64_t(a.N >> 7) * steps : ps;
    for (int m0 = int(blockIdx.y) * 16 * MT; m0 < rows; m0 += int(gridDim.y) * 16 * MT) {
        QR qr;
        qr.init(lane, a.q + (start + m0) * a.ldq, [&](int, int r) {
            return uint32_t(m0 + r < rows ? r : rows - 1 - m0) * uint32_t(a.ldq);
        });
        const float *qs[MT];
        float next[MT], next_c = 0.0f, next_up = 0.0f;  // scales of the step on its way
        if constexpr (FP8) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int r = m0 + m * 16 + (lane & 15);
                qs[m] = a.q_scale + (start + (r < rows ? r : rows - 1)) * steps;
            }
        }
        auto send = [&](int s) {
            const int64_t kb = int64_t(s) * kStepBytes;
            if constexpr (FP8) {
                next_c = ps[s];
                next_up = kWiden ? ps_up[s] : 0.0f;
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    next[m] = qs[m][s];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
                pr[h].template issue<!FP8>(own + h * PR::kBytes, lane, 0, kb, a.kbytes);
            qr.template issue<!FP8>(own + kQ, lane, 0, kb, a.kbytes);
        };
        f32x4 acc[MT][NW] = {};
        if (s0 < s1)
            send(s0);
        for (int s = s0; s < s1; ++s) {
            landed<0>();
            Frag p[NW], q[MT];
            float scale[2][MT];
            if constexpr (FP8) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    scale[0][m] = next[m] * next_c;
                    scale[1][m] = next[m] * next_up;
                    hold(scale[0][m]);  // here: behind send() it would wait for the next step's loads
                    if (kWiden)
                        hold(scale[1][m]);
                }
            }
#pragma unroll
            for (int i = 0; i < NW; ++i)
                p[i] = staged_frag(own, i * 16, lane);
#pragma unroll
            for (int m = 0; m < MT; ++m)
                q[m] = staged_frag(own + kQ, m * 16, lane);
            // read before the same LDS is loaded again
            asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
            if (s + 1 < s1)
                send(s + 1);
            if constexpr (kWiden) {
                Wide qw[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    qw[m] = widen(q[m]);
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    const Wide pw = widen(p[i]);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[m][i] += mfma_step_wide(pw, qw[m]) * scale[i >= NW / 2][m];
                }
            } else {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < NW; ++i) {
                        if constexpr (FP8)
                            acc[m][i] += mfma_step_fp8(p[i], q[m]) * scale[0][m];
                        else
                            acc[m][i] = mfma_step_bf16(p[i], q[m], acc[m][i]);
                    }
            }
        }
        f32x4 *sums = reinterpret_cast<f32x4 *>(smem);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NW; ++i)
                sums[wave * (kOwn / 16) + (m * NW + i) * kWave + lane] = acc[m][i];
        __syncthreads();
        const Tile t{g, m0, rows, int(blockIdx.x % a.nt)};
        if constexpr (Epi::kBlockWide) {  // wave w: 32 gate columns and their up columns
            f32x4 sum[MT][4] = {};
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = 2 * wave + (i & 1) + (i >> 1) * (NW / 2);
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        sum[m][i] += sums[w * (kOwn / 16) + (m * NW + at) * kWave + lane];
                }
            epi.template store_block<MT, 4, W, 16 * MT>(t, start, true, wave, 0, n0 + wave * 32, a.N, sum, lane);
        } else if (wave < 2 * MT) {  // two column tiles each: neighbours, or a gate and its up tile
            const int m = wave >> 1, h = wave & 1;
            const int i0 = F == Form::kGated ? h : 2 * h, i1 = F == Form::kGated ? h + 2 : i0 + 1;
            f32x4 sum[1][2] = {};
#pragma unroll
            for (int w = 0; w < W; ++w) {
                sum[0][0] += sums[w * (kOwn / 16) + (m * NW + i0) * kWave + lane];
                sum[0][1] += sums[w * (kOwn / 16) + (m * NW + i1) * kWave + lane];
            }
            epi.store(t, start, m0 + m * 16, n0 + h * (kCols / 2), a.N, sum, lane);
        }
        if (m0 + int(gridDim.y) * 16 * MT < rows)
            __syncthreads();  // the sums are read before the next rows are staged
    }
}

// --------------------------------------------------------------- launches

// Rows up to which a group takes this kernel: it reads the weight again (from L2)
// for every 16 MT rows.
constexpr int kFewRows = 64;

template <class Kernel, class Epi>
hipError_t launch_few_shape(Kernel kernel, int threads, FewArgs a, const Groups &G, int cols, int tile_rows,
                            int row_blocks, const Epi &epi, const char *what, hipStream_t stream)
{
    a.nt = unsigned((a.N + cols - 1) / cols);
    const int64_t blocks = int64_t(a.nt) * a.active;
    if (blocks > kMaxTileBlocks || row_blocks > 65535)
        return hipErrorInvalidValue;
    if (log_enabled())
        log_launch("%s: groups<=%d of %d N=%d K bytes=%d few rows %d cols=%d blocks=%lld x %d", what, a.active,
                   G.num, a.N, a.kbytes, tile_rows, cols, (long long)blocks, row_blocks);
    hipLaunchKernelGGL(kernel, dim3(unsigned(blocks), row_blocks), dim3(threads), 0, stream, a, G, epi);
    return hipGetLastError();
}

// Rows of a group up to which wide blocks beat tiles (16 experts of 2048 x 7168:
// bf16 of 4 rows 260 against 273 us, of 25 rows 457 against 280; FP8 64 experts of
// 768 x 2048, 4 rows 72.0 against 75.6, 8 rows 76.5 against 68.8).
template <bool FP8>
constexpr int kWideRows = FP8 ? 4 : 8;

// Whether blocks of 256 columns (128 gated) would leave compute units idle; then
// they take 64 (32) columns and split K: one token's eight bf16 experts of
// 768 x 2048, gated, 11.6 us in 192 blocks, 34 in 48 wide ones.
template <Form F>
bool splits_k(const FewArgs &a, int64_t row_blocks)
{
    constexpr int wide = F == Form::kGated ? BN / 2 : BN;
    return int64_t((a.N + wide - 1) / wide) * a.active * row_blocks < compute_units();
}

// avg: rows of an active group on average.
template <bool FP8, Form F, class Epi>
hipError_t launch_few(FewArgs a, const Groups &G, int64_t avg, int row_blocks, const Epi &epi, const char *what,
                      hipStream_t stream)
{
    using Split = SplitShape<Epi::kBlockWide>;
    constexpr int wide = F == Form::kGated ? BN / 2 : BN, split = wide / (BN / Split::kCols);
    constexpr int threads = Split::kThreads;
    auto launch = [&](auto kernel, int n, int cols, int tile_rows) {
        return launch_few_shape(kernel, n, a, G, cols, tile_rows, row_blocks, epi, what, stream);
    };
    if (!splits_k<F>(a, row_blocks))
        return launch(few_rows_kernel<FP8, 4, 2, 4, 1, F, Epi>, NT, wide, 16);
    if constexpr (!Epi::kBlockWide) {
        if (avg > 32)
            return launch(split_kernel<FP8, 4, F, Epi>, threads, split, 64);
        if (avg > 16)
            return launch(split_kernel<FP8, 2, F, Epi>, threads, split, 32);
    }
    return launch(split_kernel<FP8, 1, F, Epi>, threads, split, 16);
}

// The low-latency cells: groups of few rows by launch_few, the others by
// tiles(G, most): both walk the groups on the device, which alone knows their
// rows; most bounds the groups left for the tiles.  With K split the border is
// where groups of more than 64 rows become common (eight bf16 experts of
// 768 x 2048 with 40 rows each: 26.2 against 39.7 us, with 60: 57.5 against 40.4),
// for gated FP8, whose blocks take 16 rows, lower (8 rows: 18.9 against 24.0 us, 12
// rows: 27.9 against 24.0).
template <bool FP8, Form F, class Epi, class Tiles>
hipError_t launch_cells(FewArgs a, Groups G, int64_t max_pairs, const Epi &epi, const char *what,
                        hipStream_t stream, Tiles tiles)
{
    a.active = int(max_pairs < G.num ? max_pairs : G.num);
    const int64_t avg = max_pairs / a.active;
    const int most_avg = splits_k<F>(a, 1) ? Epi::kBlockWide ? 8 : 48 : kWideRows<FP8>;
    if (avg <= most_avg) {
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
