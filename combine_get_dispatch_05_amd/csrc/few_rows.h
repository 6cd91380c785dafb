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
};

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

__device__ __forceinline__ f32x4 mfma_step_fp8(const Frag &a, const Frag &b)
{
    const i32x8 x = __builtin_shufflevector(a.lo, a.hi, 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 y = __builtin_shufflevector(b.lo, b.hi, 0, 1, 2, 3, 4, 5, 6, 7);
    const f32x4 z = {};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, z, 0, 0, 0, 0x7f7f7f7f, 0,
                                                            0x7f7f7f7f);
}
__device__ __forceinline__ f32x4 mfma_step_bf16(const Frag &a, const Frag &b, f32x4 c)
{
    c = mfma_bf16(__builtin_bit_cast(bf16x8, a.lo), __builtin_bit_cast(bf16x8, b.lo), c);
    return mfma_bf16(__builtin_bit_cast(bf16x8, a.hi), __builtin_bit_cast(bf16x8, b.hi), c);
}

// WN x WK waves: WN share out the columns, WK the K steps.  A wave holds NW
// 16-column tiles (half gate, half up in the gated form) and MT 16-row tiles.
template <bool FP8, int WN, int WK, int NW, int MT, Form F, class Epi>
__global__ __launch_bounds__(WN *WK *kWave) void few_rows_kernel(FewArgs a, Groups G, Epi epi)
{
    constexpr int kCols = WN * (F == Form::kGated ? NW / 2 : NW) * 16;  // of a block
    constexpr int kWaveCols = kCols / WN;
    __shared__ f32x4 sums[WK > 1 ? (WK - 1) * WN * MT * NW * kWave : 1];
    const int g = blockIdx.x / a.nt, tn = int(blockIdx.x % a.nt);
    const int rows = group_rows(G, g);
    if (rows == 0)
        return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    for (int m0 = 0; m0 < rows; m0 += 16 * MT) {
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
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    if constexpr (FP8) {
                        const float sc = t.sq[m] * t.sp[F == Form::kGated && i >= NW / 2];
                        acc[m][i] += mfma_step_fp8(t.p[i], t.q[m]) * sc;
                    } else {
                        acc[m][i] = mfma_step_bf16(t.p[i], t.q[m], acc[m][i]);
                    }
                }
            }
        };
        // two steps are in flight while two are used
        constexpr int U = 2;
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
#pragma unroll
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
        if (m0 + 16 * MT < rows)
            __syncthreads();  // the sums are read before the next rows' are written
    }
}

}  // namespace ep
