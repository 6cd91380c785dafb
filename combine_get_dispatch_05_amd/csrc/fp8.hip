// fp8.hip -- products of FP8 (e4m3) operands with an fp32 scale for each block
// of 128, and the experts' gated feed-forward on low-latency cells in FP8:
//   D[m, n] = sum_b sq[m, b] sp[n / 128, b] sum_{k in block b} q[m, k] p[n, k].
// One matrix instruction sums exactly one block of K (16 x 16 x 128), so the
// scales are applied once a step to its fp32 result.
#include "few_rows.h"

namespace ep {

namespace {

// act = silu(g) u of one 128-column block per row, as codes and a scale: amax
// over the block's WN waves through LDS, then code = e4m3(a * (448 / amax)),
// scale = amax / 448, the format of the FP8 dispatch.
struct GatedFp8Out {
    static constexpr bool kBlockWide = true;
    uint8_t *codes;  // [.][I]
    float *scales;   // [.][I / 128]
    // mbase: this wave's first row inside the tile; ROWS: rows of the tile
    template <int MT, int NW, int WN, int ROWS>
    __device__ __forceinline__ void store_block(const Tile &t, int64_t start, int wn, int mbase, int n0, int I,
                                                f32x4 (&acc)[MT][NW], int lane) const
    {
        __shared__ float amaxs[WN][ROWS];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float big = 0.0f;
#pragma unroll
            for (int i = 0; i < NW / 2; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float g = acc[m][i][k];
                    const float v = g * sigmoidf(g) * acc[m][i + NW / 2][k];
                    acc[m][i][k] = v;
                    big = fmaxf(big, fabsf(v));
                }
            }
            big = fmaxf(big, __shfl_xor(big, 16));
            big = fmaxf(big, __shfl_xor(big, 32));
            if (lane < 16)
                amaxs[wn][mbase + m * 16 + lane] = big;
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = mbase + m * 16 + (lane & 15);
            if (t.m0 + r >= t.rows)
                continue;
            float amax = amaxs[0][r];
#pragma unroll
            for (int w = 1; w < WN; ++w)
                amax = fmaxf(amax, amaxs[w][r]);
            amax = amax < 1e-4f ? 1e-4f : amax;
            const float inv = 448.0f / amax;
            const int64_t row = start + t.m0 + r;
            if (wn == 0 && lane < 16)
                scales[row * (I >> 7) + (n0 >> 7)] = amax / 448.0f;
#pragma unroll
            for (int i = 0; i < NW / 2; ++i) {
                const f32x4 v = acc[m][i] * inv;
                int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
                c = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], c, true);
                *reinterpret_cast<int *>(codes + row * I + n0 + i * 16 + (lane >> 4) * 4) = c;
            }
        }
    }
};

// BM rows of one group by BN columns: the bf16 tile kernel's loop with K steps of
// one scale block, a tile a block (working through tiles takes registers that
// the scaled sums need).  The step's scales are staged behind
// the rows, one load a wave, so that every wave counts the same loads: waves 0
// to 3 the BM token scales (some twice where BM is 64), the others the two
// weight scales of the tile: its column blocks, or its gate and its up block.
// 8192 x 4096 x 7168: 232 us, 2.07 PFLOP/s (the FP8 product of equal 8192 x 8192 x
// 8192 matrices reaches 3.2 on the same card), bound by the scaled sums, which take
// vector instructions that the matrix cores wait for.  64 experts of 2048 x 7168 with
// 128 rows each: 0.52 and 0.30 ms, 3.0 GB at 3.6 TB/s.
// WIDEN: both operands to bf16 first, as in few_rows.h.
template <int BM, bool WIDEN, Form F, class Epi>
__global__ __launch_bounds__(NT) void fp8_tile_kernel(FewArgs a, Groups G, Epi epi)
{
    using QS = NearRowStage<BM, NT>;
    using PR = NearRowStage<BN, NT>;
    constexpr int kP = PR::kBytes, kQ = QS::kBytes, kStage = kP + kQ + (BM + kWave) * 4, ST = BM == 256 ? 2 : 3;
    typedef const __attribute__((address_space(3))) float lds_float;
    __shared__ __attribute__((aligned(128))) char smem[ST * kStage];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    lds_char *lds = (lds_char *)smem;
    const int steps = a.kbytes >> 7;
    const int sdst = kP + kQ + (wave < 4 ? wave % (BM / kWave) : BM / kWave) * kWave * 4;
    auto stage = [&](int s) -> lds_char * { return lds + (ST == 2 ? s & 1 : s % ST) * kStage; };

    QS qs;
    PR pr;
    const char *sq = nullptr;  // this lane's scale
    auto set_up = [&](const Tile &t) {
        const int64_t start = group_start(G, t.group);
        const int e = group_expert(G, t.group);
        const int n0 = t.n * (F == Form::kGated ? BN / 2 : BN);
        qs.init(tid, a.q + (start + t.m0) * a.ldq, [&](int, int r) {
            const int last = t.rows - 1 - t.m0;
            return uint32_t(r < last ? r : last) * uint32_t(a.ldq);
        });
        const bool up = F == Form::kGated && wave >= 4;  // as in the bf16 tile
        pr.init(tid, a.p + int64_t(e) * a.p_expert + (int64_t(n0) + (up ? a.N : 0)) * a.ldp, [&](int, int r) {
            int n = F == Form::kGated ? (r >> 6) * 32 + (r & 31) : r;
            n = n0 + n < a.N ? n : a.N - 1 - n0;
            return uint32_t(n) * uint32_t(a.ldp);
        });
        if (wave < 4) {
            const int m = t.m0 + tid % BM;
            sq = reinterpret_cast<const char *>(a.q_scale + (start + (m < t.rows ? m : t.rows - 1)) * steps);
        } else {
            int nb = n0 + (F == Form::kGated ? 0 : (lane & 1) * 128);
            nb = (nb < a.N ? nb : a.N - 1) >> 7;
            if (F == Form::kGated)
                nb += (lane & 1) * (a.N >> 7);
            sq = reinterpret_cast<const char *>(a.p_scale + e * a.p_scales + int64_t(nb) * steps);
        }
    };
    auto issue = [&](int part, int s) {
        const int64_t kb = int64_t(s) * kStepBytes;
        constexpr int JQ = QS::J > 1 ? 2 : 1;
        lds_char *b = stage(s);
        if (part == 0)
            pr.template issue<false, 0, 2>(b, tid, wave, kb, a.kbytes);
        else if (part == 1)
            pr.template issue<false, 1, 2>(b, tid, wave, kb, a.kbytes);
        else if (part == 2)
            qs.template issue<false, 0, JQ>(b + kP, tid, wave, kb, a.kbytes);
        else {
            if (QS::J > 1)
                qs.template issue<false, 1, JQ>(b + kP, tid, wave, kb, a.kbytes);
            load_lds4(sq + int64_t(s) * 4, b + sdst);
        }
    };
    auto open = [&] {
        if constexpr (ST == 2)
            open_pair(steps, issue);
        else
            open_ring<ST>(steps, issue);
    };

    const Tile cur = find_tile<BM, NT>(G, blockIdx.x, a.nt);
    if (cur.group < 0)
        return;
    set_up(cur);
    open();
    at_height<BM>(cur.rows - cur.m0, [&](auto rows_tag) {
        constexpr int R = decltype(rows_tag)::value, MT = R / 32;
        constexpr int MQ = 2, PH = MT / MQ;  // two row tiles a phase
        f32x4 acc[MT][4] = {};
        Frag pf[4], qf[MQ];
        float sc[MQ], c0 = 0.0f, c1 = 0.0f;
        auto read = [&](int s, int ph) {
            const lds_char *pb = stage(s), *qb = pb + kP;
            if (ph == 0) {
                lds_float *w = (lds_float *)(qb + kQ + BM * 4);
                c0 = w[F == Form::kGated ? 0 : wn >> 1];
                c1 = F == Form::kGated ? w[1] : c0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    pf[i] = staged_frag(pb, wn * 64 + i * 16, lane);
            }
#pragma unroll
            for (int m = 0; m < MQ; ++m) {
                const int r = wm * (R / 2) + (ph * MQ + m) * 16 + (lane & 15);
                qf[m] = staged_frag(qb, r - (lane & 15), lane);
                sc[m] = *(lds_float *)(qb + kQ + r * 4);
            }
        };
        auto compute = [&](int, int ph) {
#pragma unroll
            for (int m = 0; m < MQ; ++m) {
                hold(qf[m].lo);
                hold(qf[m].hi);
            }
            float s0[MQ], s1[MQ];
#pragma unroll
            for (int m = 0; m < MQ; ++m) {
                s0[m] = sc[m] * c0;
                s1[m] = F == Form::kGated ? sc[m] * c1 : s0[m];
            }
            if constexpr (WIDEN) {
                Wide q[MQ];
#pragma unroll
                for (int m = 0; m < MQ; ++m)
                    q[m] = widen(qf[m]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const Wide p = widen(pf[i]);
#pragma unroll
                    for (int m = 0; m < MQ; ++m)
                        acc[ph * MQ + m][i] += mfma_step_wide(p, q[m]) * (i < 2 ? s0[m] : s1[m]);
                }
            } else {
#pragma unroll
                for (int m = 0; m < MQ; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[ph * MQ + m][i] += mfma_step_fp8(pf[i], qf[m]) * (i < 2 ? s0[m] : s1[m]);
            }
#pragma unroll
            for (int m = 0; m < MQ; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    hold(acc[ph * MQ + m][i]);
        };
        if constexpr (ST == 2)
            turns_on_pair<PH, PR::J>(steps, wm, issue, read, compute);
        else
            turns_on_ring<PH, ST, PR::J + QS::J + 1>(steps, wm, issue, read, compute);
        const int64_t start = group_start(G, cur.group);
        const int n0 = cur.n * (F == Form::kGated ? BN / 2 : BN) + wn * (F == Form::kGated ? 32 : 64);
        if constexpr (Epi::kBlockWide)
            epi.template store_block<MT, 4, 4, R>(cur, start, wn, wm * (R / 2), n0, a.N, acc, lane);
        else
            epi.store(cur, start, cur.m0 + wm * (R / 2), n0, a.N, acc, lane);
    });
}

template <Form F, class Epi>
hipError_t launch_fp8_tiles(FewArgs a, const Groups &G, int64_t rows, int64_t max_tiles, const Epi &epi,
                            const char *what, hipStream_t stream)
{
    const int cols = F == Form::kGated ? BN / 2 : BN;
    a.nt = unsigned((a.N + cols - 1) / cols);
    // widened at 64 rows (so few activations take no other height on a whole card)
    const bool wide = F == Form::kGated && rows * a.N < kFewActivations;
    const int bm = wide ? 64 : tile_rows(rows, max_tiles, a.nt);
    const int64_t mt = row_tiles(rows, max_tiles, bm);
    if (mt * a.nt > kMaxTileBlocks)
        return hipErrorInvalidValue;
    if (mt == 0)
        return hipSuccess;
    if (log_enabled())
        log_launch("%s: rows<=%lld groups=%d N=%d K=%d tile=%dx%d blocks=%lld", what, (long long)rows,
                   G.num, a.N, a.kbytes, bm, BN, (long long)mt * a.nt);
    const dim3 grid(unsigned(blocks_for_tiles(mt * a.nt)));
    if constexpr (F == Form::kGated)
        if (wide) {
            hipLaunchKernelGGL((fp8_tile_kernel<64, true, F, Epi>), grid, dim3(NT), 0, stream, a, G, epi);
            return hipGetLastError();
        }
    if (bm == 256)
        hipLaunchKernelGGL((fp8_tile_kernel<256, false, F, Epi>), grid, dim3(NT), 0, stream, a, G, epi);
    else
        hipLaunchKernelGGL((fp8_tile_kernel<64, false, F, Epi>), grid, dim3(NT), 0, stream, a, G, epi);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_product(int64_t M, int N, int K, const void *a_q, const float *a_scale,
                              const void *w_q, const float *w_scale, void *out, hipStream_t stream)
{
    const Groups G{nullptr, nullptr, int32_t(M), 1, 1, 1, 1, kNoLimit};
    FewArgs a{};
    a.q = static_cast<const char *>(a_q);
    a.q_scale = a_scale;
    a.ldq = K;
    a.p = static_cast<const char *>(w_q);
    a.p_scale = w_scale;
    a.ldp = K;
    a.N = N;
    a.kbytes = K;
    const RowOut epi{static_cast<uint16_t *>(out)};
    a.active = 1;
    // K is split for up to 16 rows (16 x 16384 x 4096: 12.5 us, in 64-row tiles 23.6),
    // past that in a block for each 64 as long as all of them run at once (512 x 2048
    // x 4096, 256 blocks: 12.7 us, in tiles 23.9; 512 x 4096 x 4096, 512 blocks:
    // 24.0 and 24.1).
    const int64_t chunks = (M + 63) / 64;
    if (M <= 16 || chunks * ((N + kSplitCols - 1) / kSplitCols) <= compute_units())
        return launch_split<true, Form::kPlain>(a, G, split_rows<RowOut>(M), int(chunks), epi, "fp8_product", stream);
    return launch_fp8_tiles<Form::kPlain>(a, G, M, 1, epi, "fp8_product", stream);
}

hipError_t launch_ll_expert_ffn_fp8(int E, int R, int slots, int H, int I, int64_t max_pairs,
                                    const int32_t *counts, const void *packed_q,
                                    const float *packed_scale, const void *w13_q,
                                    const float *w13_scale, const void *w2_q, const float *w2_scale,
                                    void *act_q, float *act_scale, void *out, hipStream_t stream)
{
    const Groups G{nullptr, counts, slots, E, R, E / R, 1, kNoLimit};
    FewArgs a{};
    a.q = static_cast<const char *>(packed_q);
    a.q_scale = packed_scale;
    a.ldq = H;
    a.p = static_cast<const char *>(w13_q);
    a.p_scale = w13_scale;
    a.p_expert = int64_t(2) * I * H;
    a.p_scales = int64_t(2) * (I / 128) * (H / 128);
    a.ldp = H;
    a.N = I;
    a.kbytes = H;
    const GatedFp8Out gated{static_cast<uint8_t *>(act_q), act_scale};
    hipError_t e = launch_groups<true, Form::kGated>(
        a, G, max_pairs, slots, gated, "ll_expert_ffn_fp8 gated", stream, [&](const Groups &T, int64_t most) {
            return launch_fp8_tiles<Form::kGated>(a, T, max_pairs, most, gated, "ll_expert_ffn_fp8 gated tiles",
                                                  stream);
        });
    if (e != hipSuccess)
        return e;
    a.q = static_cast<const char *>(act_q);
    a.q_scale = act_scale;
    a.ldq = I;
    a.p = static_cast<const char *>(w2_q);
    a.p_scale = w2_scale;
    a.p_expert = int64_t(I) * H;
    a.p_scales = int64_t(I / 128) * (H / 128);
    a.ldp = I;
    a.N = H;
    a.kbytes = I;
    const RowOut rows{static_cast<uint16_t *>(out)};
    return launch_groups<true, Form::kPlain>(
        a, G, max_pairs, slots, rows, "ll_expert_ffn_fp8 down", stream, [&](const Groups &T, int64_t most) {
            return launch_fp8_tiles<Form::kPlain>(a, T, max_pairs, most, rows, "ll_expert_ffn_fp8 down tiles",
                                                  stream);
        });
}

}  // namespace ep
