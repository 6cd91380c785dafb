// experts.hip -- the experts between a dispatch and its combine, in bf16:
// rows grouped by expert, the gated feed-forward over them, and its gradients.
//
// For pair p = (row, slot) of expert e, with x the row and w its routing weight,
//   g = x Wg^T, u = x Wu^T, a = g sigmoid(g) u, z = a W2^T, y_row += w z
// and, given dy,
//   d = dy W2, dw = a . d, da = w d, du = da silu(g), dg = da u s (1 + g (1 - s)), s = sigmoid(g)
//   dx_row += [dg du] W13, dW13 = sum_p [dg du]^T x, dW2 = sum_p dy^T (w a).
#include "few_rows.h"

namespace ep {

namespace {

// ------------------------------------------------------------- grouping

constexpr int kGroupBlock = 1024;

// Rows of expert e's rank, clamped to the rows that exist.
__device__ __forceinline__ void rank_rows(const int32_t *prefix, int r, int64_t n, int64_t &a,
                                          int64_t &b)
{
    a = r > 0 ? prefix[r - 1] : 0;
    b = prefix[r];
    a = a < 0 ? 0 : (a < n ? a : n);
    b = b < a ? a : (b < n ? b : n);
}

// A thread takes kIds slots in a row, so that a block of 1024 goes through 8192
// slots between two barriers (one slot a thread took 57 us for 32 experts whose
// ranks hold 32768 slots each).
constexpr int kIds = 8;

// Bit j: slot i + j (before end) names local expert le.
__device__ __forceinline__ unsigned slots_of(const int64_t *ids, int64_t i, int64_t end, int le)
{
    unsigned m = 0;
#pragma unroll
    for (int j = 0; j < kIds; ++j) {
        const int64_t v = i + j < end ? ids[i + j] : -1;
        m |= unsigned(v == le) << j;
    }
    return m;
}

// One block for each expert counts its pairs; together they also mark every
// (row, slot) as having no pair.  Each reads the whole id table (from L2), which
// for the experts of one node is less than a sort would move: 11 us, and 15 for the
// places, for 21 thousand rows of 8 slots and 32 experts; 3.8 and 6.0 for 3 thousand
// of 6 and 64.
__global__ __launch_bounds__(kGroupBlock) void count_pairs_kernel(
    const int64_t *__restrict__ ids, const int32_t *__restrict__ prefix, int64_t n, int K, int epr,
    int32_t *__restrict__ counts, int32_t *__restrict__ row_pair)
{
    const int e = blockIdx.x, r = e / epr, le = e % epr;
    for (int64_t i = int64_t(e) * kGroupBlock + threadIdx.x; i < n * K;
         i += int64_t(gridDim.x) * kGroupBlock)
        row_pair[i] = -1;
    int64_t a, b;
    rank_rows(prefix, r, n, a, b);
    int c = 0;
    for (int64_t i = a * K + threadIdx.x * kIds; i < b * K; i += kGroupBlock * kIds)
        c += __popc(slots_of(ids, i, b * K, le));
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        c += __shfl_xor(c, d);
    __shared__ int s[kGroupBlock / kWave];
    if ((threadIdx.x & 63) == 0)
        s[threadIdx.x >> 6] = c;
    __syncthreads();
    if (threadIdx.x == 0) {
        int t = 0;
        for (int w = 0; w < kGroupBlock / kWave; ++w)
            t += s[w];
        counts[e] = t;
    }
}

// One block for each expert: its pairs' places, in (row, slot) order behind the
// pairs of the experts before it.
__global__ __launch_bounds__(kGroupBlock) void place_pairs_kernel(
    const int64_t *__restrict__ ids, const int32_t *__restrict__ prefix, int64_t n, int K, int E,
    int epr, const int32_t *__restrict__ counts, int64_t cap, int32_t *__restrict__ offsets,
    int32_t *__restrict__ pair_row, int32_t *__restrict__ pair_slot, int32_t *__restrict__ row_pair)
{
    constexpr int W = kGroupBlock / kWave;
    const int e = blockIdx.x, r = e / epr, le = e % epr;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __shared__ int64_t s[2][W];
    int64_t c = 0;  // the counts of a prefix that is none can add up to more than 2^31
    for (int i = threadIdx.x; i < e; i += kGroupBlock)
        c += counts[i];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        c += __shfl_xor(c, d);
    if (lane == 0)
        s[1][wave] = c;
    __syncthreads();
    int64_t base = 0;
    for (int w = 0; w < W; ++w)
        base += s[1][w];
    // a count past the capacity (ids that no dispatch wrote) leaves the tail out
    if (threadIdx.x == 0) {
        offsets[e] = int32_t(base < cap ? base : cap);
        if (e == E - 1) {
            const int64_t end = base + counts[e];
            offsets[E] = int32_t(end < cap ? end : cap);
        }
    }
    int64_t a, b;
    rank_rows(prefix, r, n, a, b);
    int flip = 0;
    for (int64_t i0 = a * K; i0 < b * K; i0 += kGroupBlock * kIds, flip ^= 1) {
        const int64_t i = i0 + threadIdx.x * kIds;
        unsigned hits = slots_of(ids, i, b * K, le);
        const int mine = __popc(hits);
        int pre = mine;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int o = __shfl_up(pre, d);
            pre += lane >= d ? o : 0;
        }
        if (lane == 63)
            s[flip][wave] = pre;
        __syncthreads();  // two rows of s in turn: the next round but one writes this one again
        int before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int v = int(s[flip][w]);
            before += w < wave ? v : 0;
            total += v;
        }
        for (int64_t pos = base + before + pre - mine; hits != 0 && pos < cap; ++pos) {
            const int64_t at = i + __ffs(hits) - 1;
            hits &= hits - 1;
            const int64_t row = at / K;
            int live = 0;
            for (int k = 0; k < K; ++k) {
                const int64_t v = ids[row * K + k];
                live += v >= 0 && v < epr;
            }
            pair_row[pos] = int32_t(row) | (live == 1 ? int32_t(0x80000000u) : 0);
            pair_slot[pos] = int32_t(at);
            row_pair[at] = int32_t(pos);
        }
        base += total;
    }
}

// --------------------------------------------------------- tile epilogues
//
// Each is called by every thread with its accumulators acc[mt][nt] (row
// m0 + mt * 16 + lane % 16, columns n0 + nt * 16 + 4 (lane / 16) .. + 3).

// Rows of a pair's product: the only pair of its row goes straight to the
// row's bf16 output (rounded once), a row of several keeps fp32 terms for the
// sum that follows.  weight: routing weights by pair slot (nullable).
struct PairOut {
    static constexpr bool kBlockWide = false;
    const int32_t *pair_row, *pair_slot;
    const float *weight;
    uint16_t *out;  // [rows][N]
    float *terms;   // [pairs][N]
    template <int MT, int NW>
    __device__ __forceinline__ void store(const Tile &t, int64_t start, int m0, int n0, int N,
                                          const f32x4 (&acc)[MT][NW], int lane) const
    {
        // every row's place and weight before the first store: a load behind a store
        // waits for it, and eight such waits a tile took longer than the stores
        int32_t r[MT];
        float w[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = m0 + mt * 16 + (lane & 15);
            r[mt] = m < t.rows ? pair_row[start + m] : 0;
            w[mt] = m < t.rows && weight != nullptr ? weight[pair_slot[start + m]] : 1.0f;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = m0 + mt * 16 + (lane & 15);
            f32x4 v[NW];
#pragma unroll
            for (int nt = 0; nt < NW; ++nt) {
                v[nt] = acc[mt][nt] * w[mt];
                const int n = n0 + nt * 16 + (lane >> 4) * 4;
                if (m < t.rows && r[mt] >= 0 && n < N)
                    *reinterpret_cast<f32x4 *>(terms + (start + m) * N + n) = v[nt];
            }
            store_bf16_row<NW>(r[mt] < 0 ? out + int64_t(r[mt] & kRowMask) * N : nullptr, n0, N, v, lane);
        }
    }
};

// Gate and up columns in one tile: act = silu(g) u in bf16 (what the second
// product's matrix instructions take: its rounding adds to the result what the output's
// own does, 2.3e-3 of the norm off 64 bits instead of 1.7e-3, and a second bf16 for the
// rest would double that product) and, for a backward pass, g and u in
// fp32: the routing weights' gradient is an fp32 result that bf16 copies would
// hold to three digits.
struct GatedOut {
    static constexpr bool kBlockWide = false;
    uint16_t *act;  // [.][I]
    float *gu;      // [.][2 I], nullable
    template <int MT, int NW>
    __device__ __forceinline__ void store(const Tile &t, int64_t start, int m0, int n0, int I,
                                          const f32x4 (&acc)[MT][NW], int lane) const
    {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = m0 + mt * 16 + (lane & 15);
            const bool live = m < t.rows;
            const int64_t p = start + m;
            f32x4 a[NW / 2];
#pragma unroll
            for (int nt = 0; nt < NW / 2; ++nt) {
                const int n = n0 + nt * 16 + (lane >> 4) * 4;
                const f32x4 g = acc[mt][nt], u = acc[mt][nt + NW / 2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a[nt][i] = g[i] * sigmoidf(g[i]) * u[i];
                if (gu != nullptr && live && n < I) {
                    *reinterpret_cast<f32x4 *>(gu + p * 2 * I + n) = g;
                    *reinterpret_cast<f32x4 *>(gu + p * 2 * I + I + n) = u;
                }
            }
            store_bf16_row<NW / 2>(live ? act + p * I : nullptr, n0, I, a, lane);
        }
    }
};

// d = dy W2 in the accumulators: the gate's backward and the weighted activation
// for dW2, both in bf16 as the products behind take them (the gradients are then as
// far off as the outputs), and the tile's share of the routing weight's gradient, summed in a
// fixed order over lanes, then waves, then (in rows_kernel) tiles.
struct GatedBack {
    static constexpr bool kBlockWide = true;
    const int32_t *pair_slot;
    const float *weight;
    const float *gu;      // [pairs][2 I]
    uint16_t *dgu;        // [pairs][2 I]
    uint16_t *wact;       // [pairs][I]
    float *dweight_part;  // [pairs][tiles]
    int tiles;
    // mbase: the wave's first row inside the tile of ROWS rows
    template <int MT, int NW, int WN, int ROWS>
    __device__ __forceinline__ void store_block(const Tile &t, int64_t start, int wn, int mbase, int n0, int I,
                                                f32x4 (&acc)[MT][NW], int lane) const
    {
        __shared__ float part[WN][ROWS];
        const int tid = threadIdx.x;
        float w[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = t.m0 + mbase + mt * 16 + (lane & 15);
            w[mt] = m < t.rows ? weight[pair_slot[start + m]] : 0.0f;
        }
        // g and u two column tiles at a time, the next two on their way before these
        // are stored (a load behind a store waits for it)
        f32x4 g[2][2], u[2][2];
        auto load = [&](int i) {
            const int m = t.m0 + mbase + (i >> 1) * 16 + (lane & 15);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int n = n0 + ((i & 1) * 2 + k) * 16 + (lane >> 4) * 4;
                const bool in = m < t.rows && n < I;
                const float *at = gu + (start + m) * 2 * I + n;
                g[i & 1][k] = in ? *reinterpret_cast<const f32x4 *>(at) : f32x4{};
                u[i & 1][k] = in ? *reinterpret_cast<const f32x4 *>(at + I) : f32x4{};
            }
        };
        static_assert(NW == 4, "two pairs of column tiles");
        load(0);
        float dw = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int mt = i >> 1, h = (i & 1) * 2, m = t.m0 + mbase + mt * 16 + (lane & 15);
            const bool live = m < t.rows;
            const int64_t p = start + m;
            if (i + 1 < 2 * MT)
                load(i + 1);
            f32x4 dg[2], du[2], wa[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const bool in = live && n0 + (h + k) * 16 + (lane >> 4) * 4 < I;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float gv = g[i & 1][k][j], uv = u[i & 1][k][j], d = acc[mt][h + k][j];
                    const float sg = sigmoidf(gv), si = gv * sg;
                    dw += in ? si * uv * d : 0.0f;
                    wa[k][j] = w[mt] * si * uv;
                    du[k][j] = w[mt] * d * si;
                    dg[k][j] = w[mt] * d * uv * sg * (1.0f + gv * (1.0f - sg));
                }
            }
            store_bf16_row<2>(live ? dgu + p * 2 * I : nullptr, n0 + h * 16, I, dg, lane);
            store_bf16_row<2>(live ? dgu + p * 2 * I + I : nullptr, n0 + h * 16, I, du, lane);
            store_bf16_row<2>(live ? wact + p * I : nullptr, n0 + h * 16, I, wa, lane);
            if (i & 1) {
                dw += __shfl_xor(dw, 16);
                dw += __shfl_xor(dw, 32);
                if (lane < 16)
                    part[wn][mbase + mt * 16 + lane] = dw;
                dw = 0.0f;
            }
            __builtin_amdgcn_sched_barrier(0);  // one at a time: more would not fit the registers
        }
        __syncthreads();
        if (tid < ROWS && t.m0 + tid < t.rows)
            dweight_part[(start + t.m0 + tid) * tiles + t.n] =
                (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
    }
};

// ------------------------------------------------------------ tile kernels

// Tiles of BM rows of one group by BN columns, with as many LDS stages as fit.
// A block works through every gridDim.x-th tile: it looks up the next one while
// the first stage of this one arrives, and sends off the next one's first stage
// before it stores this one.  At 32 experts of 2048 x 7168 with about 1024 rows each
// the gated product takes 1.77 ms (1090 TFLOP/s; the product of equal 8192 x 8192 x
// 8192 matrices reaches 1620 on the same card), the down product 1.05, the gate's
// backward 1.28, dx 1.89: the values themselves (on zeros 8 to 12 % less) and the wait
// for a stage's loads, which two stages of 64 KB do not hide, are what is left.  At 256
// rows the next tile is set up while 128 accumulators a lane wait to be stored, and
// registers run out there: the gate's backward spills 141 vector registers (232 bytes a
// lane), dx 6, and each of these kernels 54 to 144 scalar ones.  The K loops are free of it.
template <int BM, bool PCOL, Form F, class Epi>
__global__ __launch_bounds__(NT) void tile_kernel(TileArgs a, Groups G, Epi epi)
{
    using QS = RowStage<BM, NT>;
    using PR = NearRowStage<BN, NT>;
    using PC = ColStage<BN, NT>;
    constexpr int kP = PR::kBytes, kStage = kP + QS::kBytes, ST = BM == 256 ? 2 : 3;
    __shared__ __attribute__((aligned(128))) char smem[ST * kStage];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    lds_char *lds = (lds_char *)smem;
    const int steps = (a.K + 63) / 64;
    const int64_t kbytes = int64_t(a.K) * 2;
    auto stage = [&](int s) -> lds_char * { return lds + (ST == 2 ? s & 1 : s % ST) * kStage; };

    QS qs;
    PR pr;
    PC pc;
    const char *pw = nullptr;
    int row_at[QS::J];  // places of this thread's rows
    auto find_rows = [&](const Tile &t) {
        const int64_t start = group_start(G, t.group);
#pragma unroll
        for (int j = 0; j < QS::J; ++j) {
            int m = t.m0 + ((j * NT + tid) >> 3);
            m = m < t.rows ? m : t.rows - 1;
            row_at[j] = a.q_rows != nullptr ? a.q_rows[start + m] & kRowMask : m;
        }
    };
    auto set_up = [&](const Tile &t) {
        const int n0 = t.n * (F == Form::kGated ? BN / 2 : BN);
        pw = a.p + int64_t(group_expert(G, t.group)) * a.p_expert;
        const char *q = a.q_rows != nullptr ? a.q : a.q + group_start(G, t.group) * a.ldq;
        qs.init(tid, [&](int j, int) { return q + int64_t(row_at[j]) * a.ldq; });
        if constexpr (PCOL) {
            pc.init(tid, n0, a.N);
        } else {
            // gated: of each wave's 64 LDS rows 32 are gate columns, 32 their up columns;
            // waves 4 to 7 stage the latter
            const bool up = F == Form::kGated && wave >= 4;
            pr.init(tid, pw + (int64_t(n0) + (up ? a.N : 0)) * a.ldp, [&](int, int r) {
                int n = F == Form::kGated ? (r >> 6) * 32 + (r & 31) : r;
                n = n0 + n < a.N ? n : a.N - 1 - n0;
                return uint32_t(n) * uint32_t(a.ldp);
            });
        }
    };
    auto issue = [&](int part, int s) {
        const int64_t kb = int64_t(s) * kStepBytes;
        constexpr int JP = PR::J / 2, JQ = QS::J > 1 ? QS::J / 2 : 1;
        if (part >= 2) {  // halves of the chunks, or all of them in the first
            if (part == 2)
                qs.template issue<true, 0, QS::J / JQ>(stage(s) + kP, tid, wave, kb, kbytes);
            else if (QS::J > 1)
                qs.template issue<true, 1, QS::J / JQ>(stage(s) + kP, tid, wave, kb, kbytes);
        } else if constexpr (PCOL) {
            if (part == 0)
                pc.template issue<0, JP>(stage(s), tid, wave, pw, a.ldp, s * 64, a.K);
            else
                pc.template issue<JP, JP>(stage(s), tid, wave, pw, a.ldp, s * 64, a.K);
        } else {
            if (part == 0)
                pr.template issue<true, 0, 2>(stage(s), tid, wave, kb, kbytes);
            else
                pr.template issue<true, 1, 2>(stage(s), tid, wave, kb, kbytes);
        }
    };
    auto open = [&] {
        if constexpr (ST == 2)
            open_pair(steps, issue);
        else
            open_ring<ST>(steps, issue);
    };
    unsigned block = blockIdx.x;
    Tile t = find_tile<BM, NT>(G, block, a.nt);
    if (t.group < 0)
        return;
    find_rows(t);
    set_up(t);
    open();
    auto work = [&](auto rows_tag) {
        constexpr int R = decltype(rows_tag)::value, MT = R / 32;  // rows computed, row tiles of a wave
        const int ln = here(lane);  // the LDS addresses of one height at a time
        auto frag_p = [&](int s, int i, int ks) {
            const int c = wn * 64 + i * 16;
            if constexpr (PCOL)
                return PC::frag(stage(s), c, ks, ln);
            else
                return PR::frag(stage(s), c, ks, ln);
        };
        auto frag_q = [&](int s, int m, int ks) {
            return QS::frag(stage(s) + kP, wm * (R / 2) + m * 16, ks, ln);
        };
        f32x4 acc[MT][4] = {};
        using Phases = Bf16Phases<MT, decltype(frag_p), decltype(frag_q)>;
        Phases ph{acc, frag_p, frag_q};
        auto read = [&](int s, int i) { ph.read(s, i); };
        auto compute = [&](int, int i) { ph.compute(i); };
        if constexpr (ST == 2)
            turns_on_pair<Phases::kPhases, PR::J>(steps, wm, issue, read, compute);
        else
            turns_on_ring<Phases::kPhases, ST, PR::J + QS::J>(steps, wm, issue, read, compute);
        return [&, acc](const Tile &c) mutable {
            const int64_t start = group_start(G, c.group);
            const int n0 = c.n * (F == Form::kGated ? BN / 2 : BN) + wn * (F == Form::kGated ? 32 : 64);
            if constexpr (Epi::kBlockWide)
                epi.template store_block<MT, 4, 4, R>(c, start, wn, wm * (R / 2), n0, a.N, acc, lane);
            else
                epi.store(c, start, c.m0 + wm * (R / 2), n0, a.N, acc, lane);
        };
    };
    for (;;) {
        block += gridDim.x;
        const Tile next = block < a.blocks ? find_tile<BM, NT>(G, block, a.nt) : Tile{-1, 0, 0, 0};
        if (next.group >= 0)
            find_rows(next);
        const Tile cur = t;
        auto finish = [&](auto store) {
            if (next.group >= 0) {
                set_up(next);
                open();
            }
            store(cur);
        };
        at_height<BM>(cur.rows - cur.m0, [&](auto rows) { finish(work(rows)); });
        if (next.group < 0)
            break;
        t = next;
    }
}

// out[e][m][n] = sum over the group's rows k of Q[k][m] P[k][n], 256 x 256 a
// tile; QG / PG: the operand's rows are picked by pair_row.  A group without
// rows writes zeros.  Blocks work through the tiles as in tile_kernel.
struct GradArgs {
    const char *q, *p;
    int64_t ldq, ldp;  // bytes of a row
    const int32_t *pair_row, *offsets;
    int experts, M, N;
    unsigned mt, nt;
    uint16_t *out;
};

constexpr int kPickSlots = 10;
constexpr int kGradLds = 4 * ColStage<256, NT>::kBytes + NT / kWave * kPickSlots * kWave * 4;

// Tiles block, block + gridDim.x, ... of one gradient.
template <bool QG, bool PG>
__device__ __forceinline__ void weight_grad(const GradArgs &a, lds_char *lds, unsigned block)
{
    constexpr int B = 256;
    using CS = ColStage<B, NT>;
    // Each wave keeps the stages' 64 picked rows to itself, three stages ahead,
    // loaded straight into LDS like the stages: held in registers their copies
    // from stage to stage waited for the loads (46 us a tile of 1024 rows; this way
    // 40, its stores among them).  Slots 0 to 3 go round; a tile's first three stages
    // have slots of their own, filled while the tile before is worked on, for which
    // tiles take turns with two sets.
    constexpr int kSlot = kWave * 4;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    lds_char *picks = lds + 4 * CS::kBytes + wave * kPickSlots * kSlot;
    const unsigned per = a.mt * a.nt, total = per * unsigned(a.experts);

    struct Place {
        unsigned e, tm, tn;
        int start, rows;
    };
    auto place = [&](unsigned block) {
        Place t;
        const unsigned id = unsigned(share_of_xcd(total, block % kXcds, block / kXcds));
        t.e = id / per;
        tile_in_bands(id % per, a.mt, a.nt, t.tm, t.tn);
        t.start = uniform(a.offsets[t.e]);
        t.rows = uniform(a.offsets[t.e + 1]) - t.start;
        return t;
    };
    auto pick = [&](const Place &t, int s, int slot) {  // the rows of stage s of tile t
        const int k = s * 64 + lane;
        load_lds4(reinterpret_cast<const char *>(a.pair_row + t.start + (k < t.rows ? k : t.rows - 1)),
                  picks + slot * kSlot);
    };

    CS qs, ps;
    Place t;
    int steps = 0, set = 0;
    int idx[CS::J];  // picked rows, read from LDS a phase before their first use
    auto slot = [&](int s) { return s < 3 ? 4 + set * 3 + s : s & 3; };
    auto stage = [&](int s) -> lds_char * { return lds + (s & 1) * 2 * CS::kBytes; };
    auto issue = [&](int part, int s) {
        constexpr int JH = CS::J / 2;
        auto read_picks = [&](int of) {
            const lds_char *from = picks + slot(of) * kSlot;
#pragma unroll
            for (int j = 0; j < CS::J; ++j)
                idx[j] = *(const __attribute__((address_space(3))) int *)(from + CS::k_of(tid, j) * 4);
        };
        if (PG && part == 0 && s < 2)
            read_picks(s);
        const char *p = a.p + (PG ? 0 : t.start * a.ldp), *q = a.q + (QG ? 0 : t.start * a.ldq);
        lds_char *pb = stage(s), *qb = pb + CS::kBytes;
        auto half = [&](CS &c, auto first, lds_char *to, const char *from, int64_t ld, auto gathered) {
            constexpr int J0 = decltype(first)::value * JH;
            if constexpr (decltype(gathered)::value != 0)
                c.template issue<J0, JH>(to, tid, wave, from, ld, s * 64, t.rows, idx);
            else
                c.template issue<J0, JH>(to, tid, wave, from, ld, s * 64, t.rows);
        };
        if (part == 0 && s + 1 < steps && s >= 2)
            pick(t, s + 1, slot(s + 1));  // used a stage from now: this is phase 2 of stage s - 2
        if (part == 0)
            half(ps, Rows<0>{}, pb, p, a.ldp, Rows<PG>{});
        else if (part == 1)
            half(ps, Rows<1>{}, pb, p, a.ldp, Rows<PG>{});
        else if (part == 2)
            half(qs, Rows<0>{}, qb, q, a.ldq, Rows<QG>{});
        else
            half(qs, Rows<1>{}, qb, q, a.ldq, Rows<QG>{});
        if (QG && part == 1)
            read_picks(s);  // for Q of this stage, the next parts
        if (PG && part == 3 && s > 0 && s + 1 < steps)
            read_picks(s + 1);  // for P of the next one
    };
    auto pick_first = [&](const Place &next, int to) {
#pragma unroll
        for (int s = 0; s < 3; ++s)
            if (s * 64 < next.rows)
                pick(next, s, 4 + to * 3 + s);
    };
    auto set_up = [&](const Place &next) {  // its first rows have been picked and have landed
        t = next;
        steps = (t.rows + 63) / 64;
        qs.init(tid, int(t.tm) * B, a.M);
        ps.init(tid, int(t.tn) * B, a.N);
        if (steps > 0)
            open_pair(steps, issue);
    };
    if (block >= total)
        return;
    const Place first = place(block);
    pick_first(first, 0);
    landed<0>();
    set_up(first);
    for (;;) {
        const Place cur = t;
        block += gridDim.x;
        Place next = cur;
        if (block < total) {
            next = place(block);
            pick_first(next, set ^ 1);
        }
        auto frag_p = [&](int s, int i, int ks) { return CS::frag(stage(s), wn * 64 + i * 16, ks, lane); };
        auto frag_q = [&](int s, int m, int ks) {
            return CS::frag(stage(s) + CS::kBytes, wm * 128 + m * 16, ks, lane);
        };
        f32x4 acc[8][4] = {};
        Bf16Phases<8, decltype(frag_p), decltype(frag_q)> ph{acc, frag_p, frag_q};
        // (the pick sent off with P makes one load more in flight than P's: the
        // wait for all but P's reaches it too, which is in time)
        turns_on_pair<4, CS::J>(
            steps, wm, issue, [&](int s, int i) { ph.read(s, i); }, [&](int, int i) { ph.compute(i); });
        set ^= 1;
        if (block < total)
            set_up(next);
        uint16_t *o = a.out + int64_t(cur.e) * a.M * a.N;
        const int m0 = int(cur.tm) * B + wm * 128, n0 = int(cur.tn) * B + wn * 64;
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const int mm = m0 + m * 16 + (lane & 15);
            store_bf16_row<4>(mm < a.M ? o + int64_t(mm) * a.N : nullptr, n0, a.N, acc[m], lane);
        }
        if (block >= total)
            break;
    }
}

// Both weight gradients: dW2 (rows of dy picked), then dW13 (rows of x picked), so
// that the second fills what the first leaves idle at its end.  Its tiles start
// at the block after the first's last.  (The 32 experts above: 3.4 ms, 860 TFLOP/s;
// K is a group's rows, and both operands come through the transposing read.  16 vector
// registers are spilled between tiles.)
__global__ __launch_bounds__(NT) void weight_grads_kernel(GradArgs dw2, GradArgs dw13)
{
    __shared__ __attribute__((aligned(128))) char smem[kGradLds];
    lds_char *lds = (lds_char *)smem;
    weight_grad<true, false>(dw2, lds, blockIdx.x);
    __syncthreads();  // the first's last reads of its picks
    const unsigned used = (dw2.mt * dw2.nt * unsigned(dw2.experts) + kXcds - 1) / kXcds * kXcds % gridDim.x;
    weight_grad<false, true>(dw13, lds, (blockIdx.x + gridDim.x - used) % gridDim.x);
}

// ------------------------------------------------------------ row sums

// Rows with no pair (zero) or several (their fp32 terms in slot order); rows of
// one pair are already written.  With parts: also every slot's routing-weight
// gradient, the sum of its pair's column tiles in order.  Bound by HBM (21 thousand
// rows of 7168: 158 us).
__global__ __launch_bounds__(256) void rows_kernel(const int32_t *__restrict__ row_pair, int64_t rows, int K, int N,
                                                   const int32_t *__restrict__ pair_row,
                                                   const float *__restrict__ terms,
                                                   uint16_t *__restrict__ out,
                                                   const float *__restrict__ parts, int tiles,
                                                   float *__restrict__ dweight)
{
    const int64_t row = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    if (row >= rows)
        return;
    __shared__ int pairs[kMaxTopk];
    __shared__ int live;
    const int tid = threadIdx.x;
    if (tid < kWave) {
        const int p = tid < K ? row_pair[row * K + tid] : -1;
        const uint64_t m = wave_ballot(p >= 0);
        if (p >= 0)
            pairs[__popcll(m & lanemask_lt())] = p;
        if (tid == 0)
            live = __popcll(m);
        if (dweight != nullptr && tid < K) {
            float d = 0.0f;
            if (p >= 0)
                for (int t = 0; t < tiles; ++t)
                    d += parts[int64_t(p) * tiles + t];
            dweight[row * K + tid] = d;
        }
    }
    __syncthreads();
    const int n = live;
    if (n == 1 && pair_row[pairs[0]] < 0)
        return;
    for (int c = tid * 4; c < N; c += 1024) {
        f32x4 v = {};
        for (int k = 0; k < n; ++k)
            v += *reinterpret_cast<const f32x4 *>(terms + int64_t(pairs[k]) * N + c);
        typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
        const uint2 b = pack4(v);
        __builtin_nontemporal_store(u32x2{b.x, b.y}, reinterpret_cast<u32x2 *>(out + row * N + c));
    }
}

// --------------------------------------------------------------- launches

template <bool PCOL, Form F, class Epi>
hipError_t launch_tiles(TileArgs a, const Groups &G, int64_t rows, int64_t groups, const Epi &epi,
                        const char *what, hipStream_t stream)
{
    const int cols = F == Form::kGated ? BN / 2 : BN;
    a.nt = unsigned((a.N + cols - 1) / cols);
    const int bm = tile_rows(rows, groups, a.nt);
    const int64_t mt = row_tiles(rows, groups, bm);
    if (mt * a.nt > kMaxTileBlocks)
        return hipErrorInvalidValue;
    if (mt == 0)
        return hipSuccess;
    if (log_enabled())
        log_launch("%s: rows<=%lld groups=%d N=%d K=%d tile=%dx%d blocks=%lld", what,
                   (long long)rows, G.num, a.N, a.K, bm, BN, (long long)mt * a.nt);
    const int64_t cus = compute_units(), all = blocks_for_tiles(mt * a.nt);
    const dim3 grid(unsigned(all < cus ? all : cus));
    a.blocks = unsigned(all);
    if (bm == 256)
        hipLaunchKernelGGL((tile_kernel<256, PCOL, F, Epi>), grid, dim3(NT), 0, stream, a, G, epi);
    else
        hipLaunchKernelGGL((tile_kernel<64, PCOL, F, Epi>), grid, dim3(NT), 0, stream, a, G, epi);
    return hipGetLastError();
}

// A forward product: K split or tiles.
template <Form F, class Epi>
hipError_t launch_bf16(const FewArgs &a, const Groups &G, int64_t pairs, int64_t most_rows, const Epi &epi,
                       const char *what, hipStream_t stream)
{
    return launch_groups<false, F>(a, G, pairs, most_rows, epi, what, stream, [&](const Groups &T, int64_t most) {
        TileArgs t{};
        t.q = a.q;
        t.q_rows = a.q_rows;
        t.ldq = a.ldq;
        t.p = a.p;
        t.p_expert = a.p_expert;
        t.ldp = a.ldp;
        t.N = a.N;
        t.K = a.kbytes / 2;
        return launch_tiles<false, F>(t, T, pairs, most, epi, what, stream);
    });
}

// The products with w13 and with w2.
FewArgs gated_args(const void *x, const void *w13, int H, int I)
{
    FewArgs a{};
    a.q = static_cast<const char *>(x);
    a.ldq = int64_t(H) * 2;
    a.p = static_cast<const char *>(w13);
    a.p_expert = int64_t(2) * I * H * 2;
    a.ldp = int64_t(H) * 2;
    a.N = I;
    a.kbytes = H * 2;
    return a;
}
FewArgs down_args(const void *act, const void *w2, int H, int I)
{
    FewArgs a{};
    a.q = static_cast<const char *>(act);
    a.ldq = int64_t(I) * 2;
    a.p = static_cast<const char *>(w2);
    a.p_expert = int64_t(I) * H * 2;
    a.ldp = int64_t(I) * 2;
    a.N = H;
    a.kbytes = I * 2;
    return a;
}

Groups contiguous(const int32_t *offsets, int num)
{
    return Groups{offsets, nullptr, 0, num, 1, num, 1, kNoLimit};
}

hipError_t launch_rows(const ExpertFfn &f, const float *terms, void *out, const float *parts, int tiles,
                       float *dweight, hipStream_t stream)
{
    if (f.rows == 0)
        return hipSuccess;
    if (log_enabled())
        log_launch("expert rows sum: rows=%lld H=%d K=%d", (long long)f.rows, f.hidden, f.topk);
    hipLaunchKernelGGL(rows_kernel, row_grid(f.rows), dim3(256), 0, stream, f.row_pair, f.rows, f.topk,
                       f.hidden, f.pair_row, terms, static_cast<uint16_t *>(out), parts, tiles, dweight);
    return hipGetLastError();
}

}  // namespace

int compute_units()
{
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < kXcds)
        return 256;
    return n / kXcds * kXcds;  // whole rounds of the XCDs: a block stays with one run of tiles
}

int expert_ffn_tiles(int inter) { return (inter + BN - 1) / BN; }

hipError_t launch_expert_rows(int E, int epr, int K, int64_t rows, const int32_t *prefix,
                              const int64_t *ids, int64_t cap, int32_t *counts, int32_t *offsets,
                              int32_t *pair_row, int32_t *pair_slot, int32_t *row_pair,
                              hipStream_t stream)
{
    if (log_enabled())
        log_launch("expert_rows: rows=%lld K=%d E=%d blocks=%d x 2", (long long)rows, K, E, E);
    hipLaunchKernelGGL(count_pairs_kernel, dim3(E), dim3(kGroupBlock), 0, stream, ids, prefix, rows, K,
                       epr, counts, row_pair);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(place_pairs_kernel, dim3(E), dim3(kGroupBlock), 0, stream, ids, prefix, rows, K,
                       E, epr, counts, cap, offsets, pair_row, pair_slot, row_pair);
    return hipGetLastError();
}

hipError_t launch_expert_ffn(const ExpertFfn &f, const void *x, const void *w13, const void *w2,
                             void *act, float *gate_up, float *terms, void *y, hipStream_t stream)
{
    const int H = f.hidden, I = f.inter;
    const Groups G = contiguous(f.offsets, f.experts);
    const int64_t most_rows = f.pairs / f.topk;  // the batch's tokens: each has one row with an expert
    FewArgs a = gated_args(x, w13, H, I);
    a.q_rows = f.pair_row;
    hipError_t e = launch_bf16<Form::kGated>(
        a, G, f.pairs, most_rows, GatedOut{static_cast<uint16_t *>(act), gate_up}, "expert_ffn gated", stream);
    if (e != hipSuccess)
        return e;
    e = launch_bf16<Form::kPlain>(down_args(act, w2, H, I), G, f.pairs, most_rows,
                                  PairOut{f.pair_row, f.pair_slot, f.weights, static_cast<uint16_t *>(y), terms},
                                  "expert_ffn down", stream);
    if (e != hipSuccess)
        return e;
    return launch_rows(f, terms, y, nullptr, 0, nullptr, stream);
}

hipError_t launch_expert_ffn_backward(const ExpertFfn &f, const void *dy, const void *x, const void *w13,
                                      const void *w2, const float *gate_up, void *dgu, void *wact,
                                      float *parts, float *terms, void *dx, float *dweight, void *dw13,
                                      void *dw2, hipStream_t stream)
{
    const int H = f.hidden, I = f.inter, tiles = expert_ffn_tiles(I);
    const Groups G = contiguous(f.offsets, f.experts);
    TileArgs a{};
    a.q = static_cast<const char *>(dy);
    a.q_rows = f.pair_row;
    a.ldq = int64_t(H) * 2;
    a.p = static_cast<const char *>(w2);
    a.p_expert = int64_t(I) * H * 2;
    a.ldp = int64_t(I) * 2;
    a.N = I;
    a.K = H;
    hipError_t e = launch_tiles<true, Form::kBack>(
        a, G, f.pairs, f.experts,
        GatedBack{f.pair_slot, f.weights, gate_up, static_cast<uint16_t *>(dgu),
                  static_cast<uint16_t *>(wact), parts, tiles},
        "expert_ffn gate backward", stream);
    if (e != hipSuccess)
        return e;
    a.q = static_cast<const char *>(dgu);
    a.q_rows = nullptr;
    a.ldq = int64_t(2) * I * 2;
    a.p = static_cast<const char *>(w13);
    a.p_expert = int64_t(2) * I * H * 2;
    a.ldp = int64_t(H) * 2;
    a.N = H;
    a.K = 2 * I;
    e = launch_tiles<true, Form::kPlain>(
        a, G, f.pairs, f.experts, PairOut{f.pair_row, f.pair_slot, nullptr, static_cast<uint16_t *>(dx), terms},
        "expert_ffn dx", stream);
    if (e != hipSuccess)
        return e;
    e = launch_rows(f, terms, dx, parts, tiles, dweight, stream);
    if (e != hipSuccess)
        return e;
    auto grid = [](int m, int n) { return unsigned((m + 255) / 256) * unsigned((n + 255) / 256); };
    const unsigned hm = (H + 255) / 256, in = (I + 255) / 256, gm = (2 * I + 255) / 256;
    if (log_enabled())
        log_launch("expert_ffn dW: experts=%d blocks=%lld + %lld", f.experts,
                   (long long)f.experts * grid(H, I), (long long)f.experts * grid(2 * I, H));
    GradArgs w{};
    w.pair_row = f.pair_row;
    w.offsets = f.offsets;
    w.experts = f.experts;
    w.q = static_cast<const char *>(dy);
    w.ldq = int64_t(H) * 2;
    w.p = static_cast<const char *>(wact);
    w.ldp = int64_t(I) * 2;
    w.M = H;
    w.N = I;
    w.mt = hm;
    w.nt = in;
    w.out = static_cast<uint16_t *>(dw2);
    GradArgs v = w;
    v.q = static_cast<const char *>(dgu);
    v.ldq = int64_t(2) * I * 2;
    v.p = static_cast<const char *>(x);
    v.ldp = int64_t(H) * 2;
    v.M = 2 * I;
    v.N = H;
    v.mt = gm;
    v.nt = hm;
    v.out = static_cast<uint16_t *>(dw13);
    // whole rounds of the XCDs, so that a block stays with one of them
    const int64_t all = int64_t(f.experts) * (int64_t(hm) * in + int64_t(gm) * hm);
    const int64_t cus = compute_units(), need = (all + 2 * kXcds - 1) / kXcds * kXcds;
    hipLaunchKernelGGL(weight_grads_kernel, dim3(unsigned(need < cus ? need : cus)), dim3(NT), 0, stream, w, v);
    return hipGetLastError();
}

hipError_t launch_ll_expert_ffn(int E, int R, int slots, int H, int I, int64_t max_pairs,
                                const int32_t *counts, const void *packed, const void *w13,
                                const void *w2, void *act, void *out, hipStream_t stream)
{
    const Groups G{nullptr, counts, slots, E, R, E / R, 1, kNoLimit};
    hipError_t e = launch_bf16<Form::kGated>(gated_args(packed, w13, H, I), G, max_pairs, slots,
                                             GatedOut{static_cast<uint16_t *>(act), nullptr},
                                             "ll_expert_ffn gated", stream);
    if (e != hipSuccess)
        return e;
    return launch_bf16<Form::kPlain>(down_args(act, w2, H, I), G, max_pairs, slots,
                                     RowOut{static_cast<uint16_t *>(out)}, "ll_expert_ffn down", stream);
}

}  // namespace ep
