// adapter.hip -- low-rank adapters of many requests beside a shared projection, and their gradients:
//   h[t] = c_a (x[t] A_a^T),  out[t] = base[t] + h[t] B_a^T,   a = ids[t], A [r][K], B [N][r]
//   dh[t] = c_a (dy[t] B_a),  dx[t] = dx_base[t] + dh[t] A_a,  dA_a = sum_t dh[t]^T x[t],  dB_a = sum_t dy[t]^T h[t]
// A block takes a tile of tokens that share an adapter: of few tokens it looks for them itself, more are sorted by
// adapter first.  The inner products to the rank (shrink) split K over waves and blocks; the products back
// (expand) sum those parts to h and add the base.  Rows are what it has to move: the forward pass reads and writes each
// once, the backward pass reads x once, and dy twice, for dh and for dB.
// 8192 tokens, K = N = 7168, rank 64, 16 adapters: 113 us (sort 8, shrink 39, expand 67) for 352 MB of rows, 3.1 TB/s;
// both products hold more than 256 registers (264 and 292 with the accumulators), so one block runs on a compute unit
// and nothing hides its waits.
// A step of 4096 tokens, N = 4096, rank 32, 8 adapters: 117 us (sort 5 twice; out 16 + 22, dx 12 + 30, the
// gradients 25) for 369 MB of rows, dy among them twice; two blocks of each product a unit, two of the gradients'.
// One token 9.6 us, of which 8.8 are the kernel's; 128 tokens on 64 adapters 14 (6.7 + 6.9).
#include "stream.h"

namespace ep {

namespace {

constexpr int kAdapterThreads = 256, kAdapterWaves = kAdapterThreads / kWave;
// Compute units that launches are shaped for, the same on every device, so that workspaces and results are too: it decides,
// with T, L and r, how sums over K are split.
constexpr int kCard = 256;

struct AdapterArgs {
    int T, L, r;
    const int64_t *ids;
    int32_t *offsets;  // [L + 2] starts of the groups in `order`; the last is of the tokens without an adapter
    int32_t *order;    // [T] tokens by (adapter, token)
    const float *scales;
    const char *q;     // shrink: token rows
    const char *p;     // shrink, expand: adapters
    int64_t width;     // of the rows that are shrunk or made
    float *parts;      // [splits][T][RP]
    int splits;
    const uint16_t *base;  // nullable
    uint16_t *out;
    uint16_t *hidden;  // nullable [2][T][r]: h in bf16, and what that rounding lost in bf16 again
};

// ---------------------------------------------------------------- grouping

// Block a: where adapter a's tokens start, and they in order.  Block L: those with no adapter.  Each block reads all ids
// twice: 8 us for 8192 tokens on 16 adapters, 15 on 1024; 131072 tokens take 210 on 1024 and 1190 on 8192.
constexpr int kSortThreads = 1024;
__global__ __launch_bounds__(kSortThreads) void adapter_group_kernel(AdapterArgs a)
{
    __shared__ int less_of[kSortThreads / kWave], here_of[8 * (kSortThreads / kWave)];
    const int mine = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto group = [&](int t) {
        const int64_t id = a.ids[t < a.T ? t : a.T - 1];  // (a load that nothing waits for before the others)
        return t >= a.T ? a.L + 1 : id >= 0 && id < a.L ? int(id) : a.L;
    };
    constexpr int N = 8;  // tokens a thread at a time, their ids in flight together
    int less = 0;
    for (int t0 = 0; t0 < a.T; t0 += N * kSortThreads) {
        int g[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            g[i] = group(t0 + i * kSortThreads + int(threadIdx.x));
#pragma unroll
        for (int i = 0; i < N; ++i)
            less += g[i] < mine;
    }
    less = int(wave_scan(uint32_t(less)));
    if (lane == 63)
        less_of[wave] = less;
    __syncthreads();
    int at = 0;
    for (int w = 0; w < kSortThreads / kWave; ++w)
        at += less_of[w];
    if (threadIdx.x == 0) {
        a.offsets[mine] = at;
        if (mine == a.L)
            a.offsets[a.L + 1] = a.T;
    }
    for (int t0 = 0; t0 < a.T; t0 += N * kSortThreads) {
        int g[N];
        uint64_t m[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            g[i] = group(t0 + i * kSortThreads + int(threadIdx.x));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            m[i] = wave_ballot(g[i] == mine);
            if (lane == 0)
                here_of[i * (kSortThreads / kWave) + wave] = __popcll(m[i]);
        }
        __syncthreads();
        // 128 counts in token order; lane l holds those of 2 l and 2 l + 1 and what is before them
        const int c0 = here_of[2 * lane], c1 = here_of[2 * lane + 1];
        const int upto = int(wave_scan(uint32_t(c0 + c1)));
        const int all = __builtin_amdgcn_readlane(upto, 63);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int k = i * (kSortThreads / kWave) + uniform(wave);
            int before = at + __builtin_amdgcn_readlane(upto - c0 - c1, k >> 1);
            before += k & 1 ? __builtin_amdgcn_readlane(c0, k >> 1) : 0;
            if (g[i] == mine)
                a.order[before + __popcll(m[i] & lanemask_lt())] = t0 + i * kSortThreads + int(threadIdx.x);
        }
        at += all;
        __syncthreads();
    }
}

// The b-th tile of BM rows over all groups; group -1 past the last.  Each wave looks for itself.
struct AdapterTile {
    int group, start, rows;  // rows of the tile, from position `start` of the order
};
__device__ __forceinline__ AdapterTile adapter_tile(const AdapterArgs &a, int b, int height, int lane)
{
    int base = 0;
    for (int g0 = 0; g0 <= a.L; g0 += 64) {
        const int g = g0 + lane;
        const int from = g <= a.L ? a.offsets[g] : 0, to = g <= a.L ? a.offsets[g + 1] : 0;
        const int tiles = (to - from + height - 1) / height;
        const int last = int(wave_scan(uint32_t(tiles))) + base;  // tiles up to and with this group
        const uint64_t m = wave_ballot(last > b);
        if (m != 0) {
            const int l = __builtin_ctzll(m);
            const int first = __builtin_amdgcn_readlane(last - tiles, l);
            const int start = __builtin_amdgcn_readlane(from, l) + (b - first) * height;
            const int left = __builtin_amdgcn_readlane(to, l) - start;
            return {g0 + l, start, left < height ? left : height};
        }
        base = __builtin_amdgcn_readlane(last, 63);
    }
    return {-1, 0, 0};
}

// Few tokens are not sorted: block a of a launch takes adapter a (the last one those with none) and finds its
// tokens, which it then goes through in tiles.
constexpr int kScanTokens = kAdapterThreads, kScanAdapters = 128;
template <int W>
__device__ __forceinline__ int scan_tokens(const AdapterArgs &a, int mine, int *list, int *count_of)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = threadIdx.x;
    int64_t id = t < a.T ? a.ids[t] : -2;
    id = t < a.T && !(id >= 0 && id < a.L) ? a.L : id;
    const uint64_t m = wave_ballot(id == mine);
    if (lane == 0)
        count_of[wave] = __popcll(m);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        before += w < wave ? count_of[w] : 0;
        all += count_of[w];
    }
    if (id == mine)
        list[before + __popcll(m & lanemask_lt())] = t;
    __syncthreads();
    return uniform(all);
}

// f(adapter, tokens in LDS, how many) for each tile of this block.
template <bool SCAN, int HEIGHT, class F>
__device__ __forceinline__ void each_tile(const AdapterArgs &a, F f)
{
    __shared__ int list[SCAN ? kScanTokens : HEIGHT], count_of[kAdapterWaves];
    if constexpr (SCAN) {
        const int all = scan_tokens<kAdapterWaves>(a, blockIdx.x, list, count_of);
        for (int m0 = 0; m0 < all; m0 += HEIGHT) {
            f(int(blockIdx.x), list + m0, all - m0 < HEIGHT ? all - m0 : HEIGHT);
            __syncthreads();
        }
    } else {
        const AdapterTile t = adapter_tile(a, blockIdx.x, HEIGHT, threadIdx.x & 63);
        if (t.group < 0)
            return;
        for (int i = threadIdx.x; i < t.rows; i += kAdapterThreads)
            list[i] = a.order[t.start + i];
        __syncthreads();
        f(t.group, static_cast<const int *>(list), t.rows);
    }
}

// ------------------------------------------------------------------ shrink

// 16 rows of a transposed operand out of LDS: rows k of `stride` bytes, lane l gets the column
// that `col(q)` + l % 4 names, q = l / 4 % 4, and k = k0 + l / 16 * 8 .. + 7.
template <class Col>
__device__ __forceinline__ bf16x8 transposed(const lds_char *base, int stride, int k0, Col col, int lane)
{
    const int i = lane & 15;
    const lds_char *p = base + (k0 + (lane >> 4) * 8 + (i >> 2)) * stride + col(i & 3) * 2;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * stride));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// acc[j][m] += sum over steps of 64 of K: weight rows times token rows, a wave's own step of both staged in LDS (whole
// lines a row) and the next one sent off as soon as it is in registers.  COL: the weight is [k][r].
template <int RT, int MT>
constexpr int kStageBytes = (RT + MT) * 16 * kStepBytes;
template <int RT, int MT, bool COL, bool TAIL, class Token>
__device__ __forceinline__ void stream_staged(const char *w, const AdapterArgs &a, Token token, int s0, int s1, int stride,
                                              lds_char *own, int lane, f32x4 (&acc)[RT][MT])
{
    using QS = RowStage<16 * MT, kWave>;
    using PS = NearRowStage<16 * RT, kWave>;
    constexpr int CH = RT * 2;
    if (s0 >= s1)
        return;
    const int width = int(a.width);
    lds_char *weights = own + QS::kBytes;
    QS qs;
    qs.init(lane, [&](int, int r) { return a.q + int64_t(token(r)) * width * 2; });
    PS ps;
    if constexpr (!COL)
        ps.init(lane, w, [&](int, int r) { return uint32_t(r < a.r ? r : a.r - 1) * uint32_t(width) * 2; });
    auto send = [&](int s) {
        qs.template issue<TAIL>(own, lane, 0, int64_t(s) * kStepBytes, int64_t(width) * 2);
        if constexpr (!COL)
            ps.template issue<TAIL>(weights, lane, 0, int64_t(s) * kStepBytes, int64_t(width) * 2);
        else {
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int at = j * kWave + lane, k = s * 64 + at / CH, c = at % CH;
                load_lds16(k < width && c * 8 < a.r ? w + (int64_t(k) * a.r + c * 8) * 2
                                                    : reinterpret_cast<const char *>(kZero16),
                           weights + j * kWave * 16);
            }
        }
    };
    send(s0);
    for (int s = s0; s < s1; s += stride) {
        landed<0>();
        bf16x8 p[RT][2], q[MT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                if constexpr (COL)
                    p[j][h] = transposed(weights, RT * 32, h * 32, [&](int c) { return j * 16 + c * 4; }, lane);
                else
                    p[j][h] = PS::frag(weights, j * 16, h, lane);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
                q[m][h] = QS::frag(own, m * 16, h, lane);
        }
        // read before the same LDS is loaded again
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        if (s + stride < s1)
            send(s + stride);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    acc[j][m] = mfma_bf16(p[j][h], q[m][h], acc[j][m]);
    }
}

template <int RT, int MT, bool COL, bool TAIL>
__device__ __forceinline__ void shrink_tile(const AdapterArgs &a, int adapter, const int *tokens, int rows, f32x4 *sums)
{
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int width = int(a.width);
    auto token = [&](int i) { return tokens[i < rows ? i : rows - 1]; };
    const char *w = a.p + int64_t(adapter) * a.r * width * 2;
    const int steps = (width + 63) / 64;
    const int s0 = steps * int(blockIdx.y) / a.splits, s1 = steps * int(blockIdx.y + 1) / a.splits, own_steps = s1 - s0;
    f32x4 acc[RT][MT] = {};
    // one row tile of a Row weight has little to share: straight into registers, several steps in flight
    if constexpr (!COL && MT == 1) {
        const char *prow[RT], *qrow[1] = {a.q + int64_t(token(lane & 15)) * width * 2};
        const float *none[RT] = {};
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const int row = j * 16 + (lane & 15);
            prow[j] = w + int64_t(row < a.r ? row : a.r - 1) * width * 2;
        }
        stream<false, TAIL, (RT > 4 ? 2 : 4), 1>(prow, none, qrow, s0 + own_steps * wave / kAdapterWaves,
                                                        s0 + own_steps * (wave + 1) / kAdapterWaves, width * 2, lane, acc);
    } else {
        // (the waves take turns along a row, so that its lines are read together)
        stream_staged<RT, MT, COL, TAIL>(w, a, token, s0 + wave, s1, kAdapterWaves, (lds_char *)sums + wave * kStageBytes<RT, MT>, lane, acc);
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m)
            sums[(wave * RT * MT + j * MT + m) * kWave + lane] = acc[j][m];
    __syncthreads();
    for (int i = wave; i < RT * MT; i += kAdapterWaves) {
        f32x4 v = sums[i * kWave + lane];
#pragma unroll
        for (int w4 = 1; w4 < kAdapterWaves; ++w4)
            v += sums[(w4 * RT * MT + i) * kWave + lane];
        const int j = i / MT, m = (i % MT) * 16 + (lane & 15);
        if (m < rows)
            *reinterpret_cast<f32x4 *>(a.parts + (int64_t(blockIdx.y) * a.T + tokens[m]) * (RT * 16) + j * 16 +
                                       (lane >> 4) * 4) = v;
    }
}

template <int RT>
constexpr int kTokenTiles = RT <= 4 ? 4 : 2;  // 16-row tiles of tokens a block

template <int RT, bool COL, bool TAIL, bool SCAN>
__global__ __launch_bounds__(kAdapterThreads) void adapter_shrink_kernel(AdapterArgs a)
{
    constexpr int MT = kTokenTiles<RT>;
    constexpr int kSums = kAdapterWaves * RT * MT * kWave * 16, kStages = kAdapterWaves * kStageBytes<RT, MT>;
    __shared__ __attribute__((aligned(128))) char lds[kSums > kStages ? kSums : kStages];
    f32x4 *sums = reinterpret_cast<f32x4 *>(lds);
    each_tile<SCAN, MT * 16>(a, [&](int adapter, const int *tokens, int rows) {
        if (adapter == a.L)
            return;
        if (rows <= 16)
            shrink_tile<RT, 1, COL, TAIL>(a, adapter, tokens, rows, sums);
        else
            shrink_tile<RT, MT, COL, TAIL>(a, adapter, tokens, rows, sums);
    });
}

// ------------------------------------------------------------------ expand

// out rows of one tile, columns [n0, n1) in steps of 64 a wave.  A wave stages its own weights in LDS; its results turn
// there, 16 tokens at a time, so that eight lanes read and write a whole line of a row.  h is the matrix instruction's
// operand, as the sum of its bf16 value and of what that rounding lost: with one value the result's error against 64
// bits is 1.2 to 1.4 times that of its own rounding, and two cost 64.2 -> 67.3 us (8192 rows of 7168, rank 64), nothing at
// smaller ranks.  Up to rank 16 both lie in one operand of 32, over the weights twice.
constexpr int kTurnRow = 68;  // floats: 16 rows of 64, four apart in the banks
template <int RT, bool COL, int W>
struct ExpandLds {
    static constexpr int KS = (RT + 1) / 2;  // matrix steps of 32
    static constexpr int kHidden = kTokenTiles<RT> * 16 * KS * 32;  // bf16 values
    static constexpr int kPlanes = RT == 1 ? 1 : 2, kRest = RT == 1 ? 16 : kHidden;  // from a value to what it lost
    static constexpr int kQuads = RT == 1 ? 4 : KS * 8;                              // of a token
    char weights[W][COL ? KS * 32 * 128 : (RT + 3) / 4 * 64 * kStepBytes];
    union {  // h is in registers before the first results turn
        uint16_t hidden[kPlanes * kHidden];
        float turn[W][16 * kTurnRow];
    };
};

template <int RT, int MT, bool COL, int W, class MakeH>
__device__ __forceinline__ void expand_tile(const AdapterArgs &a, int adapter, const int *tokens, int rows,
                                            ExpandLds<RT, COL, W> &lds, int n0, int n1, MakeH make_h)
{
    using Lds = ExpandLds<RT, COL, W>;
    constexpr int KS = Lds::KS, PL = Lds::kPlanes;
    using PS = NearRowStage<64, kWave>;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), g = lane >> 4;
    const int width = int(a.width);
    const bool adapted = adapter < a.L;
    lds_char *own = (lds_char *)lds.weights[wave];
    float *turn = lds.turn[wave];
    bf16x8 h[MT][KS][PL];
    int row[MT][2];  // the token whose line this lane reads and writes a chunk of; -1: none
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = m * 16 + i * 8 + (lane >> 3);
            row[m][i] = at < rows ? tokens[at] : -1;
        }
    auto place = [&](int token, int n) {  // (worked out each time: kept, the addresses cost a wave its place, 6.7 -> 10.1 us
        hold(token);                      // with 128 tokens on 64 adapters of rank 16)
        return int64_t(token) * width + (lane & 7) * 8 + n;
    };
    const char *w = a.p + int64_t(adapter) * a.r * width * 2;
    u32x4 b[MT][2] = {};
    auto send = [&](int n) {
        if (adapted) {
            if constexpr (COL) {  // A [r][width]: r rows of 64 columns
#pragma unroll
                for (int j = 0; j < KS * 4; ++j) {
                    const int at = j * kWave + lane, k = at >> 3, col = n + (at & 7) * 8;
                    load_lds16(k < a.r && col < width ? w + (int64_t(k) * width + col) * 2
                                                      : reinterpret_cast<const char *>(kZero16),
                               own + j * kWave * 16);
                }
            } else {  // B [width][r]: 64 rows
                PS ps;
                ps.init(lane, w + int64_t(n) * a.r * 2,
                        [&](int, int r) { return uint32_t(n + r < width ? r : width - 1 - n) * uint32_t(a.r) * 2; });
#pragma unroll
                for (int k = 0; k < (RT + 3) / 4; ++k)
                    ps.template issue<true>(own + k * PS::kBytes, lane, 0, k * kStepBytes, a.r * 2);
            }
        }
        if (a.base != nullptr) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (row[m][i] >= 0 && n + (lane & 7) * 8 < width)
                        b[m][i] = *reinterpret_cast<const u32x4 *>(a.base + place(row[m][i], n));
        }
    };
    int n = n0 + wave * 64;
    if (n < n1)
        send(n);
    make_h();  // while the first loads are on their way
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int u = 0; u < PL; ++u)
                h[m][s][u] = *reinterpret_cast<const bf16x8 *>(lds.hidden + u * Lds::kRest +
                                                               (m * 16 + (lane & 15)) * (KS * 32) + s * 32 + g * 8);
    __syncthreads();
    for (; n < n1; n += W * 64) {
        landed<0>();
        u32x4 now[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                now[m][i] = b[m][i];
                hold(now[m][i]);  // here: behind send() it would wait for the next loads
            }
        f32x4 acc[4][MT] = {};
        bf16x8 p[4][KS];
        if (adapted) {
            const int from = PL == 1 ? lane & 31 : lane;  // (k 16 to 31 is k 0 to 15 again)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    if constexpr (COL)
                        p[j][s] = transposed(own, 128, s * 32, [&](int q) { return j * 16 + q * 4; }, from);
                    else
                        p[j][s] = PS::frag(own + (s >> 1) * PS::kBytes, j * 16, s & 1, from);
                }
        }
        // read before the same LDS is loaded again
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        if (n + W * 64 < n1)
            send(n + W * 64);
        if (adapted) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int u = 0; u < PL; ++u)
                            acc[j][m] = mfma_bf16(p[j][s], h[m][s][u], acc[j][m]);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f32x4 *>(turn + (lane & 15) * kTurnRow + j * 16 + g * 4) = acc[j][m];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float *from = turn + (i * 8 + (lane >> 3)) * kTurnRow + (lane & 7) * 8;
                const f32x4 lo = *reinterpret_cast<const f32x4 *>(from), hi = *reinterpret_cast<const f32x4 *>(from + 4);
                const u32x4 &c = now[m][i];
                const u32x4 v = {cvt_bf16x2(lo[0] + bf16_lo(c[0]), lo[1] + bf16_hi(c[0])),
                                 cvt_bf16x2(lo[2] + bf16_lo(c[1]), lo[3] + bf16_hi(c[1])),
                                 cvt_bf16x2(hi[0] + bf16_lo(c[2]), hi[1] + bf16_hi(c[2])),
                                 cvt_bf16x2(hi[2] + bf16_lo(c[3]), hi[3] + bf16_hi(c[3]))};
                if (row[m][i] >= 0 && n + (lane & 7) * 8 < width)
                    __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(a.out + place(row[m][i], n)));
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    }
}

template <int RT, bool COL, bool SCAN>
__global__ __launch_bounds__(kAdapterThreads) void adapter_expand_kernel(AdapterArgs a, int columns)
{
    constexpr int MT = kTokenTiles<RT>, KS = (RT + 1) / 2, RP = RT * 16;
    __shared__ __attribute__((aligned(128))) ExpandLds<RT, COL, kAdapterWaves> lds;
    const int n0 = int(blockIdx.y) * columns, n1 = n0 + columns < a.width ? n0 + columns : int(a.width);
    each_tile<SCAN, MT * 16>(a, [&](int adapter, const int *tokens, int rows) {
        // h: the parts' sum, scaled, in bf16; zeros past the rank and the rows
        auto make_h = [&] {
            const float scale = adapter < a.L ? a.scales[adapter] : 0.0f;
            for (int i = threadIdx.x; i < MT * 16 * lds.kQuads; i += kAdapterThreads) {
                const int m = i / lds.kQuads, k = i % lds.kQuads * 4;
                f32x4 v = {};
                if (adapter < a.L && m < rows && k < a.r) {
                    const float *from = a.parts + int64_t(tokens[m]) * RP + k;
                    const int64_t apart = int64_t(a.T) * RP;
                    for (int s = 0; s < a.splits; s += 8) {  // eight loads in flight
                        f32x4 l[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            l[u] = s + u < a.splits ? *reinterpret_cast<const f32x4 *>(from + (s + u) * apart) : f32x4{};
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            v += l[u];
                    }
                    v *= scale;
                }
                const uint2 b = pack4(v), rest = pack4(lost(v, b));
                *reinterpret_cast<uint2 *>(lds.hidden + m * KS * 32 + k) = b;
                *reinterpret_cast<uint2 *>(lds.hidden + lds.kRest + m * KS * 32 + k) = rest;
                if (a.hidden != nullptr && blockIdx.y == 0 && m < rows && k < a.r) {
                    uint16_t *to = a.hidden + int64_t(tokens[m]) * a.r + k;
                    *reinterpret_cast<uint2 *>(to) = b;
                    *reinterpret_cast<uint2 *>(to + int64_t(a.T) * a.r) = rest;
                }
            }
            __syncthreads();
        };
        if (rows <= 16)
            expand_tile<RT, 1, COL>(a, adapter, tokens, rows, lds, n0, n1, make_h);
        else
            expand_tile<RT, MT, COL>(a, adapter, tokens, rows, lds, n0, n1, make_h);
    });
}

// --------------------------------------------------------------- few tokens

// Both products in one launch: each block makes h of its adapter's tokens itself, 16 at a time, its waves sharing
// out K, and then its columns of out.
constexpr int kFewWaves = 8, kFewTokens = 16, kFewRank = 64;

// The waves' parts of h, [wave][token][RT * 16 ranks], for 16 / C tokens from `tokens` (C: stream.h).
template <int RT, int C, bool TAIL>
__device__ __forceinline__ void few_parts(const AdapterArgs &a, int adapter, const int *tokens, int rows, float *parts)
{
    constexpr int kRows = 16 / C, TILES = RT * C;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), i0 = (lane & 15) / C;
    const int width = int(a.width), steps = (width + 63) / 64;
    const char *w = a.p + int64_t(adapter) * a.r * width * 2, *prow[TILES];
    const char *qrow[1] = {a.q + int64_t(tokens[i0 < rows ? i0 : rows - 1]) * width * 2};
    const float *none[TILES] = {};
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
        const int row = j * kRows + i0;
        prow[j] = w + int64_t(row < a.r ? row : a.r - 1) * width * 2;
    }
    f32x4 acc[TILES][1] = {};
    // steps in flight: as many as some 100 registers hold, 12, 20 and 36 a step; 7 for 8, as runs are rounded up to them and
    // 14 steps (K = 7168) are two rounds
    stream<false, TAIL, (RT == 1 ? 7 : RT == 2 ? 5 : 3), C>(prow, none, qrow, steps * wave / kFewWaves,
                                                           steps * (wave + 1) / kFewWaves, width * 2, lane, acc);
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
        float *to = parts + (wave * 16 + i0) * (RT * 16) + j * kRows;
        if constexpr (C == 1)
            *reinterpret_cast<f32x4 *>(to + (lane >> 4) * 4) = acc[j][0];
        else
            to[(lane >> 4) * 2 + (lane & 1)] = fold(acc[j][0], lane);
    }
}

template <int RT, bool TAIL>
__global__ __launch_bounds__(kFewWaves *kWave) void adapter_few_kernel(AdapterArgs a, const char *up, int N)
{
    constexpr int KS = (RT + 1) / 2;
    __shared__ __attribute__((aligned(128))) ExpandLds<RT, false, kFewWaves> lds;
    __shared__ __attribute__((aligned(16))) float parts[kFewWaves * 16 * RT * 16];
    __shared__ int list[kFewTokens], count_of[kFewWaves];
    const int adapter = blockIdx.x;
    const int all = scan_tokens<kFewWaves>(a, adapter, list, count_of);
    const int n0 = int(blockIdx.y) * kFewWaves * 64, n1 = n0 + kFewWaves * 64 < N ? n0 + kFewWaves * 64 : N;
    AdapterArgs e = a;  // of the second product
    e.p = up;
    e.width = N;
    for (int m0 = 0; m0 < all; m0 += 16) {
        const int rows = all - m0 < 16 ? all - m0 : 16, *tokens = list + m0;
        auto make_h = [&] {
            if (adapter < a.L) {
                if (rows <= 8)
                    few_parts<RT, 2, TAIL>(a, adapter, tokens, rows, parts);
                else
                    few_parts<RT, 1, TAIL>(a, adapter, tokens, rows, parts);
            }
            __syncthreads();
            for (int i = threadIdx.x; i < 16 * lds.kQuads; i += kFewWaves * kWave) {
                const int m = i / lds.kQuads, k = i % lds.kQuads * 4;
                f32x4 v = {};
                if (m < rows && k < a.r && adapter < a.L) {
#pragma unroll
                    for (int w = 0; w < kFewWaves; ++w)
                        v += *reinterpret_cast<const f32x4 *>(parts + (w * 16 + m) * (RT * 16) + k);
                    v *= a.scales[adapter];
                }
                const uint2 b = pack4(v), rest = pack4(lost(v, b));
                *reinterpret_cast<uint2 *>(lds.hidden + m * KS * 32 + k) = b;
                *reinterpret_cast<uint2 *>(lds.hidden + lds.kRest + m * KS * 32 + k) = rest;
                if (a.hidden != nullptr && blockIdx.y == 0 && m < rows && k < a.r) {
                    uint16_t *to = a.hidden + int64_t(tokens[m]) * a.r + k;
                    *reinterpret_cast<uint2 *>(to) = b;
                    *reinterpret_cast<uint2 *>(to + int64_t(a.T) * a.r) = rest;
                }
            }
            __syncthreads();
        };
        expand_tile<RT, 1, false>(e, adapter, tokens, rows, lds, n0, n1, make_h);
        __syncthreads();
    }
}

// --------------------------------------------------------- adapters' gradients

struct AdapterGradArgs {
    AdapterArgs a;
    const char *wide[2];    // x (of K), dy (of N)
    const char *narrow[2];  // dh, h: [2][T][r], sums of two bf16 values
    uint16_t *out[2];       // dA [L][r][K], dB [L][N][r]
    int width[2];
    int blocks[2];          // of both
};

// 64 columns of one adapter: sum over its tokens of wide[t][c] * narrow[t][j].  The waves share out the tokens, 64 a
// step, both operands out of LDS transposed, the next step sent off as soon as this one is in
// registers; the waves' sums meet in LDS.
template <int RT>
constexpr int kGradStage = 64 * 128 + 2 * 64 * RT * 32;
template <int RT, bool DOWN, bool SCAN>
__device__ __forceinline__ void adapter_grad(const AdapterGradArgs &g, int block, char *lds)
{
    const AdapterArgs &a = g.a;
    constexpr int CH = RT * 2;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int width = g.width[DOWN ? 0 : 1], chunks = (width + 63) / 64;
    const int l = block / chunks, n = block % chunks * 64;
    constexpr int kRound = kAdapterWaves * 64;
    int t0 = wave * 64, from = 0, count, first;
    if constexpr (SCAN) {  // (one round: the list is in registers before the LDS is loaded)
        static_assert(kScanTokens <= kRound, "one round");
        int *list = reinterpret_cast<int *>(lds);
        count = scan_tokens<kAdapterWaves>(a, l, list, list + kScanTokens);
        first = t0 + lane < count ? list[t0 + lane] : 0;
        __syncthreads();
    } else {
        from = a.offsets[l];
        count = a.offsets[l + 1] - from;
    }
    const char *wide = g.wide[DOWN ? 0 : 1], *narrow = g.narrow[DOWN ? 0 : 1];
    lds_char *own = (lds_char *)lds + wave * kGradStage<RT>, *small = own + 64 * 128;
    auto send = [&](int t0, int mine) {  // mine: the token of step row `lane`
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = j * 8 + (lane >> 3), c = n + (lane & 7) * 8, t = __shfl(mine, i);
            load_lds16(t0 + i < count && c < width ? wide + (int64_t(t) * width + c) * 2
                                                   : reinterpret_cast<const char *>(kZero16),
                       own + j * kWave * 16);
        }
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int at = j * kWave + lane, i = at / CH, c = at % CH, t = __shfl(mine, i);
            const char *p = narrow + (int64_t(t) * a.r + c * 8) * 2;
            const bool is = t0 + i < count && c * 8 < a.r;
#pragma unroll
            for (int u = 0; u < 2; ++u)
                load_lds16(is ? p + u * int64_t(a.T) * a.r * 2 : reinterpret_cast<const char *>(kZero16),
                           small + (u * CH + j) * kWave * 16);
        }
    };
    auto tokens = [&](int t0) { return !SCAN && t0 + lane < count ? a.order[from + t0 + lane] : 0; };
    f32x4 acc[4][RT] = {};
    if constexpr (!SCAN)
        first = tokens(t0);
    if (t0 < count)
        send(t0, first);
    int next = tokens(t0 + kRound);
    for (; t0 < count; t0 += kRound) {
        landed<0>();
        bf16x8 w[4][2], v[RT][2][2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i][s] = transposed(
                    own, 128, s * 32, [&](int q) { return DOWN ? (i >> 1) * 32 + q * 8 + (i & 1) * 4 : i * 16 + q * 4; }, lane);
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    v[j][s][u] = transposed(small + u * CH * kWave * 16, RT * 32, s * 32, [&](int q) { return j * 16 + q * 4; },
                                            lane);
        }
        // read before the same LDS is loaded again
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        if (t0 + kRound < count) {
            send(t0 + kRound, next);
            next = tokens(t0 + 2 * kRound);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        acc[i][j] = DOWN ? mfma_bf16(w[i][s], v[j][s][u], acc[i][j])
                                         : mfma_bf16(v[j][s][u], w[i][s], acc[i][j]);
    }
    f32x4 *sums = reinterpret_cast<f32x4 *>(lds);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j)
            sums[(wave * RT * 4 + j * 4 + i) * kWave + lane] = acc[i][j];
    __syncthreads();
    auto sum = [&](int tile) {
        f32x4 v = sums[tile * kWave + lane];
#pragma unroll
        for (int w = 1; w < kAdapterWaves; ++w)
            v += sums[(w * RT * 4 + tile) * kWave + lane];
        return pack4(v);
    };
    const int i16 = lane & 15, g16 = lane >> 4;
    for (int p = wave; p < RT * 2; p += kAdapterWaves) {  // two tiles: rank tile p / 2
        const int j = p >> 1, h = p & 1;
        const uint2 lo = sum(j * 4 + 2 * h), hi = sum(j * 4 + 2 * h + 1);
        if constexpr (DOWN) {  // lane: rank j * 16 + l % 16, eight columns
            const int rank = j * 16 + i16, c = n + h * 32 + g16 * 8;
            if (rank < a.r && c < width)
                *reinterpret_cast<u32x4 *>(g.out[0] + (int64_t(l) * a.r + rank) * width + c) = u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {  // lane: ranks j * 16 + l / 16 * 4 .., columns h * 32 + l % 16 and 16 further on
            const int rank = j * 16 + g16 * 4, c = n + h * 32 + i16;
            if (rank < a.r && c < width)
                *reinterpret_cast<uint2 *>(g.out[1] + (int64_t(l) * width + c) * a.r + rank) = lo;
            if (rank < a.r && c + 16 < width)
                *reinterpret_cast<uint2 *>(g.out[1] + (int64_t(l) * width + c + 16) * a.r + rank) = hi;
        }
    }
}

template <int RT, bool SCAN>
__global__ __launch_bounds__(kAdapterThreads) void adapter_grads_kernel(AdapterGradArgs g)
{
    constexpr int kStages = kAdapterWaves * kGradStage<RT>, kSums = kAdapterWaves * RT * 4 * kWave * 16;
    __shared__ __attribute__((aligned(128))) char lds[kStages > kSums ? kStages : kSums];
    const int block = int(blockIdx.y) * int(kRowGrid) + int(blockIdx.x);  // (row_grid; fewer than 2^28)
    if (block < g.blocks[0])
        adapter_grad<RT, true, SCAN>(g, block, lds);
    else if (block - g.blocks[0] < g.blocks[1])
        adapter_grad<RT, false, SCAN>(g, block - g.blocks[0], lds);
}

// ---------------------------------------------------------------- launches

int rank_tiles(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }
int tile_tokens(int r) { return r <= 64 ? 64 : 32; }
bool scans(int64_t T, int L) { return T <= kScanTokens && L < kScanAdapters; }
int64_t most_tiles(int64_t T, int L, int r)
{
    const int64_t groups = L + 1 < T ? L + 1 : T;
    return T / tile_tokens(r) + groups;
}
// Blocks of a launch that go by tile, or by adapter.
unsigned tile_blocks(int64_t T, int L, int r) { return unsigned(scans(T, L) ? L + 1 : most_tiles(T, L, r)); }
// Blocks that share a tile's K: as many as make two a compute unit, each wave at least one step.  Up to rank 32 two or
// three fit a unit's registers; of rank 64 and more one does, and the second follows it.
int shrink_splits(int64_t T, int L, int r, int width)
{
    const int64_t steps = (width + 63) / 64, most = (steps + kAdapterWaves - 1) / kAdapterWaves;
    const int64_t n = 2 * kCard / most_tiles(T, L, r);
    return int(n < 1 ? 1 : n < most ? n : most);
}

// One launch for few tokens, as long as every block that makes h again has a compute unit to itself and
// little to read.  r K <= 2^17 lies between two borders (us, one launch against two, one token on 8 adapters, N = 2048; 16
// tokens and N = 7168 give the same).  Called one by one, where the host's time counts, one launch wins up to twice that:
// rank 16, K = 7168 9.8 against 14.0; rank 64, K = 1024 9.6 against 14.0, K = 2048 11.1 against 14.0, K = 4096 13.9 against
// 13.8.  Replayed in a graph it wins up to half of it: rank 16, K = 2048 6.4 against 7.2, K = 4096 8.1 against 7.7, K = 7168
// 8.3 against 8.6; rank 64, K = 1024 7.2 against 8.5, K = 2048 11.2 against 8.5 (that kernel spills 16 registers).
bool few(const AdapterShape &s)
{
    const int64_t runs = (s.N + kFewWaves * 64 - 1) / (kFewWaves * 64);
    const int64_t groups = s.L + 1 < s.T ? s.L + 1 : s.T;
    return s.T <= kFewTokens && s.L < kScanAdapters && s.r <= kFewRank && int64_t(s.r) * s.K <= (1 << 17) &&
           groups * runs <= kCard;
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

struct AdapterWork {
    int32_t *offsets, *order;
    uint16_t *dh;
    float *parts;
};
size_t adapter_layout(const AdapterShape &s, bool back, char *base, AdapterWork *w)
{
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *p = base + at;
        at += up256(bytes);
        return p;
    };
    AdapterWork m;
    m.offsets = reinterpret_cast<int32_t *>(take(size_t(s.L + 2) * 4));
    m.order = reinterpret_cast<int32_t *>(take(size_t(s.T) * 4));
    m.dh = reinterpret_cast<uint16_t *>(take(back ? size_t(s.T) * s.r * 4 : 0));
    const size_t splits = s.T > 0 ? shrink_splits(s.T, s.L, s.r, back ? s.N : s.K) : 0;
    m.parts = reinterpret_cast<float *>(take(splits * size_t(s.T) * rank_tiles(s.r) * 64));
    if (w != nullptr)
        *w = m;
    return at;
}

template <class F>
hipError_t by_rank(int r, F f)
{
    switch (rank_tiles(r)) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    default: return f(std::integral_constant<int, 8>());
    }
}

AdapterArgs adapter_args(const AdapterShape &s, const AdapterWork &w)
{
    AdapterArgs a{};
    a.T = s.T;
    a.L = s.L;
    a.r = s.r;
    a.ids = s.ids;
    a.offsets = w.offsets;
    a.order = w.order;
    a.scales = s.scales;
    a.parts = w.parts;
    return a;
}

hipError_t group_tokens(const AdapterArgs &a, hipStream_t stream)
{
    hipLaunchKernelGGL(adapter_group_kernel, dim3(a.L + 1), dim3(kSortThreads), 0, stream, a);
    return hipGetLastError();
}

// parts of rows q [T][width] times the adapters w, [r][width] or (COL) [width][r].
template <bool COL>
hipError_t shrink(AdapterArgs &a, const void *q, const void *w, int width, hipStream_t stream)
{
    a.q = static_cast<const char *>(q);
    a.p = static_cast<const char *>(w);
    a.width = width;
    a.splits = shrink_splits(a.T, a.L, a.r, width);
    return by_rank(a.r, [&](auto rt) {
        constexpr int RT = decltype(rt)::value;
        const dim3 grid(tile_blocks(a.T, a.L, a.r), unsigned(a.splits));
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kAdapterThreads), 0, stream, a); };
        const bool tail = width % 64 != 0;
        if (scans(a.T, a.L))
            go(tail ? adapter_shrink_kernel<RT, COL, true, true> : adapter_shrink_kernel<RT, COL, false, true>);
        else
            go(tail ? adapter_shrink_kernel<RT, COL, true, false> : adapter_shrink_kernel<RT, COL, false, false>);
        return hipGetLastError();
    });
}

template <bool COL>
hipError_t expand(AdapterArgs &a, const void *w, int width, const void *base, void *out, void *hidden, hipStream_t stream)
{
    a.p = static_cast<const char *>(w);
    a.width = width;
    a.base = static_cast<const uint16_t *>(base);
    a.out = static_cast<uint16_t *>(out);
    a.hidden = static_cast<uint16_t *>(hidden);
    return by_rank(a.r, [&](auto rt) {
        constexpr int RT = decltype(rt)::value;
        constexpr int kRun = kAdapterWaves * 64;
        const bool scan = scans(a.T, a.L);
        const int64_t tiles = most_tiles(a.T, a.L, a.r), runs = (width + kRun - 1) / kRun;
        // Blocks that share a tile's columns: as many as make two a compute unit, each then has several steps behind its start
        // (8192 rows of 7168, rank 64, where one fits a unit, h as one value: 64.0 us, with four 68.3); four where each finds
        // its tokens itself, many of them none (128 tokens on 64 adapters, rank 16, where two fit: 6.9 us, with two 7.4).
        int64_t n = (scan ? 4 : 2) * kCard / tiles;
        n = n < 1 ? 1 : n < runs ? n : runs;
        const int columns = int((runs + n - 1) / n) * kRun;
        hipLaunchKernelGGL((scan ? adapter_expand_kernel<RT, COL, true> : adapter_expand_kernel<RT, COL, false>),
                           dim3(tile_blocks(a.T, a.L, a.r), unsigned((width + columns - 1) / columns)),
                           dim3(kAdapterThreads), 0, stream, a, columns);
        return hipGetLastError();
    });
}

}  // namespace

// One launch hands nothing on.
size_t adapter_workspace(const AdapterShape &s, bool back)
{
    return !back && few(s) ? 0 : adapter_layout(s, back, nullptr, nullptr);
}

hipError_t launch_adapter(const AdapterShape &s, const void *x, const void *down, const void *up, const void *base, void *out,
                          void *hidden, void *workspace, hipStream_t stream)
{
    AdapterWork w{};
    if (workspace != nullptr)
        adapter_layout(s, false, static_cast<char *>(workspace), &w);
    AdapterArgs a = adapter_args(s, w);
    if (log_enabled())
        log_launch("adapter_product: T=%d K=%d N=%d r=%d L=%d splits=%d", s.T, s.K, s.N, s.r, s.L,
                   shrink_splits(s.T, s.L, s.r, s.K));
    if (few(s)) {
        a.q = static_cast<const char *>(x);
        a.p = static_cast<const char *>(down);
        a.width = s.K;
        a.base = static_cast<const uint16_t *>(base);
        a.out = static_cast<uint16_t *>(out);
        a.hidden = static_cast<uint16_t *>(hidden);
        return by_rank(s.r, [&](auto rt) {
            constexpr int RT = decltype(rt)::value < 4 ? decltype(rt)::value : 4;
            hipLaunchKernelGGL((s.K % 64 != 0 ? adapter_few_kernel<RT, true> : adapter_few_kernel<RT, false>),
                               dim3(s.L + 1, (s.N + kFewWaves * 64 - 1) / (kFewWaves * 64)), dim3(kFewWaves * kWave), 0, stream, a,
                               static_cast<const char *>(up), s.N);
            return hipGetLastError();
        });
    }
    hipError_t e = scans(s.T, s.L) ? hipSuccess : group_tokens(a, stream);
    if (e == hipSuccess)
        e = shrink<false>(a, x, down, s.K, stream);
    return e == hipSuccess ? expand<false>(a, up, s.N, base, out, hidden, stream) : e;
}

hipError_t launch_adapter_backward(const AdapterShape &s, const void *dy, const void *x, const void *down, const void *up,
                                   const void *hidden, const void *dx_base, void *dx, void *ddown, void *dup, void *workspace,
                                   hipStream_t stream)
{
    AdapterWork w;
    adapter_layout(s, true, static_cast<char *>(workspace), &w);
    AdapterArgs a = adapter_args(s, w);
    if (log_enabled())
        log_launch("adapter_product_backward: T=%d K=%d N=%d r=%d L=%d", s.T, s.K, s.N, s.r, s.L);
    hipError_t e = scans(s.T, s.L) ? hipSuccess : group_tokens(a, stream);
    if (e == hipSuccess && s.T > 0)
        e = shrink<true>(a, dy, up, s.N, stream);
    if (e == hipSuccess && s.T > 0)
        e = expand<true>(a, down, s.K, dx_base, dx, w.dh, stream);
    if (e != hipSuccess)
        return e;
    AdapterGradArgs g{};
    g.a = a;
    g.wide[0] = static_cast<const char *>(x);
    g.wide[1] = static_cast<const char *>(dy);
    g.narrow[0] = reinterpret_cast<const char *>(w.dh);
    g.narrow[1] = static_cast<const char *>(hidden);
    g.out[0] = static_cast<uint16_t *>(ddown);
    g.out[1] = static_cast<uint16_t *>(dup);
    g.width[0] = s.K;
    g.width[1] = s.N;
    for (int i = 0; i < 2; ++i)
        g.blocks[i] = s.L * ((g.width[i] + 63) / 64);
    return by_rank(s.r, [&](auto rt) {
        constexpr int RT = decltype(rt)::value;
        hipLaunchKernelGGL((scans(s.T, s.L) ? adapter_grads_kernel<RT, true> : adapter_grads_kernel<RT, false>),
                           row_grid(int64_t(g.blocks[0]) + g.blocks[1]), dim3(kAdapterThreads), 0, stream, g);
        return hipGetLastError();
    });
}

}  // namespace ep
