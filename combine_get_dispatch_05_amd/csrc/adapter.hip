// adapter.hip -- low-rank adapters of many requests beside a shared projection, and their gradients:
//   h[t] = c_a (x[t] A_a^T),  out[t] = base[t] + h[t] B_a^T,   a = ids[t], A [r][K], B [N][r]
//   dh[t] = c_a (dy[t] B_a),  dx[t] = dx_base[t] + dh[t] A_a,  dA_a = sum_t dh[t]^T x[t],  dB_a = sum_t dy[t]^T h[t]
// Tokens are grouped by adapter first (a tile of up to 16 MT rows has one adapter).  The inner products to
// the rank (shrink) split K over waves and blocks; the products back (expand) sum those parts, round h to
// bf16, the matrix instruction's operand, and add the base.  All of it is bound by memory:
// rows are read and written once in whole 128-byte lines.
#include "stream.h"

namespace ep {

namespace {

constexpr int kAdapterThreads = 256, kAdapterWaves = kAdapterThreads / kWave;
constexpr int kCard = 256;  // compute units that launches are shaped for (results do not depend on it, nor workspaces on the device)

struct AdapterArgs {
    int T, L, r;
    const int64_t *ids;
    int32_t *offsets;  // [L + 2] starts of the groups in `order`; the last is of the tokens without an adapter
    int32_t *order;    // [T] tokens by (adapter, token)
    const float *scales;
    const char *q;     // shrink: token rows
    const char *p;     // shrink, expand: adapters
    int64_t width;     // of the rows that are shrunk or made
    float *parts;      // [splits][T][RP], in `order`
    int splits;
    const uint16_t *base;  // nullable
    uint16_t *out;
    uint16_t *hidden;  // nullable [T][r]
};

// ---------------------------------------------------------------- grouping

// Block a: where adapter a's tokens start, and they in order.  Block L: those with no adapter.
constexpr int kSortThreads = 1024;
__global__ __launch_bounds__(kSortThreads) void adapter_group_kernel(AdapterArgs a)
{
    __shared__ int less_of[kSortThreads / kWave], here_of[kSortThreads / kWave];
    const int mine = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto group = [&](int t) {
        if (t >= a.T)
            return a.L + 1;
        const int64_t id = a.ids[t];
        return id >= 0 && id < a.L ? int(id) : a.L;
    };
    int less = 0;
    for (int t = threadIdx.x; t < a.T; t += kSortThreads)
        less += group(t) < mine;
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
    for (int t0 = 0; t0 < a.T; t0 += kSortThreads) {
        const int t = t0 + int(threadIdx.x);
        const bool is = group(t) == mine;
        const uint64_t m = wave_ballot(is);
        __syncthreads();
        if (lane == 0)
            here_of[wave] = __popcll(m);
        __syncthreads();
        int before = at;
        for (int w = 0; w < kSortThreads / kWave; ++w) {
            before += w < wave ? here_of[w] : 0;
            at += here_of[w];
        }
        if (is)
            a.order[before + __popcll(m & lanemask_lt())] = t;
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

// acc[j][m] += sum over k steps of 64: transposed weight rows [k][r] times token rows.
template <int RT, int MT>
__device__ __forceinline__ void stream_transposed(const char *w, int r, const char *const (&qrow)[MT], int s0, int s1, int width,
                                                  lds_char *own, int lane, f32x4 (&acc)[RT][MT])
{
    constexpr int CH = RT * 2, J = CH;  // 16-byte chunks of a staged row; loads a lane for 64 rows
    const int g = lane >> 4;
    for (int s = s0; s < s1; ++s) {
        i32x4 q[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = s * 64 + h * 32 + g * 8;
                q[m][h] = load16(k < width ? qrow[m] + k * 2 : reinterpret_cast<const char *>(kZero16));
            }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int at = j * kWave + lane, k = s * 64 + at / CH, c = at % CH;
            load_lds16(k < width && c * 8 < r ? w + (int64_t(k) * r + c * 8) * 2 : reinterpret_cast<const char *>(kZero16),
                       own + j * kWave * 16);
        }
        landed<0>();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const bf16x8 p = transposed(own, RT * 32, h * 32, [&](int c) { return j * 16 + c * 4; }, lane);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    acc[j][m] = mfma_bf16(p, __builtin_bit_cast(bf16x8, q[m][h]), acc[j][m]);
            }
        // read before the same LDS is loaded again
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    }
}

template <int RT, int MT, bool COL, bool TAIL>
__device__ __forceinline__ void shrink_tile(const AdapterArgs &a, const AdapterTile &t, f32x4 *sums)
{
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int width = int(a.width);
    const char *qrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int i = m * 16 + (lane & 15);
        qrow[m] = a.q + int64_t(a.order[t.start + (i < t.rows ? i : t.rows - 1)]) * width * 2;
    }
    const char *w = a.p + int64_t(t.group) * a.r * width * 2;
    const int steps = (width + 63) / 64, split = int(blockIdx.y) * kAdapterWaves + wave;
    const int of = a.splits * kAdapterWaves;
    const int s0 = int(int64_t(steps) * split / of), s1 = int(int64_t(steps) * (split + 1) / of);
    f32x4 acc[RT][MT] = {};
    if constexpr (COL) {
        lds_char *own = (lds_char *)sums + wave * RT * 32 * 64;
        stream_transposed<RT, MT>(w, a.r, qrow, s0, s1, width, own, lane, acc);
        __syncthreads();
    } else {
        const char *prow[RT];
        const float *none[RT] = {};
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const int row = j * 16 + (lane & 15);
            prow[j] = w + int64_t(row < a.r ? row : a.r - 1) * width * 2;
        }
        stream<false, TAIL, (RT * MT > 4 ? 2 : 4), 1>(prow, none, qrow, s0, s1, width * 2, lane, acc);
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
        if (m < t.rows)
            *reinterpret_cast<f32x4 *>(a.parts + (int64_t(blockIdx.y) * a.T + t.start + m) * (RT * 16) + j * 16 +
                                       (lane >> 4) * 4) = v;
    }
}

template <int RT>
constexpr int kTokenTiles = RT <= 4 ? 4 : 2;  // 16-row tiles of tokens a block

template <int RT, bool COL, bool TAIL>
__global__ __launch_bounds__(kAdapterThreads) void adapter_shrink_kernel(AdapterArgs a)
{
    constexpr int MT = kTokenTiles<RT>;
    __shared__ f32x4 sums[kAdapterWaves * RT * MT * kWave];
    const AdapterTile t = adapter_tile(a, blockIdx.x, MT * 16, threadIdx.x & 63);
    if (t.group < 0 || t.group == a.L)
        return;
    if (t.rows <= 16)
        shrink_tile<RT, 1, COL, TAIL>(a, t, sums);
    else
        shrink_tile<RT, MT, COL, TAIL>(a, t, sums);
}

// ------------------------------------------------------------------ expand

// out rows of one tile, columns [n0, n1) in steps of 64 a wave.  The weight row of a tile's i-th operand row is
// permuted, so that a lane ends with 16 neighbouring columns of its token and four lanes with a whole line.
template <int RT, int MT, bool COL>
__device__ __forceinline__ void expand_tile(const AdapterArgs &a, const AdapterTile &t, const uint16_t *hs, lds_char *own, int n0,
                                            int n1)
{
    constexpr int KS = (RT + 1) / 2;  // matrix steps of 32
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), g = lane >> 4;
    const int width = int(a.width);
    const bool adapted = t.group < a.L;
    bf16x8 h[MT][KS];
    int64_t row[MT];
    bool live[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int i = m * 16 + (lane & 15);
        live[m] = i < t.rows;
        row[m] = int64_t(a.order[t.start + (live[m] ? i : t.rows - 1)]) * width;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            h[m][s] = *reinterpret_cast<const bf16x8 *>(hs + i * (KS * 32) + s * 32 + g * 8);
    }
    const char *w = a.p + int64_t(t.group) * a.r * width * 2;
    for (int n = n0 + wave * 64; n < n1; n += kAdapterWaves * 64) {
        const int c = n + g * 16;  // this lane's columns
        u32x4 b[MT][2] = {};
        if (a.base != nullptr) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (live[m] && c + i * 8 < width)
                        b[m][i] = *reinterpret_cast<const u32x4 *>(a.base + row[m] + c + i * 8);
        }
        f32x4 acc[4][MT] = {};
        if (adapted) {
            if constexpr (COL) {  // A [r][width]: r rows of 64 columns in LDS
                constexpr int J = KS * 32 * 8 / kWave;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int at = j * kWave + lane, k = at >> 3, col = n + (at & 7) * 8;
                    load_lds16(k < a.r && col < width ? w + (int64_t(k) * width + col) * 2
                                                      : reinterpret_cast<const char *>(kZero16),
                               own + j * kWave * 16);
                }
                landed<0>();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    bf16x8 p;
                    if constexpr (COL)
                        p = transposed(own, 128, s * 32, [&](int q) { return q * 16 + j * 4; }, lane);
                    else {  // B [width][r]
                        const int i = lane & 15, col = n + (i >> 2) * 16 + j * 4 + (i & 3), k = s * 32 + g * 8;
                        p = __builtin_bit_cast(bf16x8,
                                               load16(k < a.r ? w + (int64_t(col < width ? col : width - 1) * a.r + k) * 2
                                                              : reinterpret_cast<const char *>(kZero16)));
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[j][m] = mfma_bf16(p, h[m][s], acc[j][m]);
                }
            if constexpr (COL)
                asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                u32x4 v;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int at = i * 8 + k * 2;
                    v[k] = cvt_bf16x2(acc[at >> 2][m][at & 3] + bf16_lo(b[m][i][k]),
                                      acc[at >> 2][m][(at & 3) + 1] + bf16_hi(b[m][i][k]));
                }
                if (live[m] && c + i * 8 < width)
                    *reinterpret_cast<u32x4 *>(a.out + row[m] + c + i * 8) = v;
            }
    }
}

template <int RT, bool COL>
__global__ __launch_bounds__(kAdapterThreads) void adapter_expand_kernel(AdapterArgs a, int columns)
{
    constexpr int MT = kTokenTiles<RT>, KS = (RT + 1) / 2, RP = RT * 16;
    __shared__ __attribute__((aligned(128))) uint16_t hs[MT * 16 * KS * 32];
    __shared__ __attribute__((aligned(128))) char stage[COL ? kAdapterWaves * KS * 32 * 128 : 16];
    const AdapterTile t = adapter_tile(a, blockIdx.x, MT * 16, threadIdx.x & 63);
    if (t.group < 0)
        return;
    // h: the parts' sum, scaled, in bf16; zeros past the rank and the rows
    const float scale = t.group < a.L ? a.scales[t.group] : 0.0f;
    for (int i = threadIdx.x; i < MT * 16 * KS * 8; i += kAdapterThreads) {
        const int m = i / (KS * 8), k = i % (KS * 8) * 4;
        f32x4 v = {};
        if (t.group < a.L && m < t.rows && k < a.r) {
            const float *from = a.parts + int64_t(t.start + m) * RP + k;
            for (int s = 0; s < a.splits; ++s)
                v += *reinterpret_cast<const f32x4 *>(from + int64_t(s) * a.T * RP);
            v *= scale;
        }
        const uint2 b = pack4(v);
        *reinterpret_cast<uint2 *>(hs + m * KS * 32 + k) = b;
        if (a.hidden != nullptr && blockIdx.y == 0 && m < t.rows && k < a.r)
            *reinterpret_cast<uint2 *>(a.hidden + int64_t(a.order[t.start + m]) * a.r + k) = b;
    }
    __syncthreads();
    const int n0 = int(blockIdx.y) * columns, n1 = n0 + columns < a.width ? n0 + columns : int(a.width);
    lds_char *own = (lds_char *)stage + (COL ? (threadIdx.x >> 6) * KS * 32 * 128 : 0);
    if (t.rows <= 16)
        expand_tile<RT, 1, COL>(a, t, hs, own, n0, n1);
    else
        expand_tile<RT, MT, COL>(a, t, hs, own, n0, n1);
}

// --------------------------------------------------------- adapters' gradients

struct AdapterGradArgs {
    AdapterArgs a;
    const char *wide[2];    // x (of K), dy (of N)
    const char *narrow[2];  // dh, h: bf16 [T][r]
    uint16_t *out[2];       // dA [L][r][K], dB [L][N][r]
    int width[2];
    int blocks;             // of the first
};

// 64 columns a wave of one adapter: sum over its tokens of wide[t][c] * narrow[t][j], 64 tokens a step,
// both out of LDS transposed.
template <int RT, bool DOWN>
__device__ __forceinline__ void adapter_grad(const AdapterGradArgs &g, int block, lds_char *own)
{
    const AdapterArgs &a = g.a;
    constexpr int CH = RT * 2, J = CH;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int width = g.width[DOWN ? 0 : 1], chunks = (width + kAdapterWaves * 64 - 1) / (kAdapterWaves * 64);
    const int l = block / chunks, n = (block % chunks) * (kAdapterWaves * 64) + wave * 64;
    if (n >= width)
        return;
    const int from = a.offsets[l], count = a.offsets[l + 1] - from;
    const char *wide = g.wide[DOWN ? 0 : 1], *narrow = g.narrow[DOWN ? 0 : 1];
    lds_char *small = own + 64 * 128;
    f32x4 acc[4][RT] = {};
    for (int t0 = 0; t0 < count; t0 += 64) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int t = t0 + j * 8 + (lane >> 3), c = n + (lane & 7) * 8;
            load_lds16(t < count && c < width ? wide + (int64_t(a.order[from + t]) * width + c) * 2
                                              : reinterpret_cast<const char *>(kZero16),
                       own + j * kWave * 16);
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int at = j * kWave + lane, t = t0 + at / CH, c = at % CH;
            load_lds16(t < count && c * 8 < a.r ? narrow + (int64_t(a.order[from + t]) * a.r + c * 8) * 2
                                                : reinterpret_cast<const char *>(kZero16),
                       small + j * kWave * 16);
        }
        landed<0>();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            bf16x8 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = transposed(own, 128, s * 32, [&](int q) { return DOWN ? q * 16 + i * 4 : i * 16 + q * 4; }, lane);
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const bf16x8 v = transposed(small, RT * 32, s * 32, [&](int q) { return j * 16 + q * 4; }, lane);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i][j] = DOWN ? mfma_bf16(w[i], v, acc[i][j]) : mfma_bf16(v, w[i], acc[i][j]);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    }
    const int i16 = lane & 15, g16 = lane >> 4;
    if constexpr (DOWN) {  // lane: rank j * 16 + l % 16, columns n + l / 16 * 16 ..
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int rank = j * 16 + i16, c = n + g16 * 16 + h * 8;
                const uint2 lo = pack4(acc[2 * h][j]), hi = pack4(acc[2 * h + 1][j]);
                if (rank < a.r && c < width)
                    *reinterpret_cast<u32x4 *>(g.out[0] + (int64_t(l) * a.r + rank) * width + c) =
                        u32x4{lo.x, lo.y, hi.x, hi.y};
            }
    } else {  // lane: column n + i * 16 + l % 16, ranks j * 16 + l / 16 * 4 ..
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const int c = n + i * 16 + i16, rank = j * 16 + g16 * 4;
                if (rank < a.r && c < width)
                    *reinterpret_cast<uint2 *>(g.out[1] + (int64_t(l) * width + c) * a.r + rank) = pack4(acc[i][j]);
            }
    }
}

template <int RT>
__global__ __launch_bounds__(kAdapterThreads) void adapter_grads_kernel(AdapterGradArgs g)
{
    constexpr int kOwn = 64 * 128 + 64 * RT * 32;
    __shared__ __attribute__((aligned(128))) char stage[kAdapterWaves * kOwn];
    lds_char *own = (lds_char *)stage + (threadIdx.x >> 6) * kOwn;
    if (int(blockIdx.x) < g.blocks)
        adapter_grad<RT, true>(g, blockIdx.x, own);
    else
        adapter_grad<RT, false>(g, int(blockIdx.x) - g.blocks, own);
}

// ---------------------------------------------------------------- launches

int rank_tiles(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }
int tile_tokens(int r) { return r <= 64 ? 64 : 32; }
int64_t most_tiles(int64_t T, int L, int r)
{
    const int64_t groups = L + 1 < T ? L + 1 : T;
    return T / tile_tokens(r) + groups;
}
// Blocks that share a tile's K: so many that the card is full twice, each wave at least one step.
int shrink_splits(int64_t T, int L, int r, int width)
{
    const int64_t steps = (width + 63) / 64, most = (steps + kAdapterWaves - 1) / kAdapterWaves;
    const int64_t n = 2 * kCard / most_tiles(T, L, r);
    return int(n < 1 ? 1 : n < most ? n : most);
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
    m.dh = reinterpret_cast<uint16_t *>(take(back ? size_t(s.T) * s.r * 2 : 0));
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
        const dim3 grid(unsigned(most_tiles(a.T, a.L, a.r)), unsigned(a.splits));
        if (!COL && width % 64 != 0)
            hipLaunchKernelGGL((adapter_shrink_kernel<RT, COL, !COL>), grid, dim3(kAdapterThreads), 0, stream, a);
        else
            hipLaunchKernelGGL((adapter_shrink_kernel<RT, COL, false>), grid, dim3(kAdapterThreads), 0, stream, a);
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
        const int64_t tiles = most_tiles(a.T, a.L, a.r), runs = (width + kRun - 1) / kRun;
        int64_t n = 4 * kCard / tiles;  // blocks that share a tile's columns
        n = n < 1 ? 1 : n < runs ? n : runs;
        const int columns = int((runs + n - 1) / n) * kRun;
        hipLaunchKernelGGL((adapter_expand_kernel<RT, COL>), dim3(unsigned(tiles), unsigned((width + columns - 1) / columns)),
                           dim3(kAdapterThreads), 0, stream, a, columns);
        return hipGetLastError();
    });
}

}  // namespace

size_t adapter_workspace(const AdapterShape &s, bool back) { return adapter_layout(s, back, nullptr, nullptr); }

hipError_t launch_adapter(const AdapterShape &s, const void *x, const void *down, const void *up, const void *base, void *out,
                          void *hidden, void *workspace, hipStream_t stream)
{
    AdapterWork w;
    adapter_layout(s, false, static_cast<char *>(workspace), &w);
    AdapterArgs a = adapter_args(s, w);
    if (log_enabled())
        log_launch("adapter_product: T=%d K=%d N=%d r=%d L=%d splits=%d", s.T, s.K, s.N, s.r, s.L,
                   shrink_splits(s.T, s.L, s.r, s.K));
    hipError_t e = group_tokens(a, stream);
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
    hipError_t e = group_tokens(a, stream);
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
    constexpr int kRun = kAdapterWaves * 64;
    g.blocks = s.L * ((s.K + kRun - 1) / kRun);
    const unsigned all = unsigned(g.blocks + s.L * ((s.N + kRun - 1) / kRun));
    return by_rank(s.r, [&](auto rt) {
        hipLaunchKernelGGL((adapter_grads_kernel<decltype(rt)::value>), dim3(all), dim3(kAdapterThreads), 0, stream, g);
        return hipGetLastError();
    });
}

}  // namespace ep
