// moe.hip -- a whole mixture-of-experts layer for a few tokens: router, experts and
// weighted sum, without packing rows in between.
//   logits = x Wr^T, route (route.h), y[t] = residual[t] + sum_k w_k (silu(x Wg^T) * (x Wu^T)) W2^T
// The weights of the reached experts are read once and are the cost.  They go straight from
// memory into the matrix instruction's registers, 16 weight rows by the tokens of one
// expert, K shared out over the waves of a block, each keeping ahead() steps of 128 bytes a row
// in flight.  FP8 weights are widened to bf16 there, exactly, so that rows and
// activations keep their bf16 values.
// Bound by the weights where there are many, 32 tokens on 64 FP8 experts of 2048 x 7168: 472 us for 2.8 GB,
// 6.0 TB/s (logits 9, choice 13, gate and up 310, down 151).  One token, eight experts: FP8 2048 x 7168 82 us
// (5 + 52 + 25) for 356 MB; bf16 768 x 2048 22 us (3 + 13.5 + 7.4) for 76 MB, three launches whose starts and ends
// are half of it.
#include "route.h"
#include "stream.h"

namespace ep {

namespace {

struct alignas(32) ActiveExpert {
    int32_t expert, start, count, unused;  // its pairs: [start, start + count)
    uint64_t tokens;                       // bit t: token t
};
// The token of its i-th pair.
__device__ __forceinline__ int token_of(uint64_t tokens, int i)
{
    for (; i > 0; --i)
        tokens &= tokens - 1;
    return __builtin_ctzll(tokens);
}

// K steps that a wave keeps in flight: as many as fit some 100 registers, at most four (a run's length is
// rounded up to them).
constexpr int ahead(bool fp8, int C, int RT, int MT, int planes = 1)
{
    const int n = 100 / (4 * (RT * 2 / C + MT * planes * (fp8 ? 4 : 2) / C));
    return n < 2 ? 2 : n < 4 ? n : 4;
}

constexpr int kLogitSplits = 8;    // at most, a power of two
constexpr int kLogitLeaves = 256;  // at most, likewise

// The activation between the products is the matrix instruction's operand.  One rounding to bf16 makes the result's
// error against 64 bits 1.4 times what its own rounding is (2.4e-3 of the norm instead of 1.7e-3).  Beside bf16
// weights it is kept as a sum of two bf16 values, which costs 0.7 us of 22 (one token, eight experts of 768 x 2048).
// Beside FP8 weights, whose codes are off by up to 2^-4, it is rounded once: the second load of
// tokens would take 45 us of 470 (32 tokens, 64 experts of 2048 x 7168).
template <bool FP8>
constexpr int kActPlanes = FP8 ? 1 : 2;

struct MoeWork {
    double *logits;        // [splits][T][E] parts
    int splits;
    ActiveExpert *active;  // [min(P, E)], those that tokens chose first, the others with no pairs
    float *pair_weight;    // [P], by (expert, token)
    uint16_t *act;         // [planes][P][I]: bf16, and (kActPlanes) what that rounding lost in bf16 again
    int64_t act_plane;     // bytes of one
};

// ----------------------------------------------------------------- router

// logits[t][e] in 64 bits, so that a choice does not depend on fp32's order of a sum, and in one order, so that it does
// not depend on the batch: chunks of eight values lie in `leaves` classes, chunk v in class v % leaves; a class is a
// sum of its own, four chunks at a time and value by value of them; and the classes are the leaves of a binary tree.
__host__ __device__ inline int logit_leaves(int V)
{
    int n = 4 * kLogitSplits;  // (one a wave at least)
    while (n < kLogitLeaves && n * 4 < V)
        n *= 2;
    return n;
}

// Eight values of a row, zeros where there are none.
template <bool F32>
struct Chunk {
    u32x4 bits[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *row, int v, int V)
    {
        const u32x4 none = {};
#pragma unroll
        for (int h = 0; h < (F32 ? 2 : 1); ++h) {
            const u32x4 b = static_cast<const u32x4 *>(row)[int64_t(v < V ? v : V - 1) * (F32 ? 2 : 1) + h];
            bits[h] = v < V ? b : none;
        }
    }
    __device__ __forceinline__ double at(int i) const
    {
        if constexpr (F32)
            return __uint_as_float(bits[i >> 2][i & 3]);
        else
            return i & 1 ? bf16_hi(bits[0][i >> 1]) : bf16_lo(bits[0][i >> 1]);
    }
};
template <bool F32>
__device__ __forceinline__ const void *router_row(const void *w, int e, int V)
{
    return static_cast<const u32x4 *>(w) + int64_t(e) * V * (F32 ? 2 : 1);
}

// One token: an expert a block, a class a thread (H = 7168, 256 experts: 4.9 us, on the matrix cores 8.3).
template <bool F32>
__global__ __launch_bounds__(256) void moe_logits_one_kernel(const u32x4 *x, const void *w_router, int E, int V, double *logits)
{
    __shared__ double red[4];
    const int leaves = logit_leaves(V), leaf = threadIdx.x;
    const void *row = router_row<F32>(w_router, blockIdx.x, V);
    double acc = 0;
    if (leaf < leaves)
        for (int v = leaf; v < V; v += 4 * leaves) {
            Chunk<F32> w[4];
            Chunk<false> q[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                w[g].load(row, v + g * leaves, V);
                q[g].load(x, v + g * leaves, V);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    acc = fma(w[g].at(i), q[g].at(i), acc);
        }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        acc += __shfl_xor(acc, d);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = acc;
    __syncthreads();
    if (threadIdx.x == 0)
        logits[blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// More: 16 experts by 16 tokens a block on the matrix cores, whose 64-bit instruction adds its four products one after the
// other, each rounded, as fma() does.  A wave has whole branches of the tree, gridDim.z blocks share a tile's.
template <bool F32>
__global__ __launch_bounds__(256) void moe_logits_kernel(const u32x4 *x, const void *w_router, int T, int E, int V,
                                                         double *logits)
{
    typedef double f64x4 __attribute__((ext_vector_type(4)));
    __shared__ double sums[4][16][16];
    constexpr int kOnce = 8, kLevels = 3;  // classes whose loads are in flight together; levels above them inside a wave
    static_assert(kLogitLeaves / 4 <= kOnce << kLevels, "a wave's branches");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
    const int e = e0 + (lane & 15) < E ? e0 + (lane & 15) : E - 1, t = t0 + (lane & 15) < T ? t0 + (lane & 15) : T - 1;
    const void *row = router_row<F32>(w_router, e, V), *token = router_row<false>(x, t, V);
    const int leaves = logit_leaves(V), per = leaves / (4 * int(gridDim.z));
    f64x4 left[kLevels], sum = {};  // of a level's pair, the first
    for (int n = 0; n * kOnce < per; ++n) {
        const int first = (int(blockIdx.z) * 4 + wave) * per + n * kOnce;
        f64x4 acc[kOnce] = {};
        for (int v0 = first; v0 < V; v0 += 4 * leaves) {
            Chunk<F32> w[kOnce];
            Chunk<false> q[kOnce];
#pragma unroll
            for (int k = 0; k < kOnce; ++k)
                if (k < per) {
                    w[k].load(row, v0 + k + (lane >> 4) * leaves, V);
                    q[k].load(token, v0 + k + (lane >> 4) * leaves, V);
                }
#pragma unroll
            for (int k = 0; k < kOnce; ++k)
                if (k < per)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        acc[k] = __builtin_amdgcn_mfma_f64_16x16x4f64(w[k].at(c), q[k].at(c), acc[k], 0, 0, 0);
        }
#pragma unroll
        for (int d = 1; d < kOnce; d <<= 1)
#pragma unroll
            for (int k = 0; k < kOnce; k += 2 * d)
                acc[k] += acc[k + d];
        sum = acc[0];
        bool pair = true;  // (a binary counter: where a level's first is there, the two go up together)
#pragma unroll
        for (int k = 0; k < kLevels; ++k) {
            const bool second = n >> k & 1;
            if (pair && second)
                sum = left[k] + sum;
            else if (pair)
                left[k] = sum;
            pair = pair && second;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)  // expert 4 k + l / 16, token l % 16
        sums[wave][lane & 15][4 * k + (lane >> 4)] = sum[k];
    __syncthreads();
    const int i = threadIdx.x >> 4, j = threadIdx.x & 15;
    if (t0 + i < T && e0 + j < E)
        logits[(int64_t(blockIdx.z) * T + t0 + i) * E + e0 + j] =
            (sums[0][i][j] + sums[1][i][j]) + (sums[2][i][j] + sums[3][i][j]);
}

// The sum of the blocks' parts, the upper levels of their tree, all loads in flight; -inf past the last expert.
__device__ __forceinline__ float logit_of(const MoeWork &work, int T, int E, int t, int e)
{
    double part[kLogitSplits] = {};
#pragma unroll
    for (int i = 0; i < kLogitSplits; ++i)
        if (i < work.splits && e < E)
            part[i] = work.logits[(int64_t(i) * T + t) * E + e];
#pragma unroll
    for (int n = kLogitSplits / 2; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i)
            part[i] = part[2 * i] + part[2 * i + 1];
    return e < E ? float(part[0]) : -INFINITY;
}

// The logit of expert e out of the lane that has it.
template <int V>
__device__ __forceinline__ float held_logit(const float (&l)[V], int e)
{
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float o = __shfl(l[j], e & 63);
        v = e >> 6 == j ? o : v;
    }
    return v;
}

// All tokens' choices, and the pairs by expert: bit t of an expert's mask is token t.
template <int V>
__global__ __launch_bounds__(1024) void moe_select_kernel(RouteRule r, int T, MoeWork work, int64_t *topk_idx, float *topk_weights)
{
    __shared__ double scratch[16][V * 64];
    __shared__ float row[16][V * 64], weights[kMoeTokens * kMaxTopk];
    __shared__ int16_t ids[kMoeTokens * kMaxTopk];
    __shared__ unsigned long long mask[kWaveExperts];
    __shared__ int start[kWaveExperts];
    __shared__ uint32_t totals[kWaveExperts / 64];
    __shared__ int used;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (threadIdx.x < kWaveExperts)
        mask[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t live = live_experts<V>(r, lane);
    float bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        bias[j] = r.bias != nullptr && j * 64 + lane < r.experts ? r.bias[j * 64 + lane] : 0.0f;
    for (int t = wave; t < T; t += 16) {
        float l[V], s[V] = {}, w;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = j * 64 + lane;
            l[j] = logit_of(work, T, r.experts, t, e);
            row[wave][e] = l[j];
        }
        const int e = route_row(r, l, bias, live, lane, scratch[wave], false, false, s, [&](int i) { return row[wave][i]; }, w);
        if (lane < r.topk) {
            topk_idx[t * r.topk + lane] = e;
            topk_weights[t * r.topk + lane] = w;
            ids[t * r.topk + lane] = int16_t(e);
            weights[t * r.topk + lane] = w;
            if (e >= 0)
                atomicOr(&mask[e], 1ull << t);
        }
    }
    __syncthreads();
    // experts before this one, and their pairs
    uint32_t own = 0, before = 0;
    if (threadIdx.x < kWaveExperts) {
        const uint32_t n = __popcll(mask[threadIdx.x]);
        own = n << 16 | (n > 0);
        before = wave_scan(own);
        if (lane == 63)
            totals[wave] = before;
    }
    __syncthreads();
    if (threadIdx.x < kWaveExperts) {
        before -= own;
        for (int w = 0; w < wave; ++w)
            before += totals[w];
        start[threadIdx.x] = int(before >> 16);
        if (own != 0)
            work.active[before & 0xffff] =
                ActiveExpert{int(threadIdx.x), int(before >> 16), int(own >> 16), 0, mask[threadIdx.x]};
        if (threadIdx.x == kWaveExperts - 1)
            used = int((before + own) & 0xffff);
    }
    __syncthreads();
    const int room = T * r.topk < r.experts ? T * r.topk : r.experts;
    for (int i = used + int(threadIdx.x); i < room; i += 1024)
        work.active[i] = ActiveExpert{};
    for (int i = threadIdx.x; i < T * r.topk; i += 1024) {
        const int t = i / r.topk;
        const int e = ids[i];
        if (e >= 0)
            work.pair_weight[start[e] + __popcll(mask[e] & ((1ull << t) - 1))] = weights[i];
    }
}

// ---------------------------------------------------------------- experts

struct MoeArgs {
    MoeWork work;
    const char *p;         // weights [E][rows][K]
    const float *p_scale;  // FP8: [E][rows / 128][K / 128]
    const char *q;         // token rows (or activations), bf16
    int I, H, T;
    int kbytes;            // bytes of a weight row
};

// act of 16 G gate and their up columns for up to 16 / C * MT tokens of one expert.
constexpr int kGateWaves = 8, kGateSums = 2 * 32 * 16;  // floats of a wave's sums
template <bool FP8, bool TAIL, int G, int C, int MT>
__device__ __forceinline__ void gate_tile(const MoeArgs &a, const ActiveExpert &x, int n0, int m0, float *sums)
{
    constexpr int kRows = 16 / C, RG = C * G, RT = 2 * RG;  // of a tile; tiles: RG of the gate, RG of up
    constexpr int kTokens = kRows * MT, kCols = 16 * G;
    static_assert(2 * kTokens * kCols <= kGateSums, "the sums' place");
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), i0 = (lane & 15) / C;
    const char *w = a.p + int64_t(x.expert) * 2 * a.I * a.kbytes;
    const int steps = (a.kbytes + kStepBytes - 1) / kStepBytes;
    const char *prow[RT];
    const float *scale[RT] = {};
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int n = n0 + r % RG * kRows + i0;
        prow[r] = w + (int64_t(r / RG) * a.I + (n < a.I ? n : a.I - 1)) * a.kbytes;
        if constexpr (FP8)  // (a block's columns lie in one scale block: they divide 128)
            scale[r] = a.p_scale + ((int64_t(x.expert) * 2 + r / RG) * (a.I >> 7) + (n0 >> 7)) * steps;
    }
    const char *qrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int i = m0 + m * kRows + i0;
        qrow[m] = a.q + int64_t(token_of(x.tokens, i < x.count ? i : x.count - 1)) * a.H * 2;
    }
    f32x4 acc[RT][MT] = {};
    stream<FP8, TAIL, ahead(FP8, C, RT, MT), C>(prow, scale, qrow, steps * wave / kGateWaves,
                                                steps * (wave + 1) / kGateWaves, a.kbytes, lane, acc);
    // the waves' sums, [wave][gate, up][token][columns]
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float *to = sums + wave * kGateSums + (r / RG * kTokens + m * kRows + i0) * kCols + r % RG * kRows;
            if constexpr (C == 1)
                *reinterpret_cast<f32x4 *>(to + (lane >> 4) * 4) = acc[r][m];
            else
                to[(lane >> 4) * 2 + (lane & 1)] = fold(acc[r][m], lane);
        }
    __syncthreads();
    const int i = threadIdx.x / (kCols / 4), c = threadIdx.x % (kCols / 4) * 4;
    if (i < kTokens) {
        f32x4 gate = {}, up = {};
#pragma unroll
        for (int w8 = 0; w8 < kGateWaves; ++w8) {
            gate += *reinterpret_cast<const f32x4 *>(sums + w8 * kGateSums + i * kCols + c);
            up += *reinterpret_cast<const f32x4 *>(sums + w8 * kGateSums + (kTokens + i) * kCols + c);
        }
        f32x4 v;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = gate[k] * sigmoidf(gate[k]) * up[k];
        if (m0 + i < x.count && n0 + c < a.I) {
            const int64_t at = int64_t(x.start + m0 + i) * a.I + n0 + c;
            const uint2 b = pack4(v);
            *reinterpret_cast<uint2 *>(a.work.act + at) = b;
            if constexpr (kActPlanes<FP8> == 2)
                *reinterpret_cast<uint2 *>(a.work.act + a.work.act_plane / 2 + at) = pack4(lost(v, b));
        }
    }
    __syncthreads();
}

// Few tokens (V > 0): each block chooses for itself, which takes less than a launch in between; the first block
// writes the choice down.  One token:
struct MoeChoice {
    RouteRule rule;
    int64_t *topk_idx;
    float *topk_weights;
};
template <int V>
__device__ __forceinline__ ActiveExpert choose_one(const MoeArgs &a, const MoeChoice &c, float *lds)
{
    __shared__ int chosen[kMaxTopk];
    const RouteRule &r = c.rule;
    const int lane = threadIdx.x & 63;
    if (threadIdx.x < 64) {
        float l[V], s[V] = {}, bias[V], w;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = j * 64 + lane;
            l[j] = logit_of(a.work, 1, r.experts, 0, e);
            bias[j] = r.bias != nullptr && e < r.experts ? r.bias[e] : 0.0f;
        }
        const int e = route_row(r, l, bias, live_experts<V>(r, lane), lane, reinterpret_cast<double *>(lds), false, false, s,
                                [&](int i) { return held_logit(l, i); }, w);
        chosen[lane] = e;
        if (blockIdx.x == 0 && blockIdx.y == 0 && lane < r.topk) {
            c.topk_idx[lane] = e;
            c.topk_weights[lane] = w;
            if (lane < int(gridDim.y)) {
                a.work.active[lane] = ActiveExpert{e, lane, e >= 0, 0, 1};
                a.work.pair_weight[lane] = w;
            }
        }
    }
    __syncthreads();
    const int e = uniform(chosen[blockIdx.y]);
    return ActiveExpert{e, int(blockIdx.y), e >= 0, 0, 1};
}

// Up to a token a wave: each wave chooses for one, the block takes the blockIdx.y-th of the experts that some token
// chose (launch_moe has the rule)
constexpr int kChooseTokens = kGateWaves;
template <int V>
__device__ __forceinline__ ActiveExpert choose_few(const MoeArgs &a, const MoeChoice &c, float *lds)
{
    __shared__ uint32_t mask[kWaveExperts], totals[kGateWaves];
    __shared__ int16_t ids[kChooseTokens * kMaxTopk], start[kWaveExperts];
    __shared__ float weights[kChooseTokens * kMaxTopk];
    __shared__ ActiveExpert found;
    const RouteRule &r = c.rule;
    const int lane = threadIdx.x & 63, t = uniform(threadIdx.x >> 6), me = threadIdx.x;
    static_assert(kGateWaves * kWave == kWaveExperts, "a thread an expert");
    mask[me] = 0;
    if (me == 0)
        found = ActiveExpert{};
    __syncthreads();
    if (t < a.T) {
        float l[V], s[V] = {}, bias[V], w;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = j * 64 + lane;
            l[j] = logit_of(a.work, a.T, r.experts, t, e);
            bias[j] = r.bias != nullptr && e < r.experts ? r.bias[e] : 0.0f;
        }
        double *scratch = reinterpret_cast<double *>(lds) + t * V * 64;
        const int e = route_row(r, l, bias, live_experts<V>(r, lane), lane, scratch, false, false, s,
                                [&](int i) { return held_logit(l, i); }, w);
        if (lane < r.topk) {
            ids[t * r.topk + lane] = int16_t(e);
            weights[t * r.topk + lane] = w;
            if (e >= 0)
                atomicOr(&mask[e], 1u << t);
        }
    }
    __syncthreads();
    const uint32_t n = __popc(mask[me]), own = n << 16 | (n > 0);
    uint32_t before = wave_scan(own);
    if (lane == 63)
        totals[t] = before;
    __syncthreads();
    before -= own;
    uint32_t all = 0;
#pragma unroll
    for (int w = 0; w < kGateWaves; ++w) {
        before += w < t ? totals[w] : 0;
        all += totals[w];
    }
    const ActiveExpert mine{me, int(before >> 16), int(n), 0, mask[me]};
    if (n > 0 && (before & 0xffff) == blockIdx.y)
        found = mine;
    if (blockIdx.x == 0 && blockIdx.y == 0) {  // the records, for the next launch and the caller
        start[me] = int16_t(before >> 16);
        if (n > 0)
            a.work.active[before & 0xffff] = mine;
        for (int i = int(all & 0xffff) + me; i < int(gridDim.y); i += kGateWaves * kWave)
            a.work.active[i] = ActiveExpert{};
        __syncthreads();
        for (int i = me; i < a.T * r.topk; i += kGateWaves * kWave) {
            const int e = ids[i];
            c.topk_idx[i] = e;
            c.topk_weights[i] = weights[i];
            if (e >= 0)
                a.work.pair_weight[start[e] + __popc(mask[e] & ((1u << i / r.topk) - 1))] = weights[i];
        }
    }
    __syncthreads();
    ActiveExpert x = found;
    x.expert = uniform(x.expert);
    x.start = uniform(x.start);
    x.count = uniform(x.count);
    return x;
}

// 32 columns a block, so that the tokens' loads serve twice the weights, where an expert's tokens are few; else 16 by 16.
template <bool FP8, bool TAIL, int V, bool ONE>
__global__ __launch_bounds__(kGateWaves *kWave) void moe_gate_kernel(MoeArgs a, MoeChoice c)
{
    __shared__ __attribute__((aligned(16))) float sums[kGateWaves * kGateSums];
    constexpr int G = 2;
    const int n0 = blockIdx.x * 16 * G;
    if constexpr (V > 0) {
        ActiveExpert x;
        if constexpr (ONE)
            x = choose_one<V>(a, c, sums);
        else
            x = choose_few<V>(a, c, sums);
        if (x.count > 0)
            gate_tile<FP8, TAIL, G, 2, 1>(a, x, n0, 0, sums);
        return;
    }
    const ActiveExpert x = a.work.active[blockIdx.y];
    if (x.count <= 8) {
        if (x.count > 0)
            gate_tile<FP8, TAIL, G, 2, 1>(a, x, n0, 0, sums);
        return;
    }
    for (int g = 0; g < G && n0 + g * 16 < a.I; ++g)
        for (int m0 = 0; m0 < x.count; m0 += 32) {
            if (x.count - m0 > 16)
                gate_tile<FP8, TAIL, 1, 1, 2>(a, x, n0 + g * 16, m0, sums);
            else
                gate_tile<FP8, TAIL, 1, 2, 2>(a, x, n0 + g * 16, m0, sums);
        }
}

// COLS columns of y for every token: the block's waves share out the experts (each in `parts` pieces of
// K), a wave adds each piece's weighted product to its own sums [token][COLS] in LDS.
template <bool FP8, bool TAIL, int COLS, int C, int MT>
__device__ __forceinline__ void down_piece(const MoeArgs &a, const ActiveExpert &x, int n0, int m0, int s0, int s1, float *own)
{
    constexpr int kRows = 16 / C, RT = COLS / kRows;
    const int lane = threadIdx.x & 63, i0 = (lane & 15) / C;
    const int steps = (a.kbytes + kStepBytes - 1) / kStepBytes;
    const char *prow[RT];
    const float *scale[RT] = {};
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int n = n0 + r * kRows + i0;
        prow[r] = a.p + (int64_t(x.expert) * a.H + (n < a.H ? n : a.H - 1)) * a.kbytes;
        if constexpr (FP8)
            scale[r] = a.p_scale + (int64_t(x.expert) * (a.H >> 7) + (n0 >> 7)) * steps;
    }
    const char *qrow[MT];
    int token[MT];
    float weight[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int i = m0 + m * kRows + i0, at = x.start + (i < x.count ? i : x.count - 1);
        qrow[m] = a.q + int64_t(at) * a.I * 2;
        token[m] = i < x.count ? token_of(x.tokens, i) : -1;
        weight[m] = a.work.pair_weight[at];
    }
    f32x4 acc[RT][MT] = {};
    constexpr int PLANES = kActPlanes<FP8>;
    stream<FP8, TAIL, ahead(FP8, C, RT, MT, PLANES), C, PLANES>(prow, scale, qrow, s0, s1, a.kbytes, lane, acc,
                                                                a.work.act_plane);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if constexpr (C == 1) {
                if (token[m] >= 0)
                    *reinterpret_cast<f32x4 *>(own + token[m] * COLS + r * kRows + (lane >> 4) * 4) += acc[r][m] * weight[m];
            } else {
                const float v = fold(acc[r][m], lane) * weight[m];
                if (token[m] >= 0)
                    own[token[m] * COLS + r * kRows + (lane >> 4) * 2 + (lane & 1)] += v;
            }
        }
}

constexpr int kDownWaves = 8;
template <bool FP8, bool TAIL, int COLS>
__global__ __launch_bounds__(kDownWaves *kWave) void moe_down_kernel(MoeArgs a, int room, const uint16_t *residual, uint16_t *y)
{
    constexpr int W = kDownWaves, Q = COLS / 4;  // Q: vectors of a token's columns
    extern __shared__ f32x4 own[];               // [W][T][Q]
    __shared__ ActiveExpert list[kMoeExperts];
    __shared__ int used[W];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int n0 = blockIdx.x * COLS;
    const f32x4 zero = {};
    for (int i = lane; i < a.T * Q; i += 64)
        own[wave * a.T * Q + i] = zero;
    int n = 0;
    for (int i = threadIdx.x; i < room; i += W * kWave) {
        list[i] = a.work.active[i];
        n += list[i].count > 0;
    }
    n = int(wave_scan(uint32_t(n)));
    if (lane == 63)
        used[wave] = n;
    __syncthreads();
    int experts = 0;
#pragma unroll
    for (int w = 0; w < W; ++w)
        experts += used[w];
    experts = uniform(experts);
    const int steps = (a.kbytes + kStepBytes - 1) / kStepBytes;
    int parts = experts > 0 ? (W + experts - 1) / experts : 1;
    parts = parts < steps ? parts : steps;
    float *sums = reinterpret_cast<float *>(own + wave * a.T * Q);
    for (int i = wave; i < experts * parts; i += W) {
        ActiveExpert x = list[i / parts];
        x.expert = uniform(x.expert);
        x.start = uniform(x.start);
        x.count = uniform(x.count);
        const int part = i % parts, s0 = steps * part / parts, s1 = steps * (part + 1) / parts;
        for (int m0 = 0; m0 < x.count; m0 += 32) {
            if (x.count - m0 > 16) {
                if constexpr (COLS == 16)
                    down_piece<FP8, TAIL, COLS, 1, 2>(a, x, n0, m0, s0, s1, sums);
                else
                    down_piece<FP8, TAIL, COLS, 2, 4>(a, x, n0, m0, s0, s1, sums);
            } else if (x.count - m0 > 8)
                down_piece<FP8, TAIL, COLS, 2, 2>(a, x, n0, m0, s0, s1, sums);
            else
                down_piece<FP8, TAIL, COLS, 2, 1>(a, x, n0, m0, s0, s1, sums);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * Q; i += W * kWave) {
        const int c = n0 + i % Q * 4;
        if (c >= a.H)
            continue;
        f32x4 v = own[i];
#pragma unroll
        for (int w = 1; w < W; ++w)
            v += own[w * a.T * Q + i];
        const int64_t at = int64_t(i / Q) * a.H + c;
        if (residual != nullptr) {
            const uint2 b = *reinterpret_cast<const uint2 *>(residual + at);
            v[0] += bf16_lo(b.x), v[1] += bf16_hi(b.x), v[2] += bf16_lo(b.y), v[3] += bf16_hi(b.y);
        }
        *reinterpret_cast<uint2 *>(y + at) = pack4(v);
    }
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Blocks that share a tile's K: at most 256 in all, and whole branches of the classes' tree.
int logit_splits(int T, int E)
{
    if (T <= 1)
        return 1;
    const int tiles = (E + 15) / 16 * ((T + 15) / 16);
    int n = kLogitSplits;
    while (n > 1 && n * tiles > 256)
        n /= 2;
    return n;
}

// Lays the workspace out at base; returns its bytes.
size_t moe_layout(int T, int E, int K, int I, char *base, MoeWork *w)
{
    const size_t P = size_t(T) * K, n = P < size_t(E) ? P : size_t(E);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *p = base + at;
        at += up256(bytes);
        return p;
    };
    MoeWork m;
    m.splits = logit_splits(T, E);
    m.logits = reinterpret_cast<double *>(take(size_t(m.splits) * T * E * 8));
    m.active = reinterpret_cast<ActiveExpert *>(take(n * sizeof(ActiveExpert)));
    m.pair_weight = reinterpret_cast<float *>(take(P * 4));
    m.act_plane = int64_t(up256(P * I * 2));
    m.act = reinterpret_cast<uint16_t *>(take(2 * m.act_plane));
    if (w != nullptr)
        *w = m;
    return at;
}

}  // namespace

size_t moe_workspace(int T, int E, int K, int I) { return moe_layout(T, E, K, I, nullptr, nullptr); }

hipError_t launch_moe(const RouteRule &rule, const MoeCall &c, hipStream_t stream)
{
    MoeArgs a{};
    moe_layout(c.T, rule.experts, rule.topk, c.I, static_cast<char *>(c.workspace), &a.work);
    const int E = rule.experts, V = c.H / 8;
    const bool fp8 = c.w13_scale != nullptr;
    const int most = c.T * rule.topk < E ? c.T * rule.topk : E;
    if (log_enabled())
        log_launch("ll_moe: T=%d H=%d I=%d E=%d K=%d%s", c.T, c.H, c.I, E, rule.topk, fp8 ? " fp8" : "");
    const u32x4 *x = static_cast<const u32x4 *>(c.x);
    if (c.T == 1)
        hipLaunchKernelGGL((c.router_f32 ? moe_logits_one_kernel<true> : moe_logits_one_kernel<false>), dim3(E), dim3(256), 0,
                           stream, x, c.w_router, E, V, a.work.logits);
    else
        hipLaunchKernelGGL((c.router_f32 ? moe_logits_kernel<true> : moe_logits_kernel<false>),
                           dim3((E + 15) / 16, (c.T + 15) / 16, a.work.splits), dim3(256), 0, stream, x, c.w_router, c.T, E, V,
                           a.work.logits);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    // The gate's blocks choose for themselves for one token (eight experts of 768 x 2048: 20.2 us, with a launch
    // for it 23.5), and for up to eight where no block has to wait for another's choice (2 tokens, 6 of 24 experts of 520 x
    // 1000: 17.3 against 19.1; with 4 blocks a compute unit, 8 tokens, 64 experts of 768 x 2048, 101 against 87).
    const unsigned gate_columns = unsigned(c.I + 31) / 32;
    const bool inside = c.T == 1 || (c.T <= kChooseTokens && int64_t(gate_columns) * most <= compute_units());
    if (!inside) {
        auto select = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3(1), dim3(1024), 0, stream, rule, c.T, a.work, c.topk_idx, c.topk_weights);
        };
        if (E <= 64)
            select(moe_select_kernel<1>);
        else if (E <= 128)
            select(moe_select_kernel<2>);
        else if (E <= 256)
            select(moe_select_kernel<4>);
        else
            select(moe_select_kernel<8>);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    a.I = c.I;
    a.H = c.H;
    a.T = c.T;
    a.p = static_cast<const char *>(c.w13);
    a.p_scale = c.w13_scale;
    a.q = static_cast<const char *>(c.x);
    a.kbytes = c.H * (fp8 ? 1 : 2);
    const MoeChoice choice{rule, c.topk_idx, c.topk_weights};
    auto gate = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(gate_columns, most), dim3(kGateWaves * kWave), 0, stream, a, choice);
    };
    auto gates = [&](auto experts, auto one) {
        constexpr int V = decltype(experts)::value;
        constexpr bool ONE = decltype(one)::value;
        if (fp8)
            gate(moe_gate_kernel<true, false, V, ONE>);
        else if (a.kbytes % kStepBytes == 0)
            gate(moe_gate_kernel<false, false, V, ONE>);
        else
            gate(moe_gate_kernel<false, true, V, ONE>);
    };
    auto by_experts = [&](auto one) {
        if (E <= 64)
            gates(std::integral_constant<int, 1>(), one);
        else if (E <= 256)
            gates(std::integral_constant<int, 4>(), one);
        else
            gates(std::integral_constant<int, 8>(), one);
    };
    if (!inside)
        gates(std::integral_constant<int, 0>(), std::false_type());
    else if (c.T > 1)
        by_experts(std::false_type());
    else
        by_experts(std::true_type());
    e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    a.p = static_cast<const char *>(c.w2);
    a.p_scale = c.w2_scale;
    a.q = reinterpret_cast<const char *>(a.work.act);
    a.kbytes = c.I * (fp8 ? 1 : 2);
    auto down = [&](auto cols) {
        constexpr int COLS = decltype(cols)::value;
        auto go = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3((c.H + COLS - 1) / COLS), dim3(kDownWaves * kWave),
                               size_t(kDownWaves) * c.T * COLS * 4, stream, a, most, static_cast<const uint16_t *>(c.residual),
                               static_cast<uint16_t *>(c.y));
        };
        if (fp8)
            go(moe_down_kernel<true, false, COLS>);
        else if (a.kbytes % kStepBytes == 0)
            go(moe_down_kernel<false, false, COLS>);
        else
            go(moe_down_kernel<false, true, COLS>);
    };
    // 8 columns a block where blocks of 16 would be fewer than the compute units (H = 2048, eight experts of 768: 6.6
    // against 8.2 us, with activations of one bf16 value; where they are not, 16 share the activations' loads: H = 7168, FP8, 24.9 against 32)
    if (c.H < 16 * compute_units())
        down(std::integral_constant<int, 8>());
    else
        down(std::integral_constant<int, 16>());
    return hipGetLastError();
}

}  // namespace ep
