// moe.hip -- a whole mixture-of-experts layer for a few tokens: router, experts and
// weighted sum, without packing rows in between.
//   logits = x Wr^T, route (route.h), y[t] = residual[t] + sum_k w_k (silu(x Wg^T) * (x Wu^T)) W2^T
// The weights of the reached experts are read once and are the cost.  They go straight from
// memory into the matrix instruction's registers, 16 weight rows by the tokens of one
// expert, K shared out over the waves of a block, each keeping kAhead steps of 128 bytes a row
// in flight.  FP8 weights are widened to bf16 there, exactly, so that rows and
// activations keep their bf16 values.
#include "route.h"
#include "stream.h"

namespace ep {

namespace {

constexpr int kAhead = 4;

struct ActiveExpert {
    int32_t expert, start, count, unused;  // its pairs: [start, start + count)
};

struct MoeWork {
    float *logits;         // [T][E]
    int32_t *active_count;
    ActiveExpert *active;  // [min(P, E)]
    int32_t *pair_token;   // [P], sorted by (expert, token)
    float *pair_weight;    // [P]
    uint16_t *act;         // [P][I]
};

// ----------------------------------------------------------------- router

// One expert a block, up to TT tokens: logits[t][e] in 64 bits, so that a choice depends neither on the batch
// nor on the order of a sum.
template <int TT, bool F32>
__global__ __launch_bounds__(256) void moe_logits_kernel(const u32x4 *x, const void *w_router, int T, int E, int V,
                                                         float *logits)
{
    __shared__ double red[4][TT];
    const int e = blockIdx.x, t0 = blockIdx.y * TT;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double acc[TT] = {};
    for (int v = threadIdx.x; v < V; v += 256) {
        double w[8];
        if constexpr (F32) {
            const float4 *p = static_cast<const float4 *>(w_router) + (int64_t(e) * V + v) * 2;
            const float4 a = p[0], b = p[1];
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        } else {
            const u32x4 a = static_cast<const u32x4 *>(w_router)[int64_t(e) * V + v];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w[2 * q] = bf16_lo(a[q]), w[2 * q + 1] = bf16_hi(a[q]);
        }
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const int t = t0 + i < T ? t0 + i : T - 1;
            const u32x4 b = x[int64_t(t) * V + v];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                acc[i] = fma(w[2 * q], double(bf16_lo(b[q])), acc[i]);
                acc[i] = fma(w[2 * q + 1], double(bf16_hi(b[q])), acc[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        acc[i] = wave_sum(acc[i]);
        if (lane == 0)
            red[wave][i] = acc[i];
    }
    __syncthreads();
    if (threadIdx.x < TT && t0 + int(threadIdx.x) < T) {
        const int i = threadIdx.x;
        logits[int64_t(t0 + i) * E + e] = float(red[0][i] + red[1][i] + red[2][i] + red[3][i]);
    }
}

// All tokens' choices, and the pairs by expert: bit t of an expert's mask is token t.
template <int V>
__global__ __launch_bounds__(1024) void moe_select_kernel(RouteRule r, int T, MoeWork work, int64_t *topk_idx, float *topk_weights)
{
    __shared__ double scratch[16][V * 64];
    __shared__ unsigned long long mask[kWaveExperts];
    __shared__ int start[kWaveExperts];
    __shared__ uint32_t totals[kWaveExperts / 64];
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
        const float *row = work.logits + int64_t(t) * r.experts;
        float l[V], s[V] = {}, w;
#pragma unroll
        for (int j = 0; j < V; ++j)
            l[j] = j * 64 + lane < r.experts ? row[j * 64 + lane] : -INFINITY;
        const int e = route_row(r, l, bias, live, lane, scratch[wave], false, s, [&](int i) { return row[i]; }, w);
        if (lane < r.topk) {
            topk_idx[t * r.topk + lane] = e;
            topk_weights[t * r.topk + lane] = w;
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
            work.active[before & 0xffff] = ActiveExpert{int(threadIdx.x), int(before >> 16), int(own >> 16), 0};
        if (threadIdx.x == kWaveExperts - 1)
            *work.active_count = int((before + own) & 0xffff);
    }
    __syncthreads();
    // (this block's own stores)
    for (int i = threadIdx.x; i < T * r.topk; i += 1024) {
        const int t = i / r.topk;
        const int e = int(topk_idx[i]);
        if (e >= 0) {
            const int at = start[e] + __popcll(mask[e] & ((1ull << t) - 1));
            work.pair_token[at] = t;
            work.pair_weight[at] = topk_weights[i];
        }
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

// act of 16 gate and their 16 up columns for the tokens of one expert.
constexpr int kGateWaves = 8;
template <bool FP8, bool TAIL, int MT>
__device__ __forceinline__ void gate_tile(const MoeArgs &a, const ActiveExpert &x, int n0, int m0, f32x4 *sums)
{
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int n = n0 + (lane & 15) < a.I ? n0 + (lane & 15) : a.I - 1;
    const char *w = a.p + int64_t(x.expert) * 2 * a.I * a.kbytes;
    const char *prow[2] = {w + int64_t(n) * a.kbytes, w + int64_t(a.I + n) * a.kbytes};
    const int steps = (a.kbytes + kStepBytes - 1) / kStepBytes;
    const float *scale[2] = {};
    if constexpr (FP8) {
        scale[0] = a.p_scale + (int64_t(x.expert) * 2 * (a.I >> 7) + (n0 >> 7)) * steps;
        scale[1] = scale[0] + int64_t(a.I >> 7) * steps;
    }
    const char *qrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int i = m0 + m * 16 + (lane & 15);
        qrow[m] = a.q + int64_t(a.work.pair_token[x.start + (i < x.count ? i : x.count - 1)]) * a.H * 2;
    }
    f32x4 acc[2][MT] = {};
    stream<FP8, TAIL, kAhead>(prow, scale, qrow, steps * wave / kGateWaves, steps * (wave + 1) / kGateWaves, a.kbytes, lane, acc);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m)
            sums[(wave * 2 * MT + h * MT + m) * kWave + lane] = acc[h][m];
    __syncthreads();
    if (wave < MT) {
        const int m = wave;
        f32x4 gate = {}, up = {};
#pragma unroll
        for (int w8 = 0; w8 < kGateWaves; ++w8) {
            gate += sums[(w8 * 2 * MT + m) * kWave + lane];
            up += sums[(w8 * 2 * MT + MT + m) * kWave + lane];
        }
        const int i = m0 + m * 16 + (lane & 15), c = n0 + (lane >> 4) * 4;
        f32x4 v;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = gate[k] * sigmoidf(gate[k]) * up[k];
        if (i < x.count && c < a.I)
            *reinterpret_cast<uint2 *>(a.work.act + int64_t(x.start + i) * a.I + c) = pack4(v);
    }
    __syncthreads();
}

template <bool FP8, bool TAIL>
__global__ __launch_bounds__(kGateWaves *kWave) void moe_gate_kernel(MoeArgs a)
{
    __shared__ f32x4 sums[kGateWaves * 2 * 2 * kWave];
    if (int(blockIdx.y) >= *a.work.active_count)
        return;
    const ActiveExpert x = a.work.active[blockIdx.y];
    const int n0 = blockIdx.x * 16;
    for (int m0 = 0; m0 < x.count; m0 += 32) {
        if (x.count - m0 > 16)
            gate_tile<FP8, TAIL, 2>(a, x, n0, m0, sums);
        else
            gate_tile<FP8, TAIL, 1>(a, x, n0, m0, sums);
    }
}

// 16 columns of y for every token: the block's waves share out the experts (each in `parts` pieces of
// K), a wave adds each piece's weighted product to its own sums in LDS.
template <bool FP8, bool TAIL, int MT>
__device__ __forceinline__ void down_piece(const MoeArgs &a, const ActiveExpert &x, int n0, int m0, int s0, int s1, f32x4 *own)
{
    const int lane = threadIdx.x & 63;
    const int n = n0 + (lane & 15) < a.H ? n0 + (lane & 15) : a.H - 1;
    const char *prow[1] = {a.p + (int64_t(x.expert) * a.H + n) * a.kbytes};
    const int steps = (a.kbytes + kStepBytes - 1) / kStepBytes;
    const float *scale[1] = {};
    if constexpr (FP8)
        scale[0] = a.p_scale + (int64_t(x.expert) * (a.H >> 7) + (n0 >> 7)) * steps;
    const char *qrow[MT];
    int token[MT];
    float weight[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int i = m0 + m * 16 + (lane & 15), at = x.start + (i < x.count ? i : x.count - 1);
        qrow[m] = a.q + int64_t(at) * a.I * 2;
        token[m] = i < x.count ? a.work.pair_token[at] : -1;
        weight[m] = a.work.pair_weight[at];
    }
    f32x4 acc[1][MT] = {};
    stream<FP8, TAIL, kAhead>(prow, scale, qrow, s0, s1, a.kbytes, lane, acc);
#pragma unroll
    for (int m = 0; m < MT; ++m)
        if (token[m] >= 0)
            own[token[m] * 4 + (lane >> 4)] += acc[0][m] * weight[m];
}

template <int W, bool FP8, bool TAIL>
__global__ __launch_bounds__(W *kWave) void moe_down_kernel(MoeArgs a, const uint16_t *residual, uint16_t *y)
{
    extern __shared__ f32x4 own[];  // [W][T][4]
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16;
    const f32x4 zero = {};
    for (int i = lane; i < a.T * 4; i += 64)
        own[wave * a.T * 4 + i] = zero;
    const int experts = uniform(*a.work.active_count);
    const int steps = (a.kbytes + kStepBytes - 1) / kStepBytes;
    int parts = experts > 0 ? (W + experts - 1) / experts : 1;
    parts = parts < steps ? parts : steps;
    for (int i = wave; i < experts * parts; i += W) {
        const ActiveExpert x = a.work.active[i / parts];
        const int part = i % parts, s0 = steps * part / parts, s1 = steps * (part + 1) / parts;
        for (int m0 = 0; m0 < x.count; m0 += 32) {
            if (x.count - m0 > 16)
                down_piece<FP8, TAIL, 2>(a, x, n0, m0, s0, s1, own + wave * a.T * 4);
            else
                down_piece<FP8, TAIL, 1>(a, x, n0, m0, s0, s1, own + wave * a.T * 4);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * 4; i += W * kWave) {
        const int n = n0 + (i & 3) * 4;
        if (n >= a.H)
            continue;
        f32x4 v = own[i];
#pragma unroll
        for (int w = 1; w < W; ++w)
            v += own[w * a.T * 4 + i];
        const int64_t at = int64_t(i >> 2) * a.H + n;
        if (residual != nullptr) {
            const uint2 b = *reinterpret_cast<const uint2 *>(residual + at);
            v[0] += bf16_lo(b.x), v[1] += bf16_hi(b.x), v[2] += bf16_lo(b.y), v[3] += bf16_hi(b.y);
        }
        *reinterpret_cast<uint2 *>(y + at) = pack4(v);
    }
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

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
    m.logits = reinterpret_cast<float *>(take(size_t(T) * E * 4));
    m.active_count = reinterpret_cast<int32_t *>(take(4));
    m.active = reinterpret_cast<ActiveExpert *>(take(n * sizeof(ActiveExpert)));
    m.pair_token = reinterpret_cast<int32_t *>(take(P * 4));
    m.pair_weight = reinterpret_cast<float *>(take(P * 4));
    m.act = reinterpret_cast<uint16_t *>(take(P * I * 2));
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
    auto logits = [&](auto bf, auto f32, int tokens) {
        hipLaunchKernelGGL(c.router_f32 ? f32 : bf, dim3(E, (c.T + tokens - 1) / tokens), dim3(256), 0, stream, x, c.w_router,
                           c.T, E, V, a.work.logits);
    };
    if (c.T == 1)
        logits(moe_logits_kernel<1, false>, moe_logits_kernel<1, true>, 1);
    else
        logits(moe_logits_kernel<8, false>, moe_logits_kernel<8, true>, 8);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
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
    a.I = c.I;
    a.H = c.H;
    a.T = c.T;
    a.p = static_cast<const char *>(c.w13);
    a.p_scale = c.w13_scale;
    a.q = static_cast<const char *>(c.x);
    a.kbytes = c.H * (fp8 ? 1 : 2);
    auto gate = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((c.I + 15) / 16, most), dim3(kGateWaves * kWave), 0, stream, a);
    };
    if (fp8)
        gate(moe_gate_kernel<true, false>);
    else if (a.kbytes % kStepBytes == 0)
        gate(moe_gate_kernel<false, false>);
    else
        gate(moe_gate_kernel<false, true>);
    e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    a.p = static_cast<const char *>(c.w2);
    a.p_scale = c.w2_scale;
    a.q = reinterpret_cast<const char *>(a.work.act);
    a.kbytes = c.I * (fp8 ? 1 : 2);
    auto down = [&](auto kernel, int waves) {
        hipLaunchKernelGGL(kernel, dim3((c.H + 15) / 16), dim3(waves * kWave), size_t(waves) * c.T * 64, stream, a,
                           static_cast<const uint16_t *>(c.residual), static_cast<uint16_t *>(c.y));
    };
    if (fp8)
        down(moe_down_kernel<8, true, false>, 8);
    else if (a.kbytes % kStepBytes == 0)
        down(moe_down_kernel<8, false, false>, 8);
    else
        down(moe_down_kernel<8, false, true>, 8);
    return hipGetLastError();
}

}  // namespace ep
