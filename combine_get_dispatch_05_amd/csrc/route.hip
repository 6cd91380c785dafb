// route.hip -- the router: the experts of each token and their weights from its
// logits, the sums that a balancing loss takes, and the gradients of both.
//   s = softmax(l) or sigmoid(l), keys s + bias (l without a bias), groups by their best keys,
//   the K largest keys; w = scale s_k, or over the sum of the chosen; sums = sum_t p, p = s / sum s
// A wave a token, the logits in registers: every byte crosses memory once, and the vector
// instructions are what the time goes into (some 850 a token with groups, 9 of them each of
// the K + 1 maxima over the wave): 8192 tokens of 256 experts in 8 groups, 8 chosen, 17 us,
// of which the 8 MB of logits are 2; one token 4.4; 4096 tokens of softmax scores with their
// sums 9 + 4, and the gradient 7.  bf16 logits take the same: 8192 tokens of 256 with a bias 15, their gradient 10.
#include "route.h"

namespace ep {

namespace {

constexpr int kRouteThreads = 256, kRouteWaves = kRouteThreads / kWave;

template <bool BF16>
__device__ __forceinline__ float logit_at(const void *logits, int64_t i)
{
    if constexpr (BF16)
        return __uint_as_float(uint32_t(static_cast<const uint16_t *>(logits)[i]) << 16);
    else
        return static_cast<const float *>(logits)[i];
}

struct RouteArgs {
    RouteRule rule;
    const void *logits;  // [T][E]
    int64_t T;
    int64_t *topk_idx;   // [T][K]
    float *weights;      // [T][K]
    float *parts;        // nullable [blocks][E]: each block's score sums
};

template <int V, bool BF16>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a)
{
    __shared__ double scratch[kRouteWaves][V * 64];
    const RouteRule &r = a.rule;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t live = live_experts<V>(r, lane);
    float bias[V], acc[V] = {};
#pragma unroll
    for (int j = 0; j < V; ++j)
        bias[j] = r.bias != nullptr && j * 64 + lane < r.experts ? r.bias[j * 64 + lane] : 0.0f;
    for (int64_t t = int64_t(blockIdx.x) * kRouteWaves + wave; t < a.T; t += int64_t(gridDim.x) * kRouteWaves) {
        float l[V], s[V] = {}, w;
#pragma unroll
        for (int j = 0; j < V; ++j)
            l[j] = j * 64 + lane < r.experts ? logit_at<BF16>(a.logits, t * r.experts + j * 64 + lane) : -INFINITY;
        const int e = route_row(r, l, bias, live, lane, scratch[wave], a.parts != nullptr, BF16, s,
                                [&](int i) { return logit_at<BF16>(a.logits, t * r.experts + i); }, w);
        if (lane < r.topk) {
            a.topk_idx[t * r.topk + lane] = e;
            a.weights[t * r.topk + lane] = w;
        }
        if (a.parts != nullptr) {
            if (r.soft) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    acc[j] += s[j];
            } else {
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < V; ++j)
                    sum += j * 64 + lane < r.experts ? s[j] : 0.0f;
                sum = wave_sum(sum);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    acc[j] += sum != 0.0f ? s[j] / sum : 0.0f;
            }
        }
    }
    if (a.parts == nullptr)
        return;
    float *sums = reinterpret_cast<float *>(scratch[0]);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j)
        sums[(wave * V + j) * 64 + lane] = acc[j];
    __syncthreads();
    for (int e = threadIdx.x; e < r.experts; e += kRouteThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kRouteWaves; ++w)
            v += sums[w * V * 64 + e];
        a.parts[int64_t(blockIdx.x) * r.experts + e] = v;
    }
}

// More experts than a wave holds: a block a token, keys of 64 bits in LDS, each thread every
// 256th of them.  4096 tokens of 1024 experts in 8 groups: 165 us for 17 MB, and 32 for the gradient; the time is the
// K choices one after the other, each with four barriers, and the groups' scan by a thread each.
template <class Op>
__device__ __forceinline__ double block_reduce(double v, double *red, Op op)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v = op(v, __shfl_xor(v, d));
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < kRouteWaves; ++w)
        v = op(v, red[w]);
    return v;
}

template <bool BF16>
__global__ __launch_bounds__(kRouteThreads) void route_wide_kernel(RouteArgs a)
{
    __shared__ double key[kMaxExperts], red[kRouteWaves], group[kMaxRouteGroups];
    __shared__ int found[kRouteWaves], chosen[kMaxTopk];
    const RouteRule &r = a.rule;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const double none = -INFINITY;
    const auto larger = [](double x, double y) { return x > y ? x : y; };
    const auto plus = [](double x, double y) { return x + y; };
    float *part = a.parts != nullptr ? a.parts + int64_t(blockIdx.x) * r.experts : nullptr;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = t * r.experts;
        double big = none, sum = 0.0;
        for (int e = tid; e < r.experts; e += kRouteThreads)
            big = larger(logit_at<BF16>(a.logits, row + e), big);
        big = block_reduce(big, red, larger);
        big = big == none ? 0.0 : big;
        auto raw = [&](double l) { return r.soft ? exp(l - big) : 1.0 / (1.0 + exp(-l)); };
        for (int e = tid; e < r.experts; e += kRouteThreads)
            sum += raw(logit_at<BF16>(a.logits, row + e));
        sum = block_reduce(sum, red, plus);
        const double whole = r.soft ? sum : 1.0;  // what a score is divided by
        auto score = [&](double l) { return whole == 0.0 ? 0.0 : raw(l) / whole; };
        for (int e = tid; e < r.experts; e += kRouteThreads) {
            const float l = logit_at<BF16>(a.logits, row + e);
            const bool live = l > -INFINITY && (r.rank_mask == nullptr || r.rank_mask[e / r.epr] == 0);
            const double k = r.bias != nullptr ? score(l) + double(r.bias[e]) : double(l);
            key[e] = live && k > none ? k : none;
            if (part != nullptr) {
                const float p = sum == 0.0 ? 0.0f : float(raw(l) / sum);
                part[e] = t == int64_t(blockIdx.x) ? p : part[e] + p;
            }
        }
        __syncthreads();
        if (r.groups > 1) {
            const int size = r.size;
            if (tid < r.groups) {
                double one = none, two = none;
                for (int i = 0; i < size; ++i) {
                    const double v = key[tid * size + i];
                    two = v > one ? one : v > two ? v : two;
                    one = v > one ? v : one;
                }
                group[tid] = r.bias == nullptr || two == none ? one : one + two;
            }
            __syncthreads();
            for (int g = wave; g < r.groups; g += kRouteWaves) {
                int ahead = 0;
                for (int o = 0; o < r.groups; ++o)
                    ahead += group[o] > group[g] || (group[o] == group[g] && o < g);
                if (ahead >= r.topk_groups)
                    for (int i = lane; i < size; i += 64)
                        key[g * size + i] = none;
            }
            __syncthreads();
        }
        for (int k = 0; k < r.topk; ++k) {
            double m = none;
            int at = kMaxExperts;
            for (int e = tid; e < r.experts; e += kRouteThreads)
                if (key[e] > m) {
                    m = key[e];
                    at = e;
                }
            const double best = block_reduce(m, red, larger);
            at = m == best ? at : kMaxExperts;
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) {
                const int o = __shfl_xor(at, d);
                at = o < at ? o : at;
            }
            if (lane == 0)
                found[wave] = at;
            __syncthreads();
            if (tid == 0) {
                int first = found[0];
                for (int w = 1; w < kRouteWaves; ++w)
                    first = found[w] < first ? found[w] : first;
                chosen[k] = best > none ? first : -1;
                if (best > none)
                    key[first] = none;
            }
            __syncthreads();
        }
        if (wave == 0) {
            const int e = lane < r.topk ? chosen[lane] : -1;
            const double v = e >= 0 ? double(logit_at<BF16>(a.logits, row + e)) : none;
            double one, of = 1.0;
            if (r.soft && r.normalize) {
                const double top = wave_max(v);
                one = e >= 0 ? exp(v - top) : 0.0;
                of = wave_sum(one);
            } else {
                one = e >= 0 ? score(v) : 0.0;
                if (r.normalize)
                    of = wave_sum(one) + double(kShareFloor);
            }
            if (lane < r.topk) {
                a.topk_idx[t * r.topk + lane] = e;
                a.weights[t * r.topk + lane] = e >= 0 ? float(one / of * double(r.scale)) : 0.0f;
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- backward
//
// With c_k = scale dw_k of the chosen and q = dsums (of p):
//   softmax:  ds = q + (not normalised: c at the chosen),  dl = s (ds - sum ds s)
//             normalised: dl_k += share_k (c_k - sum c share)
//   sigmoid:  ds = (q - sum q p) / sum s  +  c at the chosen
//             (normalised: (c_k - sum c share) / sum of the chosen),  dl = ds s (1 - s)
//
// Where one expert is nearly all of a mean, its own difference from it is nothing but roundings.  The differences sum to
// zero under the mean's weights, so that of an expert with more than half of them is taken from the others', which keep
// their digits.
constexpr float kLead = 0.5f;

struct RouteBackArgs {
    RouteRule rule;
    const void *logits;
    int64_t T;
    const int64_t *topk_idx;
    const float *dweights;  // [T][K]
    const float *dsums;     // nullable [E]
    void *dlogits;
};

template <bool BF16>
__device__ __forceinline__ void put_logit(void *out, int64_t i, float v)
{
    if constexpr (BF16)
        static_cast<uint16_t *>(out)[i] = uint16_t(bf16_rne(v));
    else
        static_cast<float *>(out)[i] = v;
}

// VREG > 0: the row in registers; 0: any row, read again for each pass.
template <int VREG, bool BF16>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(RouteBackArgs a)
{
    constexpr int R = VREG > 0 ? VREG : 1;
    const RouteRule &r = a.rule;
    const int lane = threadIdx.x & 63;
    const int64_t t = int64_t(blockIdx.x) * kRouteWaves + (threadIdx.x >> 6);
    if (t >= a.T)
        return;
    const int64_t row = t * r.experts;
    const int V = VREG > 0 ? VREG : (r.experts + 63) / 64;
    float held[R];
    if constexpr (VREG > 0) {
#pragma unroll
        for (int j = 0; j < R; ++j)
            held[j] = j * 64 + lane < r.experts ? logit_at<BF16>(a.logits, row + j * 64 + lane) : -INFINITY;
    }
    auto get = [&](int j) {
        if constexpr (VREG > 0)
            return held[j];
        else
            return j * 64 + lane < r.experts ? logit_at<BF16>(a.logits, row + j * 64 + lane) : -INFINITY;
    };
    auto each = [&](auto f) {
        if constexpr (VREG > 0) {
#pragma unroll
            for (int j = 0; j < R; ++j)
                f(j, held[j]);
        } else {
            for (int j = 0; j < V; ++j)
                f(j, get(j));
        }
    };
    // the chosen: slot k in lane k
    int e = -1;
    float c = 0.0f, v = -INFINITY;
    if (lane < r.topk) {
        const int64_t id = a.topk_idx[t * r.topk + lane];
        e = id >= 0 && id < r.experts ? int(id) : -1;
        if (e >= 0) {
            c = a.dweights[t * r.topk + lane] * r.scale;
            v = logit_at<BF16>(a.logits, row + e);
        }
    }
    const bool have = e >= 0;
    float mine = 0.0f;  // what slot `lane` adds to its logit's gradient (softmax, normalised), or to its score's
    if (r.normalize) {
        float one, of;
        if (r.soft) {
            const float big = wave_max(v);
            one = have ? expf(v - big) : 0.0f;
            of = wave_sum(one);
        } else {
            one = have ? 1.0f / (1.0f + expf(-v)) : 0.0f;
            of = wave_sum(one) + kShareFloor;
        }
        const float share = have ? one / of : 0.0f;
        const float mean = wave_sum(c * share);  // (every lane takes part)
        float off = have ? c - mean : 0.0f;
        if (wave_ballot(share > kLead) != 0) {  // sum share (c - mean) = mean (1 - sum share)
            const float rest = wave_sum(share > kLead ? 0.0f : share * off);
            off = share > kLead ? ((r.soft ? 0.0f : mean * (kShareFloor / of)) - rest) / share : off;
        }
        mine = !have ? 0.0f : r.soft ? share * off : off / of;
    } else
        mine = c;
    // row statistics
    float big = 0.0f, sum = 0.0f, per = 0.0f, inner = 0.0f, most = 0.0f, score[R] = {};
    const bool whole = a.dsums != nullptr || (r.soft && !r.normalize);  // every logit has a gradient
    auto raw = [&](float l) { return r.soft ? expf(l - big) : 1.0f / (1.0f + expf(-l)); };
    auto q_at = [&](int j) { return a.dsums != nullptr && j * 64 + lane < r.experts ? a.dsums[j * 64 + lane] : 0.0f; };
    if (whole) {
        if (r.soft) {
            big = -INFINITY;
            each([&](int, float l) { big = fmaxf(big, l); });
            big = wave_max(big);
            big = big == -INFINITY ? 0.0f : big;
        }
        each([&](int j, float l) {
            const float s = j * 64 + lane < r.experts ? raw(l) : 0.0f;
            if constexpr (VREG > 0)
                score[j] = s;
            sum += s;
            most = fmaxf(most, s);
            inner += q_at(j) * s;
        });
        sum = wave_sum(sum);
        per = sum != 0.0f ? 1.0f / sum : 0.0f;
        inner = sum != 0.0f ? wave_sum(inner) / sum : 0.0f;
        if (r.soft && !r.normalize) {
            const float s = have ? raw(v) * per : 0.0f;
            inner += wave_sum(c * s);
        }
    }
    // what the slots that chose an expert add
    float adds[R] = {};
    auto slots = [&](auto f) {
        for (int k = 0; k < r.topk; ++k)
            f(__builtin_amdgcn_readlane(e, k), lane_of(mine, k));
    };
    if constexpr (VREG > 0)
        slots([&](int o, float m) {
#pragma unroll
            for (int j = 0; j < R; ++j)
                adds[j] += o == j * 64 + lane ? m : 0.0f;
        });
    auto add_of = [&](int j) {
        float add = VREG > 0 ? adds[VREG > 0 ? j : 0] : 0.0f;
        if constexpr (VREG == 0)
            slots([&](int o, float m) { add += o == j * 64 + lane ? m : 0.0f; });
        return add;
    };
    // p, and ds - sum p ds, of an expert of the row
    auto p_of = [&](int j, float l) {
        return whole && j * 64 + lane < r.experts ? (VREG > 0 ? score[VREG > 0 ? j : 0] : raw(l)) * per : 0.0f;
    };
    float held_off[R] = {};
    auto off_of = [&](int j) {
        return VREG > 0 ? held_off[VREG > 0 ? j : 0] : q_at(j) + (r.soft && !r.normalize ? add_of(j) : 0.0f) - inner;
    };
    if constexpr (VREG > 0)
        if (whole)
#pragma unroll
            for (int j = 0; j < R; ++j)
                held_off[j] = q_at(j) + (r.soft && !r.normalize ? adds[j] : 0.0f) - inner;
    float rest = 0.0f;
    const bool led = wave_ballot(most * per > kLead) != 0;
    if (led) {
        each([&](int j, float l) {
            const float p = p_of(j, l);
            rest += p > kLead ? 0.0f : p * off_of(j);
        });
        rest = wave_sum(rest);
    }
    each([&](int j, float l) {
        const int at = j * 64 + lane;
        const float p = r.soft || led ? p_of(j, l) : 0.0f, off = led && p > kLead ? -rest / p : off_of(j);
        const float add = !r.soft || r.normalize ? add_of(j) : 0.0f;
        if (at >= r.experts)
            return;
        float d;
        if (r.soft) {
            d = (whole ? p * off : 0.0f) + add;
        } else {
            const float ds = add + (whole && sum != 0.0f ? off / sum : 0.0f);
            // s (1 - s), from exp(-|l|): 1 - s of a rounded s would be nothing from l = 17 on
            const float x = expf(-fabsf(l)), y = 1.0f + x;
            d = ds * (x / (y * y));
        }
        put_logit<BF16>(a.dlogits, row + at, d);
    });
}

}  // namespace

// Two waves' worth of tokens a SIMD at the most where the blocks' sums have to be joined.
int route_parts(int64_t T, int experts)
{
    const int64_t blocks = experts <= kWaveExperts ? (T + kRouteWaves - 1) / kRouteWaves : T;
    return int(blocks < 512 ? blocks : 512);
}

hipError_t launch_route(const RouteRule &rule, int64_t T, const void *logits, bool bf16, int64_t *topk_idx,
                        float *weights, float *score_sums, float *parts, hipStream_t stream)
{
    RouteArgs a{rule, logits, T, topk_idx, weights, score_sums != nullptr ? parts : nullptr};
    const int E = rule.experts, n = route_parts(T, E);
    const int64_t tokens = E <= kWaveExperts ? (T + kRouteWaves - 1) / kRouteWaves : T;
    const int64_t blocks = a.parts != nullptr ? n : tokens;
    if (log_enabled())
        log_launch("route: T=%lld E=%d K=%d groups=%d/%d blocks=%lld", (long long)T, E, rule.topk, rule.topk_groups,
                   rule.groups, (long long)blocks);
    if (T > 0) {
        auto go = [&](auto narrow, auto wide) {
            hipLaunchKernelGGL(bf16 ? wide : narrow, dim3(unsigned(blocks < kRowGrid ? blocks : kRowGrid)),
                               dim3(kRouteThreads), 0, stream, a);
        };
        if (E <= 64)
            go(route_kernel<1, false>, route_kernel<1, true>);
        else if (E <= 128)
            go(route_kernel<2, false>, route_kernel<2, true>);
        else if (E <= 256)
            go(route_kernel<4, false>, route_kernel<4, true>);
        else if (E <= kWaveExperts)
            go(route_kernel<8, false>, route_kernel<8, true>);
        else
            go(route_wide_kernel<false>, route_wide_kernel<true>);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return score_sums != nullptr ? launch_sum_parts(parts, n, E, score_sums, stream) : hipSuccess;
}

hipError_t launch_route_backward(const RouteRule &rule, int64_t T, const float *dweights, const void *logits, bool bf16,
                                 const int64_t *topk_idx, const float *dsums, void *dlogits, hipStream_t stream)
{
    if (T == 0)
        return hipSuccess;
    const RouteBackArgs a{rule, logits, T, topk_idx, dweights, dsums, dlogits};
    const int E = rule.experts;
    const int64_t blocks = (T + kRouteWaves - 1) / kRouteWaves;
    if (log_enabled())
        log_launch("route_backward: T=%lld E=%d K=%d", (long long)T, E, rule.topk);
    auto go = [&](auto narrow, auto wide) {
        hipLaunchKernelGGL(bf16 ? wide : narrow, dim3(unsigned(blocks)), dim3(kRouteThreads), 0, stream, a);
    };
    if (E <= 64)
        go(route_backward_kernel<1, false>, route_backward_kernel<1, true>);
    else if (E <= 128)
        go(route_backward_kernel<2, false>, route_backward_kernel<2, true>);
    else if (E <= 256)
        go(route_backward_kernel<4, false>, route_backward_kernel<4, true>);
    else if (E <= kWaveExperts)
        go(route_backward_kernel<8, false>, route_backward_kernel<8, true>);
    else
        go(route_backward_kernel<0, false>, route_backward_kernel<0, true>);
    return hipGetLastError();
}

}  // namespace ep
