// route.h -- choosing the experts of one token in one wave: shared by the router
// (route.hip) and the layer for a few tokens (moe.hip).  Device code.
//
// Lane l holds experts l, 64 + l, ...; the chosen ones end in lanes 0 to K - 1.
// What is chosen never depends on a rounding: without a bias the logits themselves
// are compared, and with one the 32-bit keys decide only where the gaps between them
// are larger than what they can be off by; a token with a smaller gap (less than one in
// a hundred) is chosen again with keys of 64 bits.
#pragma once

#include "ep_internal.h"

namespace ep {

constexpr int kMaxRouteGroups = 64;
constexpr int kWaveExperts = 512;  // the most that one wave holds
constexpr float kShareFloor = 1e-20f;  // beside the sum that sigmoid scores are divided by

struct RouteRule {
    int experts, topk, groups, topk_groups, epr;
    int soft;       // softmax scores, else sigmoid
    int normalize;
    float scale;
    const float *bias;         // nullable [E]
    const int32_t *rank_mask;  // nullable [R]
};

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or(float old, float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float last_lane(float v)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// Over the wave, the same in every lane and in every run.
__device__ __forceinline__ float wave_max(float v)
{
    v = fmaxf(v, dpp_or<0x111, 0xF>(v, v));
    v = fmaxf(v, dpp_or<0x112, 0xF>(v, v));
    v = fmaxf(v, dpp_or<0x114, 0xF>(v, v));
    v = fmaxf(v, dpp_or<0x118, 0xF>(v, v));
    v = fmaxf(v, dpp_or<0x142, 0xA>(v, v));
    v = fmaxf(v, dpp_or<0x143, 0xC>(v, v));
    return last_lane(v);
}
__device__ __forceinline__ float wave_sum(float v)
{
    v += dpp_or<0x111, 0xF>(0.0f, v);
    v += dpp_or<0x112, 0xF>(0.0f, v);
    v += dpp_or<0x114, 0xF>(0.0f, v);
    v += dpp_or<0x118, 0xF>(0.0f, v);
    v += dpp_or<0x142, 0xA>(0.0f, v);
    v += dpp_or<0x143, 0xC>(0.0f, v);
    return last_lane(v);
}
__device__ __forceinline__ double wave_max(double v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v = fmax(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// e / size for e < 8192 and any size: half a step away from every border.
__device__ __forceinline__ int group_of(int e, float per_size) { return int((float(e) + 0.5f) * per_size); }

// Scores of a row, and keys of what may be chosen.  A row with nothing but -inf has no scores.
template <int V, class T>
__device__ __forceinline__ void scores_of(bool soft, const float (&l)[V], T (&s)[V])
{
    if (soft) {
        float big = l[0];
#pragma unroll
        for (int j = 1; j < V; ++j)
            big = fmaxf(big, l[j]);
        big = wave_max(big);
        if (big == -INFINITY)
            big = 0.0f;
        T sum = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s[j] = exp(T(l[j]) - T(big));
            sum += s[j];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int j = 0; j < V; ++j)
            s[j] = sum > T(0) ? s[j] / sum : sum != sum ? sum : T(0);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            s[j] = T(1) / (T(1) + exp(-T(l[j])));
    }
}

// Takes the keys of all groups but the best out.  Returns whether the border between the kept groups
// and the others is nearer than slack.  scratch: V * 64 values of this wave.
template <int V, class T>
__device__ __forceinline__ bool keep_groups(const RouteRule &r, T (&key)[V], int lane, T *scratch, T slack)
{
    const T none = T(-INFINITY);
#pragma unroll
    for (int j = 0; j < V; ++j)
        scratch[j * 64 + lane] = key[j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    const int size = r.experts / r.groups;
    int lanes = 64;  // of a group: a power of two
    while (lanes * r.groups > 64)
        lanes >>= 1;
    const int group = lane / lanes, part = lane & (lanes - 1);
    T one = none, two = none;
    if (group < r.groups)
        for (int i = part; i < size; i += lanes) {
            const T v = scratch[group * size + i];
            two = v > one ? one : v > two ? v : two;
            one = v > one ? v : one;
        }
    for (int d = 1; d < lanes; d <<= 1) {
        const T o1 = __shfl_xor(one, d), o2 = __shfl_xor(two, d);
        const T low = o1 > one ? one : o1;
        two = o2 > two ? o2 : two;
        two = low > two ? low : two;
        one = o1 > one ? o1 : one;
    }
    const T score = r.bias == nullptr || two == none ? one : one + two;
    int ahead = 0;
    for (int g = 0; g < r.groups; ++g) {
        const T other = __shfl(score, g * lanes);
        ahead += other > score || (other == score && g < group);
    }
    const bool keep = group < r.groups && ahead < r.topk_groups;
    const uint64_t kept = wave_ballot(keep && part == 0);
    const float per_size = 1.0f / float(size);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = j * 64 + lane;
        if (e < r.experts && !(kept >> (group_of(e, per_size) * lanes) & 1))
            key[j] = none;
    }
    if (!(slack > T(0)))
        return false;
    const T low = -wave_max(keep ? -score : none), high = wave_max(keep || group >= r.groups ? none : score);
    return high > none && !(low - high > slack * (T(1) + (low < 0 ? -low : low)));
}

// The K largest keys, largest first, ties to the lowest index: lane k returns the k-th, -1 where
// nothing is left.  unsure: some gap on the way was within slack.
template <int V, class T>
__device__ __forceinline__ int pick(T (&key)[V], int K, int lane, T slack, bool &unsure)
{
    int mine = -1;
    T last = T(INFINITY);
    for (int k = 0;; ++k) {
        if (k == K && !(slack > T(0)))
            break;
        T m = key[0];
#pragma unroll
        for (int j = 1; j < V; ++j)
            m = key[j] > m ? key[j] : m;
        m = wave_max(m);
        if (!(m > T(-INFINITY)))
            break;
        unsure |= slack > T(0) && !(last - m > slack * (T(1) + (m < 0 ? -m : m)));
        if (k == K)
            break;
        last = m;
        int at = 0;
#pragma unroll
        for (int j = V - 1; j >= 0; --j) {
            const uint64_t b = wave_ballot(key[j] == m);
            at = b != 0 ? j * 64 + __builtin_ctzll(b) : at;
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            key[j] = at == j * 64 + lane ? T(-INFINITY) : key[j];
        mine = lane == k ? at : mine;
    }
    return mine;
}

// The keys of expert scores s (of the logits l without a bias), -inf for what may not be chosen: bit j of
// `live` is this lane's j-th expert.
template <int V, class T>
__device__ __forceinline__ void keys_of(const RouteRule &r, const float (&l)[V], const T (&s)[V], const float (&bias)[V],
                                        uint32_t live, T (&key)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j) {
        T k = r.bias != nullptr ? s[j] + T(bias[j]) : T(l[j]);
        // (a NaN fails the comparison)
        key[j] = (live >> j & 1) && l[j] > -INFINITY && k > T(-INFINITY) ? k : T(-INFINITY);
    }
}

// With 64-bit keys.
template <int V>
__device__ __forceinline__ int choose_exactly(const RouteRule &r, const float (&l)[V], const float (&bias)[V],
                                                        uint32_t live, int lane, double *scratch)
{
    double s[V], key[V];
    scores_of(r.soft, l, s);
    keys_of(r, l, s, bias, live, key);
    if (r.groups > 1)
        keep_groups(r, key, lane, scratch, 0.0);
    bool unsure;
    return pick(key, r.topk, lane, 0.0, unsure);
}

// Which of this lane's experts may be chosen at all.
template <int V>
__device__ __forceinline__ uint32_t live_experts(const RouteRule &r, int lane)
{
    uint32_t live = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = j * 64 + lane;
        if (e < r.experts && (r.rank_mask == nullptr || r.rank_mask[e / r.epr] == 0))
            live |= 1u << j;
    }
    return live;
}

// One token: the expert of slot k in lane k (-1 where there are too few, and past K) and its weight.
// l: the logits, -inf past E; s: the scores, made where want_scores or the rule needs them.
// at(e): the logit of expert e.
template <int V, class At>
__device__ __forceinline__ int route_row(const RouteRule &r, const float (&l)[V], const float (&bias)[V], uint32_t live,
                                         int lane, double *scratch, bool want_scores, float (&s)[V], At at, float &weight)
{
    if (want_scores || r.bias != nullptr || (r.soft && !r.normalize))
        scores_of(r.soft, l, s);
    // a score is off by at most some 15 roundings of its sum (of its quotient), a key by one more
    const float slack = r.bias != nullptr ? 4e-6f : 0.0f;
    float key[V];
    keys_of(r, l, s, bias, live, key);
    bool unsure = false;
    if (r.groups > 1)
        unsure = keep_groups(r, key, lane, reinterpret_cast<float *>(scratch), 2 * slack);
    int e = pick(key, r.topk, lane, slack, unsure);
    if (unsure)
        e = choose_exactly(r, l, bias, live, lane, scratch);
    const bool have = e >= 0;
    const float v = have ? at(e) : -INFINITY;
    float one, sum;
    if (r.soft && r.normalize) {  // the softmax of the chosen alone
        const float big = wave_max(v);
        one = have ? expf(v - big) : 0.0f;
        sum = wave_sum(one);
    } else if (r.soft) {  // the score, from the lane that has it
        one = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float o = __shfl(s[j], e & 63);
            one = have && e >> 6 == j ? o : one;
        }
        sum = 1.0f;
    } else {
        one = have ? 1.0f / (1.0f + expf(-v)) : 0.0f;
        sum = r.normalize ? wave_sum(one) + kShareFloor : 1.0f;
    }
    weight = have ? one / sum * r.scale : 0.0f;
    return e;
}

}  // namespace ep
