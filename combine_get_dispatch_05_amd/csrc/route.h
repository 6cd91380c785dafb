// route.h -- choosing the experts of one token in one wave: shared by the router
// (route.hip) and the layer for a few tokens (moe.hip).  Device code.
//
// Lane l holds experts l, 64 + l, ...; the chosen ones end in lanes 0 to K - 1.
// What is chosen never depends on a rounding: the 32-bit keys decide only where the gaps between
// them are larger than what they can be off by (the bits that hold the index, and with a
// bias the rounding of the scores); a token with a smaller gap (4 of 1000 of normal logits) is chosen
// again with keys of 64 bits.
#pragma once

#include "gemm.h"

namespace ep {

constexpr int kMaxRouteGroups = 64;
constexpr int kWaveExperts = 512;  // the most that one wave holds
constexpr float kShareFloor = 1e-20f;  // beside the sum that sigmoid scores are divided by

struct RouteRule {
    int experts, topk, groups, topk_groups, epr;
    int size, lanes;   // experts of a group; lanes that look at one: a power of two
    float per_size;    // 1 / size
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
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    auto step = [&](uint32_t o) { v = o > v ? o : v; };
    step(uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x111, 0xF, 0xF, true)));
    step(uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x112, 0xF, 0xF, true)));
    step(uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x114, 0xF, 0xF, true)));
    step(uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x118, 0xF, 0xF, true)));
    step(uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x142, 0xA, 0xF, false)));
    step(uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x143, 0xC, 0xF, false)));
    return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}
__device__ __forceinline__ float lane_of(float v, int lane)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double lane_of(double v, int lane)
{
    const uint64_t u = uint64_t(__double_as_longlong(v));
    const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(u)), lane));
    const uint32_t hi = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(u >> 32)), lane));
    return __longlong_as_double(static_cast<long long>(uint64_t(hi) << 32 | lo));
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

// Floats as integers in the same order.
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);  // (-0 equals 0)
    return int32_t(u) < 0 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u)
{
    return __uint_as_float(int32_t(u) < 0 ? u & 0x7fffffffu : ~u);
}

// e / size for e < 8192 and any size: half a step away from every border.
__device__ __forceinline__ int group_of(int e, float per_size) { return int((float(e) + 0.5f) * per_size); }

// Scores of a row.  A row with nothing but -inf has no softmax.  FOR_KEYS: of a NaN, which has no key, any number.
template <bool FOR_KEYS, int V, class T>
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
        // (a quotient of two roundings: one division a lane; without a score or with a NaN it is 0 or NaN times 0)
        const T per = sum > T(0) ? T(1) / sum : sum;
#pragma unroll
        for (int j = 0; j < V; ++j)
            s[j] *= per;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (FOR_KEYS && sizeof(T) == 4)
                s[j] = sigmoidf(l[j]);
            else
                s[j] = T(1) / (T(1) + exp(-T(l[j])));
        }
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
    const int size = r.size, lanes = r.lanes;
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
        const T other = lane_of(score, g * lanes);
        ahead += other > score || (other == score && g < group);
    }
    const bool keep = group < r.groups && ahead < r.topk_groups;
    const uint64_t kept = wave_ballot(keep && part == 0);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = j * 64 + lane;
        if (e < r.experts && !(kept >> (group_of(e, r.per_size) * lanes) & 1))
            key[j] = none;
    }
    if (!(slack > T(0)))
        return false;
    // (of the fp32 keys alone; the largest of the negated is the lowest)
    const float low = -unordered(wave_max(keep ? ordered(-float(score)) : 0u));
    const float high = unordered(wave_max(keep || group >= r.groups ? 0u : ordered(float(score))));
    // a sum is off by what its two keys are, which goes with their size: with biases that cancel the sum is small, its
    // error is not
    const float most = wave_max(fmaxf(one > none ? fabsf(float(one)) : 0.0f, two > none ? fabsf(float(two)) : 0.0f));
    // (two keys near the lowest number, as of barred experts, are not the -inf of a group without any)
    const bool past = one > none && !(score > none);
    return wave_ballot(past) != 0 || (high > -INFINITY && !(low - high > float(slack) * (1.0f + most)));
}

// The K largest keys, largest first, ties to the lowest index: lane k returns the k-th, -1 where
// nothing is left.  As integers in the same order, whose halves are compared one after the other.
template <int V>
__device__ __forceinline__ int pick(const double (&key)[V], int K, int lane)
{
    uint64_t u[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint64_t b = uint64_t(__double_as_longlong(key[j] + 0.0));  // (-0 equals 0)
        u[j] = !(key[j] > -INFINITY) ? 0 : int64_t(b) < 0 ? ~b : b | 1ull << 63;
    }
    int mine = -1;
    for (int k = 0; k < K; ++k) {
        uint64_t m = u[0];
        int tag = lane;
#pragma unroll
        for (int j = 1; j < V; ++j) {
            tag = u[j] > m ? j * 64 + lane : tag;
            m = u[j] > m ? u[j] : m;
        }
        const uint32_t high = wave_max(uint32_t(m >> 32));
        if (high == 0)
            break;
        const uint32_t low = wave_max(uint32_t(m >> 32) == high ? uint32_t(m) : 0u);
        const int at = int(~wave_max(m == (uint64_t(high) << 32 | low) ? ~uint32_t(tag) : 0u));
#pragma unroll
        for (int j = 0; j < V; ++j)
            u[j] = at == j * 64 + lane ? 0 : u[j];
        mine = lane == k ? at : mine;
    }
    return mine;
}

// The same from 32-bit keys, as integers that end in the index (its complement, so that ties go to the
// lowest): a round is one maximum over the wave.  Each lane keeps its keys sorted and shows the largest.
// The rest of the bits holds the key in steps of its range (so 2^-23 or less of it), or where 16 bits are
// all of it (whole) the key itself.  unsure: a gap on the way, that to the K + 1st included, was
// within slack, or keys fell on the same step.
template <int V>
__device__ __forceinline__ int pick(const float (&key)[V], int K, int lane, float slack, bool whole, bool &unsure)
{
    constexpr int kBits = V == 1 ? 6 : V == 2 ? 7 : V == 4 ? 8 : 9;
    constexpr uint32_t kIndex = (1u << kBits) - 1, kSteps = 1u << (kBits < 8 ? 24 : 32 - kBits);
    static_assert(64 * V == 1 << kBits, "an index a bit pattern");
    uint32_t u[V];
    float scale = 0.0f, most = 0.0f;
    if (whole) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            u[j] = ordered(key[j]) & ~kIndex;
    } else {
        uint32_t top = 0, down = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool is = key[j] > -INFINITY;
            const uint32_t a = is ? ordered(key[j]) : 0u, b = is ? ordered(-key[j]) : 0u;
            top = a > top ? a : top;
            down = b > down ? b : down;
        }
        const float high = unordered(wave_max(top)), low = -unordered(wave_max(down));
        scale = high > low ? float(kSteps - 2) / (high - low) : 0.0f;
        unsure |= !(high - low < INFINITY);
        most = fmaxf(fabsf(high), fabsf(low));
#pragma unroll
        for (int j = 0; j < V; ++j)
            u[j] = (uint32_t(fminf((key[j] - low) * scale, float(kSteps - 2))) + 1u) << kBits;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
        u[j] = key[j] > -INFINITY ? u[j] | (kIndex - uint32_t(j * 64 + lane)) : 0u;
#pragma unroll
    for (int i = 1; i < V; ++i)
#pragma unroll
        for (int j = i; j > 0; --j) {
            const uint32_t a = u[j - 1], b = u[j];
            u[j - 1] = a > b ? a : b;
            u[j] = a > b ? b : a;
        }
    const bool exact = whole && !(slack > 0.0f);
    const int rounds = exact ? K : K + 1;
    uint32_t got = 0, next = 0;  // of lane k: the k-th, and the K + 1st
    for (int k = 0; k < rounds; ++k) {
        next = wave_max(u[0]);
        got = lane == k ? next : got;
        const uint32_t taken = u[0] == next ? ~0u : 0u;
#pragma unroll
        for (int j = 0; j + 1 < V; ++j)
            u[j] = (u[j + 1] & taken) | (u[j] & ~taken);
        u[V - 1] &= ~taken;
    }
    if (!exact) {
        // (with 64 slots the K + 1st has no lane; where fewer are left it is the last one of them)
        const uint32_t behind = uint32_t(__shfl_down(int(got), 1));  // (every lane takes part)
        const uint32_t after = lane < 63 ? behind : K == 64 ? next : 0u;
        const float gap = float((got >> kBits) - (after >> kBits));
        const float least = slack > 0.0f ? slack * (1.0f + most) * scale + 2.0f : 0.0f;
        unsure |= wave_ballot(lane < K && after != 0 && after != got && !(gap > least)) != 0;
    }
    return lane < K && got != 0 ? int(kIndex - (got & kIndex)) : -1;
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
    double s[V] = {}, key[V];
    if (r.bias != nullptr)
        scores_of<true>(r.soft, l, s);
    keys_of(r, l, s, bias, live, key);
    if (r.groups > 1)
        keep_groups(r, key, lane, scratch, 0.0);
    return pick(key, r.topk, lane);
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
// l: the logits, -inf past E (whole: bf16 values without a bias); s: the scores, made where want_scores or the rule needs them.
// at(e): the logit of expert e.
template <int V, class At>
__device__ __forceinline__ int route_row(const RouteRule &r, const float (&l)[V], const float (&bias)[V], uint32_t live,
                                         int lane, double *scratch, bool want_scores, bool whole, float (&s)[V],
                                         At at, float &weight)
{
    if (want_scores || (r.soft && !r.normalize))
        scores_of<false>(r.soft, l, s);
    else if (r.bias != nullptr)
        scores_of<true>(r.soft, l, s);
    // a score is off by at most some 15 roundings of its sum (of its quotient), a key by one more
    const float slack = r.bias != nullptr ? 4e-6f : 0.0f;
    float key[V];
    keys_of(r, l, s, bias, live, key);
    bool unsure = false;
    if (r.groups > 1)
        unsure = keep_groups(r, key, lane, reinterpret_cast<float *>(scratch), 2 * slack);
    int e = pick(key, r.topk, lane, slack, whole && r.bias == nullptr, unsure);
    if (unsure)
        e = choose_exactly(r, l, bias, live, lane, scratch);
    const bool have = e >= 0;
    const float of = at(have ? e : 0);  // (every lane takes part)
    const float v = have ? of : -INFINITY;
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
