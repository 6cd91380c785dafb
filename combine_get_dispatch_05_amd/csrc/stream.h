// stream.h -- products of a weight's rows with bf16 token rows, both straight from memory into the
// matrix instruction's registers.  Device code; included by moe.hip and adapter.hip.
//
// The instruction takes 16 operand rows of four 16-byte chunks, lane l the chunk l / 16 of row l % 16, so with
// one weight row an operand row the lanes of a load are 16 rows apart and the load takes as many
// cycles as lanes.  With C = 2 an operand row is half of a weight row's 128 bytes: lane l holds chunk
// 2 (l / 16) + l % 2 of row l % 16 / 2, on both sides, pairs of lanes read 32 neighbouring bytes, and the result
// has what belongs together where the halves are the same (fold()).  It takes 8 rows by 8 tokens then.
#pragma once

#include "gemm.h"

namespace ep {

// What rounding v to the bf16 values b lost (nothing where those are not finite).
__device__ __forceinline__ f32x4 lost(const f32x4 &v, const uint2 &b)
{
    const f32x4 kept = {bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y)};
    f32x4 rest;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        rest[k] = fabsf(kept[k]) < INFINITY ? v[k] - kept[k] : 0.0f;
    return rest;
}

__device__ __forceinline__ i32x4 load16(const char *p) { return *reinterpret_cast<const i32x4 *>(p); }

// One K step, 128 bytes a weight row, of a tile of 16 / C weight rows.
template <int C>
struct WeightStep {
    i32x4 c[2 / C];
};
// The same K values of 16 / C token rows: bf16 beside bf16 weights the same chunks, beside FP8 ones two for each.
template <bool FP8, int C>
struct TokenStep {
    i32x4 c[(FP8 ? 4 : 2) / C];
};

// Byte of this lane's h-th chunk inside a step.
template <int C>
__device__ __forceinline__ int chunk_at(int h, int lane)
{
    return (h * 4 + (lane >> 4) * C + lane % C) * 16;
}

// TAIL: chunks at or past `end` (bytes of a weight row) are zeros.
template <bool TAIL, int C>
__device__ __forceinline__ void load_step(WeightStep<C> &f, const char *row, int at, int lane, int end)
{
#pragma unroll
    for (int h = 0; h < 2 / C; ++h) {
        const int b = at + chunk_at<C>(h, lane);
        f.c[h] = load16(TAIL && b >= end ? reinterpret_cast<const char *>(kZero16) : row + b);
    }
}
template <bool TAIL, bool FP8, int C>
__device__ __forceinline__ void load_step(TokenStep<FP8, C> &f, const char *row, int at, int lane, int end)
{
#pragma unroll
    for (int h = 0; h < 2 / C; ++h) {
        const int b = at + chunk_at<C>(h, lane);
        if constexpr (FP8) {
            f.c[2 * h] = load16(row + 2 * b);
            f.c[2 * h + 1] = load16(row + 2 * b + 16);
        } else
            f.c[h] = load16(TAIL && b >= end ? reinterpret_cast<const char *>(kZero16) : row + b);
    }
}

// C = 2: of an 8 x 8 tile, the sum of the halves: row 2 (l / 16) + l % 2, token l % 16 / 2.
__device__ __forceinline__ float fold(const f32x4 &v, int lane)
{
    const bool odd = lane & 1;
    return (odd ? v[3] : v[0]) + __shfl_xor(odd ? v[1] : v[2], 1);
}

// Eight FP8 values as bf16.
__device__ __forceinline__ bf16x8 widen8(int lo, int hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    bf16x8 v;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = h ? hi : lo;
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true);
        v[4 * h] = a[0], v[4 * h + 1] = a[1], v[4 * h + 2] = b[0], v[4 * h + 3] = b[1];
    }
    return v;
}

// acc[r][m] += weight rows of tile r times token tile m over steps [s0, s1).  PLANES: the token rows are a sum of that many
// bf16 rows, `plane` bytes apart.
template <bool FP8, bool TAIL, int AHEAD, int C, int PLANES, int RT, int MT>
__device__ __forceinline__ void stream_run(const char *const (&prow)[RT], const float *const (&scale)[RT],
                                           const char *const (&qrow)[MT], int64_t plane, int s0, int s1, int kbytes, int lane,
                                           f32x4 (&acc)[RT][MT])
{
    if (s0 >= s1)
        return;
    WeightStep<C> p[AHEAD][RT];
    TokenStep<FP8, C> q[AHEAD][MT][PLANES];
    float scales[AHEAD][RT];
    auto load = [&](int d, int s) {
        s = s < s1 ? s : s1 - 1;  // (past the end: loaded again, not used)
        const int at = s * kStepBytes;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            load_step<TAIL>(p[d][r], prow[r], at, lane, kbytes);
            if constexpr (FP8)
                scales[d][r] = scale[r][s];
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int u = 0; u < PLANES; ++u)
                load_step<TAIL>(q[d][m][u], qrow[m] + u * plane, at, lane, kbytes);
    };
    auto compute = [&](int d, int s) {
        if (s >= s1)
            return;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            if constexpr (FP8) {
                f32x4 part[MT] = {};
#pragma unroll
                for (int h = 0; h < 2 / C; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bf16x8 w = widen8(p[d][r].c[h][2 * i], p[d][r].c[h][2 * i + 1]);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int u = 0; u < PLANES; ++u)
                                part[m] = mfma_bf16(w, __builtin_bit_cast(bf16x8, q[d][m][u].c[2 * h + i]), part[m]);
                    }
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    acc[r][m] += part[m] * scales[d][r];
            } else {
#pragma unroll
                for (int h = 0; h < 2 / C; ++h)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int u = 0; u < PLANES; ++u)
                            acc[r][m] = mfma_bf16(__builtin_bit_cast(bf16x8, p[d][r].c[h]),
                                                  __builtin_bit_cast(bf16x8, q[d][m][u].c[h]), acc[r][m]);
            }
        }
    };
#pragma unroll
    for (int d = 0; d < AHEAD; ++d)
        load(d, s0 + d);
    int s = s0;
    for (; s + AHEAD < s1; s += AHEAD) {
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
            compute(d, s + d);
            load(d, s + d + AHEAD);
        }
    }
#pragma unroll
    for (int d = 0; d < AHEAD; ++d)
        compute(d, s + d);
}

// A run is rounded up to the steps in flight, so a short one has fewer.
template <bool FP8, bool TAIL, int AHEAD, int C, int PLANES = 1, int RT, int MT>
__device__ __forceinline__ void stream(const char *const (&prow)[RT], const float *const (&scale)[RT],
                                       const char *const (&qrow)[MT], int s0, int s1, int kbytes, int lane, f32x4 (&acc)[RT][MT],
                                       int64_t plane = 0)
{
    if (AHEAD > 2 && s1 - s0 <= 2)
        stream_run<FP8, TAIL, 2, C, PLANES>(prow, scale, qrow, plane, s0, s1, kbytes, lane, acc);
    else
        stream_run<FP8, TAIL, AHEAD, C, PLANES>(prow, scale, qrow, plane, s0, s1, kbytes, lane, acc);
}

}  // namespace ep
