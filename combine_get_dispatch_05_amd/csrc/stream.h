// stream.h -- products of 16-row tiles of a weight with 16-row tiles of bf16 token rows, both
// straight from memory into the matrix instruction's registers.  Device code; included by
// moe.hip and adapter.hip.
#pragma once

#include "gemm.h"

namespace ep {

// One K step (128 bytes a weight row) of 16 weight rows: lane l holds row l % 16, chunks l / 16 and
// 4 + l / 16 of eight.
struct WeightStep {
    i32x4 c[2];
};
// The same K values of 16 token rows: bf16 beside bf16 weights the same two chunks, beside FP8 ones the four that
// hold the 32 values of the weight's two.
template <bool FP8>
struct TokenStep {
    i32x4 c[FP8 ? 4 : 2];
};

__device__ __forceinline__ i32x4 load16(const char *p) { return *reinterpret_cast<const i32x4 *>(p); }

// TAIL: chunks at or past `end` (bytes of a weight row) are zeros.
template <bool TAIL>
__device__ __forceinline__ void load_step(WeightStep &f, const char *row, int at, int g, int end)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int b = at + h * 64 + g * 16;
        f.c[h] = load16(TAIL && b >= end ? reinterpret_cast<const char *>(kZero16) : row + b);
    }
}
template <bool TAIL, bool FP8>
__device__ __forceinline__ void load_step(TokenStep<FP8> &f, const char *row, int at, int g, int end)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int b = at + h * 64 + g * 16;
        if constexpr (FP8) {
            f.c[2 * h] = load16(row + 2 * b);
            f.c[2 * h + 1] = load16(row + 2 * b + 16);
        } else
            f.c[h] = load16(TAIL && b >= end ? reinterpret_cast<const char *>(kZero16) : row + b);
    }
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

// acc[r][m] += weight rows of tile r times token tile m over steps [s0, s1).
template <bool FP8, bool TAIL, int AHEAD, int RT, int MT>
__device__ __forceinline__ void stream(const char *const (&prow)[RT], const float *const (&scale)[RT],
                                       const char *const (&qrow)[MT], int s0, int s1, int kbytes, int lane,
                                       f32x4 (&acc)[RT][MT])
{
    const int g = lane >> 4;
    if (s0 >= s1)
        return;
    WeightStep p[AHEAD][RT];
    TokenStep<FP8> q[AHEAD][MT];
    float c[AHEAD][RT];
    auto load = [&](int d, int s) {
        s = s < s1 ? s : s1 - 1;  // (past the end: loaded again, not used)
        const int at = s * kStepBytes;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            load_step<TAIL>(p[d][r], prow[r], at, g, kbytes);
            if constexpr (FP8)
                c[d][r] = scale[r][s];
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
            load_step<TAIL, FP8>(q[d][m], qrow[m], at, g, kbytes);
    };
    auto compute = [&](int d, int s) {
        if (s >= s1)
            return;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            if constexpr (FP8) {
                f32x4 part[MT] = {};
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bf16x8 w = widen8(p[d][r].c[h][2 * i], p[d][r].c[h][2 * i + 1]);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            part[m] = mfma_bf16(w, __builtin_bit_cast(bf16x8, q[d][m].c[2 * h + i]), part[m]);
                    }
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    acc[r][m] += part[m] * c[d][r];
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[r][m] = mfma_bf16(__builtin_bit_cast(bf16x8, p[d][r].c[h]),
                                              __builtin_bit_cast(bf16x8, q[d][m].c[h]), acc[r][m]);
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

}  // namespace ep
