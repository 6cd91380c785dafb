// norm.hip -- root-mean-square norm of token rows with the residual's addition,
// an output in bf16 and/or in 8 bits with scales, and its gradients.
//   s = x + residual, rstd = 1 / sqrt(mean(s^2) + eps), y = s rstd w
//   a = dout w, xh = h rstd, dx = rstd (a - xh mean(a xh)) + dresidual, dw = sum_t dout xh
// One block a row, the row held in registers between its sum and its outputs,
// so every byte crosses HBM once; rows too long for that are read twice.  HBM bounds
// it: 8192 rows of 7168 with residual and all outputs are 530 MB, 74 us and 7.1 TB/s
// by themselves, 97 us (5.4, the rate of a copy) one launch behind the other.
#include "ep_internal.h"

namespace ep {

namespace {

__device__ __forceinline__ void unpack8(const u32x4 &v, float (&f)[8])
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        f[2 * q] = bf16_lo(v[q]);
        f[2 * q + 1] = bf16_hi(v[q]);
    }
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8])
{
    u32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        v[q] = cvt_bf16x2(f[2 * q], f[2 * q + 1]);
    return v;
}

// Sum over the block; every thread gets it.  s: NTH / 64 floats.
template <int NTH>
__device__ __forceinline__ float block_sum(float v, float *s)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d);
    if constexpr (NTH == kWave)
        return v;
    if ((threadIdx.x & 63) == 0)
        s[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < NTH / kWave; ++w)
        t += s[w];
    return t;
}

struct NormArgs {
    const u32x4 *x, *residual, *weight;  // residual nullable
    u32x4 *residual_out, *out;           // nullable
    uint2 *out_q;                        // nullable
    float *out_scale, *rstd;             // rstd nullable
    int64_t T;
    int V;  // 16-byte vectors of a row
    float eps, inv_h;
};

// The outputs of one vector of a row.  A 128-element block is 16 lanes.
__device__ __forceinline__ void norm_store(const NormArgs &a, int64_t row, int v, const float (&s)[8],
                                           const u32x4 &w, float rstd)
{
    float wf[8], y[8];
    unpack8(w, wf);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = s[i] * rstd * wf[i];
    const int64_t at = row * a.V + v;
    if (a.out != nullptr)
        __builtin_nontemporal_store(pack8(y), &a.out[at]);
    if (a.out_q == nullptr)
        return;
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        amax = fmaxf(amax, fabsf(y[i]));
#pragma unroll
    for (int d = 1; d < 16; d <<= 1)
        amax = fmaxf(amax, __shfl_xor(amax, d, 16));
    amax = amax < 1e-4f ? 1e-4f : amax;
    const float inv = 448.0f / amax;
    uint2 q;
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * inv, y[1] * inv, 0, false);
    q.x = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * inv, y[3] * inv, c, true);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(y[4] * inv, y[5] * inv, 0, false);
    q.y = __builtin_amdgcn_cvt_pk_fp8_f32(y[6] * inv, y[7] * inv, c, true);
    typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
    __builtin_nontemporal_store(u32x2{q.x, q.y}, reinterpret_cast<u32x2 *>(&a.out_q[at]));
    if ((v & 15) == 0)
        a.out_scale[at >> 4] = amax / 448.0f;
}

// VPT vectors a thread, kept in registers; VPT = 0: any row, read twice.
template <int NTH, int VPT>
__global__ __launch_bounds__(NTH) void rms_norm_kernel(NormArgs a)
{
    constexpr int R = VPT > 0 ? VPT : 1;
    __shared__ float red[NTH / kWave];
    const int64_t row = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    if (row >= a.T)
        return;
    const int64_t base = row * a.V;
    float s[R][8], sum = 0.0f;
    u32x4 w[R];
    auto load = [&](int v, float (&f)[8]) {
        unpack8(a.x[base + v], f);
        if (a.residual != nullptr) {
            float r[8];
            unpack8(a.residual[base + v], r);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                f[k] += r[k];
        }
    };
    if constexpr (VPT > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int v = threadIdx.x + i * NTH;
            if (v < a.V) {
                w[i] = a.weight[v];
                load(v, s[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int v = threadIdx.x + i * NTH;
            if (v < a.V) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    sum += s[i][k] * s[i][k];
                if (a.residual_out != nullptr)
                    __builtin_nontemporal_store(pack8(s[i]), &a.residual_out[base + v]);
            }
        }
    } else {
        for (int v = threadIdx.x; v < a.V; v += NTH) {
            load(v, s[0]);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sum += s[0][k] * s[0][k];
        }
    }
    const float rstd = 1.0f / sqrtf(block_sum<NTH>(sum, red) * a.inv_h + a.eps);
    if (threadIdx.x == 0 && a.rstd != nullptr)
        a.rstd[row] = rstd;
    if constexpr (VPT > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int v = threadIdx.x + i * NTH;
            if (v < a.V)
                norm_store(a, row, v, s[i], w[i], rstd);
        }
    } else {
        for (int v = threadIdx.x; v < a.V; v += NTH) {
            // the residual stream may be updated in place: this thread reads
            // its vector again before it overwrites it
            load(v, s[0]);
            if (a.residual_out != nullptr)
                a.residual_out[base + v] = pack8(s[0]);
            norm_store(a, row, v, s[0], a.weight[v], rstd);
        }
    }
}

// ---------------------------------------------------------------- backward

struct NormBackArgs {
    const u32x4 *dout, *h, *weight, *dresidual;  // dresidual nullable
    const float *rstd;
    u32x4 *dx;
    float *parts;  // [blocks][H]
    int64_t T;
    int V;
    float inv_h;
};

__device__ __forceinline__ void norm_back(const float (&d)[8], const float (&h)[8], const float (&w)[8],
                                          float rstd, float c, const u32x4 *dres, u32x4 *dx)
{
    float r[8];
    if (dres != nullptr)
        unpack8(*dres, r);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float g = rstd * (d[k] * w[k] - h[k] * rstd * c);
        r[k] = dres != nullptr ? g + r[k] : g;
    }
    __builtin_nontemporal_store(pack8(r), dx);
}

// Each block takes every gridDim.x-th row and sums its own part of dw: in
// registers (VPT > 0), or in its row of parts.  HBM bounds it (4096 rows of 7168,
// 235 MB: 35.6 us, 6.6 TB/s).
template <int NTH, int VPT>
__global__ __launch_bounds__(NTH) void rms_norm_backward_kernel(NormBackArgs a)
{
    constexpr int R = VPT > 0 ? VPT : 1;
    __shared__ float red[2][NTH / kWave];
    float dw[R][8] = {};
    float *part = a.parts + int64_t(blockIdx.x) * a.V * 8;
    u32x4 w[R];
    if constexpr (VPT > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int v = threadIdx.x + i * NTH;
            w[i] = v < a.V ? a.weight[v] : u32x4{};
        }
    }
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const int64_t base = row * a.V;
        const float rstd = a.rstd[row];
        float sum = 0.0f, wf[8], df[8], hf[8];
        u32x4 d[R], h[R];
        auto dot = [&](const u32x4 &dv, const u32x4 &hv, const u32x4 &wv) {
            unpack8(dv, df);
            unpack8(hv, hf);
            unpack8(wv, wf);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sum += df[k] * wf[k] * hf[k];
        };
        if constexpr (VPT > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int v = threadIdx.x + i * NTH;
                d[i] = v < a.V ? a.dout[base + v] : u32x4{};
                h[i] = v < a.V ? a.h[base + v] : u32x4{};
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
                dot(d[i], h[i], w[i]);
        } else {
            for (int v = threadIdx.x; v < a.V; v += NTH)
                dot(a.dout[base + v], a.h[base + v], a.weight[v]);
        }
        // two LDS rows in turn: a row's sum is read before the next but one writes
        const float c = block_sum<NTH>(sum, red[flip]) * rstd * a.inv_h;
        flip ^= 1;
        auto finish = [&](int v, const u32x4 &dv, const u32x4 &hv, const u32x4 &wv, float (&acc)[8]) {
            unpack8(dv, df);
            unpack8(hv, hf);
            unpack8(wv, wf);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                acc[k] += df[k] * (hf[k] * rstd);
            norm_back(df, hf, wf, rstd, c, a.dresidual != nullptr ? a.dresidual + base + v : nullptr,
                      a.dx + base + v);
        };
        if constexpr (VPT > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int v = threadIdx.x + i * NTH;
                if (v < a.V)
                    finish(v, d[i], h[i], w[i], dw[i]);
            }
        } else {
            for (int v = threadIdx.x; v < a.V; v += NTH) {
                float acc[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    acc[k] = row == int64_t(blockIdx.x) ? 0.0f : part[int64_t(v) * 8 + k];
                finish(v, a.dout[base + v], a.h[base + v], a.weight[v], acc);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    part[int64_t(v) * 8 + k] = acc[k];
            }
        }
    }
    if constexpr (VPT > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int v = threadIdx.x + i * NTH;
            if (v < a.V) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    part[int64_t(v) * 8 + k] = dw[i][k];
            }
        }
    }
}

// dw[c] = the parts' sum: 16 threads a column take every 16th part, then add
// up in a fixed order.
__global__ __launch_bounds__(1024) void sum_parts_kernel(const float *__restrict__ parts, int n, int H,
                                                         float *__restrict__ dw)
{
    __shared__ float s[16][64];
    const int col = blockIdx.x * 64 + (threadIdx.x & 63), g = threadIdx.x >> 6;
    float v = 0.0f;
    if (col < H) {
        int p = g;
        for (; p + 112 < n; p += 128) {  // eight loads in flight
            float l[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                l[i] = parts[int64_t(p + 16 * i) * H + col];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v += l[i];
        }
        for (; p < n; p += 16)
            v += parts[int64_t(p) * H + col];
    }
    s[g][threadIdx.x & 63] = v;
    __syncthreads();
    if (g == 0 && col < H) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            t += s[i][threadIdx.x & 63];
        dw[col] = t;
    }
}

}  // namespace

hipError_t launch_sum_parts(const float *parts, int n, int width, float *out, hipStream_t stream)
{
    hipLaunchKernelGGL(sum_parts_kernel, dim3((width + 63) / 64), dim3(1024), 0, stream, parts, n, width, out);
    return hipGetLastError();
}

hipError_t launch_rms_norm(int64_t T, int H, float eps, const void *x, const void *residual,
                           const void *weight, void *residual_out, void *out, void *out_q,
                           float *out_scale, float *rstd, hipStream_t stream)
{
    if (T == 0)
        return hipSuccess;
    NormArgs a{};
    a.x = static_cast<const u32x4 *>(x);
    a.residual = static_cast<const u32x4 *>(residual);
    a.weight = static_cast<const u32x4 *>(weight);
    a.residual_out = static_cast<u32x4 *>(residual_out);
    a.out = static_cast<u32x4 *>(out);
    a.out_q = static_cast<uint2 *>(out_q);
    a.out_scale = out_scale;
    a.rstd = rstd;
    a.T = T;
    a.V = H / 8;
    a.eps = eps;
    a.inv_h = 1.0f / float(H);
    const dim3 grid = row_grid(T);
    if (log_enabled())
        log_launch("rms_norm: T=%lld H=%d%s%s", (long long)T, H, residual != nullptr ? " residual" : "",
                   out_q != nullptr ? " fp8" : "");
    // a thread a vector as far as a block goes: the shortest path through one row (one
    // row of 7168: 3.0 us, with four vectors a thread 4.9) and no slower for many
    // (8192 of them: 74.2 us, with four vectors 78.2)
    if (a.V <= 64)
        hipLaunchKernelGGL((rms_norm_kernel<64, 1>), grid, dim3(64), 0, stream, a);
    else if (a.V <= 256)
        hipLaunchKernelGGL((rms_norm_kernel<256, 1>), grid, dim3(256), 0, stream, a);
    else if (a.V <= 512)
        hipLaunchKernelGGL((rms_norm_kernel<512, 1>), grid, dim3(512), 0, stream, a);
    else if (a.V <= 1024)
        hipLaunchKernelGGL((rms_norm_kernel<1024, 1>), grid, dim3(1024), 0, stream, a);
    else if (a.V <= 4096)
        hipLaunchKernelGGL((rms_norm_kernel<1024, 4>), grid, dim3(1024), 0, stream, a);
    else
        hipLaunchKernelGGL((rms_norm_kernel<1024, 0>), grid, dim3(1024), 0, stream, a);
    return hipGetLastError();
}

// Two blocks a compute unit (4096 rows of 7168: 35.6 us and 4.7 for their sum; of
// 256 blocks 38.7 and 4.7, of 1024 39.5 and 5.8).
int rms_norm_parts(int64_t T) { return int(T < 512 ? T : 512); }

hipError_t launch_rms_norm_backward(int64_t T, int H, const void *dout, const void *h,
                                    const void *weight, const float *rstd, const void *dresidual,
                                    void *dx, float *dweight, float *parts, hipStream_t stream)
{
    const int n = rms_norm_parts(T);
    NormBackArgs a{};
    a.dout = static_cast<const u32x4 *>(dout);
    a.h = static_cast<const u32x4 *>(h);
    a.weight = static_cast<const u32x4 *>(weight);
    a.dresidual = static_cast<const u32x4 *>(dresidual);
    a.rstd = rstd;
    a.dx = static_cast<u32x4 *>(dx);
    a.parts = parts;
    a.T = T;
    a.V = H / 8;
    a.inv_h = 1.0f / float(H);
    if (log_enabled())
        log_launch("rms_norm_backward: T=%lld H=%d blocks=%d", (long long)T, H, n);
    if (n > 0) {
        if (a.V <= 64)
            hipLaunchKernelGGL((rms_norm_backward_kernel<64, 1>), dim3(n), dim3(64), 0, stream, a);
        else if (a.V <= 256)
            hipLaunchKernelGGL((rms_norm_backward_kernel<256, 1>), dim3(n), dim3(256), 0, stream, a);
        else if (a.V <= 512)
            hipLaunchKernelGGL((rms_norm_backward_kernel<512, 1>), dim3(n), dim3(512), 0, stream, a);
        else if (a.V <= 1024)
            hipLaunchKernelGGL((rms_norm_backward_kernel<512, 2>), dim3(n), dim3(512), 0, stream, a);
        else if (a.V <= 2048)
            hipLaunchKernelGGL((rms_norm_backward_kernel<1024, 2>), dim3(n), dim3(1024), 0, stream, a);
        else
            hipLaunchKernelGGL((rms_norm_backward_kernel<1024, 0>), dim3(n), dim3(1024), 0, stream, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return launch_sum_parts(parts, n, H, dweight, stream);
}

}  // namespace ep
