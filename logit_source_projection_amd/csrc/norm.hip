// Layer norm of rows and its gradient (gfx950).
//
//   mean = sum_h x / H,  rstd = 1 / sqrt(sum_h (x - mean)^2 / H + eps)
//   xh = (x - mean) rstd,  y = xh w + b
//   g = dy w,  dx = rstd (g - sum_h g / H - xh sum_h g xh / H)
//   dw = sum_b dy xh,  db = sum_b dy
//
// Sums are fp32; the variance is that of the differences from the mean, not a
// difference of two large sums.  y, dx, dw and db are rounded once.
#include "norm.h"

#include <algorithm>

#include "values.h"

namespace sbk {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int64_t kMostRows = 1 << 20;  // workgroups that rows are dealt to

// The sum over the workgroup; every thread has it.  `scratch` holds a float per
// wave and is free again after the next barrier.
__device__ __forceinline__ float group_sum(float v, float *scratch)
{
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0)
        scratch[threadIdx.x >> 6] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
        v += scratch[w];
    return v;
}

// Values c .. of a parameter, `other` where there is none.
__device__ __forceinline__ void load_param(const void *p, bool bf16, int c, int n, float other, float (&v)[8])
{
    if (!p) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = other;
    } else if (bf16) {
        values_of(load_some(static_cast<const bf16_t *>(p) + c, n), v);
    } else {
        values_of(load_some(static_cast<const float *>(p) + c, n), v);
    }
}

// ---------------------------------------------------------------------------
// One workgroup per row, reading it once per sum.
// ---------------------------------------------------------------------------
template <typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void norm_rows_kernel(const NormArgs a)
{
    __shared__ float scratch[2][kWaves];
    const int H = a.H, units = (H + 7) / 8;
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        const TX *x = static_cast<const TX *>(a.x) + b * a.ldx;
        TY *y = static_cast<TY *>(a.y) + b * a.ldy;
        float sum = 0.f, v[8];
        for (int u = threadIdx.x; u < units; u += kThreads) {
            values_of(load_some(x + 8 * u, H - 8 * u), v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum += v[e];
        }
        const float mean = group_sum(sum, scratch[0]) / H;
        float squares = 0.f;
        for (int u = threadIdx.x; u < units; u += kThreads) {
            values_of(load_some(x + 8 * u, H - 8 * u), v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = 8 * u + e < H ? v[e] - mean : 0.f;
                squares += d * d;
            }
        }
        const float rstd = 1.f / sqrtf(group_sum(squares, scratch[1]) / H + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[b] = mean;
            if (a.rstd)
                a.rstd[b] = rstd;
        }
        for (int u = threadIdx.x; u < units; u += kThreads) {
            float w[8], s[8];
            values_of(load_some(x + 8 * u, H - 8 * u), v);
            load_param(a.weight, a.params_bf16, 8 * u, H - 8 * u, 1.f, w);
            load_param(a.bias, a.params_bf16, 8 * u, H - 8 * u, 0.f, s);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = (v[e] - mean) * rstd * w[e] + s[e];
            store_some(y + 8 * u, v, H - 8 * u);
        }
    }
}

// dx, a workgroup per row.
template <typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void norm_grad_rows_kernel(const NormArgs a)
{
    __shared__ float scratch[2][kWaves];
    const int H = a.H, units = (H + 7) / 8;
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        const TX *x = static_cast<const TX *>(a.x) + b * a.ldx;
        const TY *dy = static_cast<const TY *>(a.dy) + b * a.lddy;
        TX *dx = static_cast<TX *>(a.dx) + b * a.lddx;
        const float mean = a.mean_in[b], rstd = a.rstd_in[b];
        float sum = 0.f, cross = 0.f;
        float xv[8], gv[8], w[8];
        for (int u = threadIdx.x; u < units; u += kThreads) {
            const int n = H - 8 * u;
            values_of(load_some(x + 8 * u, n), xv);
            values_of(load_some(dy + 8 * u, n), gv);
            load_param(a.weight, a.params_bf16, 8 * u, n, 1.f, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = e < n ? gv[e] * w[e] : 0.f;
                sum += g;
                cross += e < n ? g * ((xv[e] - mean) * rstd) : 0.f;
            }
        }
        // (both scratch arrays are free: the last read of each is a barrier away)
        const float m = group_sum(sum, scratch[0]) / H, k = group_sum(cross, scratch[1]) / H;
        for (int u = threadIdx.x; u < units; u += kThreads) {
            const int n = H - 8 * u;
            values_of(load_some(x + 8 * u, n), xv);
            values_of(load_some(dy + 8 * u, n), gv);
            load_param(a.weight, a.params_bf16, 8 * u, n, 1.f, w);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                xv[e] = rstd * (gv[e] * w[e] - m - (xv[e] - mean) * rstd * k);
            store_some(dx + 8 * u, xv, n);
        }
    }
}

// The parameters' sums over one run of rows, a unit of columns per thread.
template <typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void norm_grad_columns_kernel(const NormArgs a)
{
    const int u = blockIdx.x * kThreads + threadIdx.x, n = a.H - 8 * u;
    if (n <= 0)
        return;
    float dw[8] = {}, db[8] = {};
    for (int64_t b = blockIdx.y; b < a.B; b += gridDim.y) {
        float xv[8], gv[8];
        values_of(load_some(static_cast<const TX *>(a.x) + b * a.ldx + 8 * u, n), xv);
        values_of(load_some(static_cast<const TY *>(a.dy) + b * a.lddy + 8 * u, n), gv);
        const float mean = a.mean_in[b], rstd = a.rstd_in[b];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw[e] += gv[e] * ((xv[e] - mean) * rstd);
            db[e] += gv[e];
        }
    }
    float *part = a.part + (int64_t)blockIdx.y * 2 * a.ldpart + 8 * u;
    store_some(part, dw, 8);
    store_some(part + a.ldpart, db, 8);
}

// dw and db: the runs' sums added in order.
__global__ __launch_bounds__(kThreads) void norm_params_kernel(const NormArgs a)
{
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.H)
        return;
    float dw = 0.f, db = 0.f;
    for (int p = 0; p < a.parts; ++p) {
        dw += a.part[(int64_t)2 * p * a.ldpart + c];
        db += a.part[((int64_t)2 * p + 1) * a.ldpart + c];
    }
    if (a.dweight)
        a.params_bf16 ? put(static_cast<bf16_t *>(a.dweight) + c, dw) : put(static_cast<float *>(a.dweight) + c, dw);
    if (a.dbias)
        a.params_bf16 ? put(static_cast<bf16_t *>(a.dbias) + c, db) : put(static_cast<float *>(a.dbias) + c, db);
}

template <typename TX, typename TY>
hipError_t forward(const NormArgs &a, hipStream_t s)
{
    const unsigned rows = (unsigned)std::min<int64_t>(a.B, kMostRows);
    hipLaunchKernelGGL((norm_rows_kernel<TX, TY>), dim3(rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

template <typename TX, typename TY>
hipError_t gradient(const NormArgs &a, hipStream_t s)
{
    if (a.dx) {
        const unsigned rows = (unsigned)std::min<int64_t>(a.B, kMostRows);
        hipLaunchKernelGGL((norm_grad_rows_kernel<TX, TY>), dim3(rows), dim3(kThreads), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || !a.part)
            return e;
    }
    const unsigned chunks = (unsigned)(((a.H + 7) / 8 + kThreads - 1) / kThreads);
    hipLaunchKernelGGL((norm_grad_columns_kernel<TX, TY>), dim3(chunks, (unsigned)a.parts), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

int norm_parts(int32_t B, int32_t H)
{
    return std::min(B, 256);
}

hipError_t launch_norm(const NormArgs &a, hipStream_t s)
{
    if (a.x_bf16)
        return a.y_bf16 ? forward<bf16_t, bf16_t>(a, s) : forward<bf16_t, float>(a, s);
    return a.y_bf16 ? forward<float, bf16_t>(a, s) : forward<float, float>(a, s);
}

hipError_t launch_norm_grad(const NormArgs &a, hipStream_t s)
{
    if (a.x_bf16)
        return a.y_bf16 ? gradient<bf16_t, bf16_t>(a, s) : gradient<bf16_t, float>(a, s);
    return a.y_bf16 ? gradient<float, bf16_t>(a, s) : gradient<float, float>(a, s);
}

hipError_t launch_norm_params(const NormArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(norm_params_kernel, dim3((unsigned)((a.H + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace sbk
