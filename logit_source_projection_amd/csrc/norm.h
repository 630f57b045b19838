// Internal launch interface of the layer norm kernels (not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sbk {

struct NormArgs {
    const void *x;             // [B][ldx], fp32 or bf16
    const void *weight, *bias; // [H] of one type, or NULL (1 and 0)
    int64_t ldx;
    int32_t B, H;
    float eps;
    bool x_bf16, y_bf16, params_bf16;  // else fp32
    // forward
    void *y;                   // [B][ldy]
    int64_t ldy;
    float *mean, *rstd;        // [B], or NULL
    // gradient
    const void *dy;            // [B][lddy], of y's type
    int64_t lddy;
    const float *mean_in, *rstd_in;  // [B]
    void *dx;                  // [B][lddx], of x's type, or NULL
    int64_t lddx;
    void *dweight, *dbias;     // [H] of the parameters' type, or NULL
    float *part;               // fp32 [parts][2][ldpart]: sums of dy xh and of dy
    int64_t ldpart;
    int32_t parts;
};

// Whether the whole gradient is one launch, without partial sums.
bool norm_grad_few(int32_t B, int32_t H);

// Runs of rows whose sums for the parameters' gradients are kept apart.
int norm_parts(int32_t B, int32_t H);

hipError_t launch_norm(const NormArgs &a, hipStream_t s);
// dx, and the partial sums where a.part is set.
hipError_t launch_norm_grad(const NormArgs &a, hipStream_t s);
// dweight and dbias from the partial sums (zeros of no rows).
hipError_t launch_norm_params(const NormArgs &a, hipStream_t s);

}  // namespace sbk
