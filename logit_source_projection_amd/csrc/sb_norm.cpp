// libsb C ABI: layer norm and its gradient -- argument validation, workspace
// layout and launches.  Everything is checked on the host before the first
// launch, so an error status means nothing was enqueued.
#include <string.h>

#include "../../include/sb.h"
#include "norm.h"
#include "values.h"

namespace {

constexpr int32_t kMostColumns = 1 << 24;

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool is_type(int t) { return t == SB_FP32 || t == SB_BF16; }
int bytes_of(int t) { return t == SB_BF16 ? 2 : 4; }

// A matrix of B rows of H values.
sb_status check_rows(const void *p, int type, int64_t ld, int32_t B, int32_t H)
{
    if (!is_type(type) || ld < H)
        return SB_ERR_SHAPE;
    if (B > 0) {
        if (!p)
            return SB_ERR_NULL;
        if (!aligned(p, 16) || ld % (16 / bytes_of(type)) != 0)
            return SB_ERR_ALIGN;
    }
    return sbk::spans_addresses(B, ld, bytes_of(type)) ? SB_ERR_UNSUPPORTED : SB_OK;
}

sb_status check(const sb_norm_desc *d)
{
    if (!d)
        return SB_ERR_NULL;
    // (a NaN eps is no number >= 0)
    if (d->B < 0 || d->H < 1 || !is_type(d->param_type) || !(d->eps >= 0.f) || d->eps > 3.402823466e38f)
        return SB_ERR_SHAPE;
    const sb_status st = check_rows(d->x, d->x_type, d->ldx, d->B, d->H);
    if (st != SB_OK)
        return st;
    if (!aligned(d->weight, 16) || !aligned(d->bias, 16))
        return SB_ERR_ALIGN;
    return d->H > kMostColumns ? SB_ERR_UNSUPPORTED : SB_OK;
}

int64_t part_row(int32_t H) { return ((int64_t)H + 7) & ~(int64_t)7; }

size_t grad_bytes(const sb_norm_desc *d)
{
    return d->B == 0 ? 0 : (size_t)sbk::norm_parts(d->B, d->H) * 2 * (size_t)part_row(d->H) * sizeof(float);
}

sbk::NormArgs args_of(const sb_norm_desc *d)
{
    sbk::NormArgs a;
    memset(&a, 0, sizeof a);
    a.x = d->x;
    a.weight = d->weight;
    a.bias = d->bias;
    a.ldx = d->ldx;
    a.B = d->B;
    a.H = d->H;
    a.eps = d->eps;
    a.x_bf16 = d->x_type == SB_BF16;
    a.params_bf16 = d->param_type == SB_BF16;
    return a;
}

}  // namespace

extern "C" {

sb_status sb_layer_norm(const sb_norm_desc *desc, void *y, int y_type, int64_t ldy, float *mean,
                        float *rstd, void *stream)
{
    sb_status st = check(desc);
    if (st != SB_OK || (st = check_rows(y, y_type, ldy, desc->B, desc->H)) != SB_OK)
        return st;
    if (!aligned(mean, 4) || !aligned(rstd, 4))
        return SB_ERR_ALIGN;
    if (desc->B == 0)
        return SB_OK;
    sbk::NormArgs a = args_of(desc);
    a.y = y;
    a.ldy = ldy;
    a.y_bf16 = y_type == SB_BF16;
    a.mean = mean;
    a.rstd = rstd;
    return sbk::launch_norm(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SB_OK : SB_ERR_HIP;
}

size_t sb_layer_norm_grad_workspace_bytes(const sb_norm_desc *desc, sb_status *status)
{
    const sb_status st = check(desc);
    if (status)
        *status = st;
    return st == SB_OK ? grad_bytes(desc) : 0;
}

sb_status sb_layer_norm_grad(const sb_norm_desc *desc, const void *dy, int dy_type, int64_t lddy,
                             const float *mean, const float *rstd, void *dx, int64_t lddx,
                             void *dweight, void *dbias, void *ws, size_t ws_bytes, void *stream)
{
    sb_status st = check(desc);
    if (st != SB_OK || (st = check_rows(dy, dy_type, lddy, desc->B, desc->H)) != SB_OK)
        return st;
    if (dx && (st = check_rows(dx, desc->x_type, lddx, desc->B, desc->H)) != SB_OK)
        return st;
    const bool params = dweight || dbias;
    if (!dx && !params)
        return SB_ERR_NULL;
    if (desc->B > 0 && (!mean || !rstd))
        return SB_ERR_NULL;
    if (!aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 16) || !aligned(dbias, 16))
        return SB_ERR_ALIGN;
    if (params && grad_bytes(desc) > 0) {
        if (!ws)
            return SB_ERR_NULL;
        if (ws_bytes < grad_bytes(desc))
            return SB_ERR_WORKSPACE;
        if (!aligned(ws, 16))
            return SB_ERR_ALIGN;
    }
    if (desc->B == 0 && !params)
        return SB_OK;
    sbk::NormArgs a = args_of(desc);
    a.dy = dy;
    a.lddy = lddy;
    a.y_bf16 = dy_type == SB_BF16;
    a.mean_in = mean;
    a.rstd_in = rstd;
    a.dx = dx;
    a.lddx = lddx;
    a.dweight = dweight;
    a.dbias = dbias;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (params) {
        a.part = static_cast<float *>(ws);
        a.ldpart = part_row(desc->H);
        a.parts = desc->B == 0 ? 0 : sbk::norm_parts(desc->B, desc->H);
    }
    if (desc->B > 0 && sbk::launch_norm_grad(a, s) != hipSuccess)
        return SB_ERR_HIP;
    if (desc->B > 0 && sbk::norm_grad_few(desc->B, desc->H))
        return SB_OK;
    return !params || sbk::launch_norm_params(a, s) == hipSuccess ? SB_OK : SB_ERR_HIP;
}

}  // extern "C"
