// libsb C ABI: embedding lookup and its gradient -- argument validation,
// workspace layout and launches.  Everything is checked on the host before the
// first launch, so an error status means nothing was enqueued.
#include <math.h>
#include <string.h>

#include "../../include/sb.h"
#include "embed.h"
#include "values.h"

namespace {

constexpr size_t kRegionAlign = 256;
constexpr int32_t kMaxVocab = 1 << 30;
constexpr int32_t kMostGradVocab = 1 << 24, kMostGradRows = 1 << 24;
constexpr int32_t kMostColumns = 1 << 24;

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }
bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool is_type(int t) { return t == SB_FP32 || t == SB_BF16; }
int bytes_of(int t) { return t == SB_BF16 ? 2 : 4; }

sb_status check(const sb_table_desc *d)
{
    if (!d || !d->lane_off || !d->w)
        return SB_ERR_NULL;
    if (d->V < 1 || d->H < 0 || !is_type(d->type))
        return SB_ERR_SHAPE;
    if (d->k < 1 || d->k > SB_MAX_LANES || d->lane_off[0] != 0 || d->lane_off[d->k] != d->V)
        return SB_ERR_LANES;
    int32_t rows = 0;
    for (int i = 0; i < d->k; ++i) {
        if (d->lane_off[i + 1] <= d->lane_off[i])
            return SB_ERR_LANES;
        const int32_t n = d->lane_off[i + 1] - d->lane_off[i];
        rows = n > rows ? n : rows;
    }
    if (d->ldw < d->H)
        return SB_ERR_SHAPE;
    if (d->H > 0) {
        for (int i = 0; i < d->k; ++i)
            if (!d->w[i])
                return SB_ERR_NULL;
        if (d->ldw % (16 / bytes_of(d->type)) != 0)
            return SB_ERR_ALIGN;
        for (int i = 0; i < d->k; ++i)
            if (!aligned(d->w[i], 16))
                return SB_ERR_ALIGN;
    }
    if (d->V > kMaxVocab || d->H > kMostColumns || sbk::spans_addresses(rows, d->ldw, bytes_of(d->type)))
        return SB_ERR_UNSUPPORTED;
    return SB_OK;
}

// The rows of a call: IDs and a matrix of B rows of H values.
sb_status check_rows(const sb_table_desc *d, const int32_t *ids, int32_t B, const void *p, int type, int64_t ld,
                     float scale)
{
    if (B < 0 || !is_type(type) || ld < d->H || !isfinite(scale))
        return SB_ERR_SHAPE;
    if (B > 0 && d->H > 0) {
        if (!ids || !p)
            return SB_ERR_NULL;
        if (!aligned(ids, 4) || !aligned(p, 16) || ld % (16 / bytes_of(type)) != 0)
            return SB_ERR_ALIGN;
    }
    return sbk::spans_addresses(B, ld, bytes_of(type)) ? SB_ERR_UNSUPPORTED : SB_OK;
}

struct Layout {
    size_t start = 0, order = 0, sorted = 0, part = 0, total = 0;
    int32_t runs = 0;
    int64_t ldpart = 0;
};

Layout layout(const sb_table_desc *d, int32_t B, bool add)
{
    Layout L;
    if (d->H == 0 || (B == 0 && add))
        return L;
    size_t at = up((((size_t)sbk::embed_range(d->V) << sbk::embed_shift(d->V)) + 1) * sizeof(int32_t), kRegionAlign);
    L.order = at;
    at = up(at + (size_t)B * sizeof(int32_t), kRegionAlign);
    L.sorted = at;
    at = up(at + (size_t)B * sizeof(int32_t), kRegionAlign);
    L.runs = (B + sbk::kEmbedRun - 1) / sbk::kEmbedRun;
    L.ldpart = ((int64_t)d->H + 7) & ~(int64_t)7;
    L.part = at;
    const size_t pieces = ((size_t)B + sbk::kEmbedPiece - 1) / sbk::kEmbedPiece;
    // (one piece has no partial rows)
    L.total = up(at + (pieces > 1 ? pieces * 2 * (size_t)L.ldpart * sizeof(float) : 0), kRegionAlign);
    return L;
}

sb_status check_grad(const sb_table_desc *d, int32_t B)
{
    const sb_status st = check(d);
    if (st != SB_OK)
        return st;
    if (B < 0)
        return SB_ERR_SHAPE;
    return d->V > kMostGradVocab || B > kMostGradRows || !sbk::embed_grad_fits(B, d->H) ? SB_ERR_UNSUPPORTED
                                                                                     : SB_OK;
}

sbk::EmbedArgs args_of(const sb_table_desc *d, const int32_t *ids, int32_t B, float scale, int rows_type)
{
    sbk::EmbedArgs a;
    memset(&a, 0, sizeof a);
    for (int i = 0; i < d->k; ++i) {
        a.w[i] = d->w[i];
        a.off[i] = d->lane_off[i];
    }
    a.off[d->k] = d->lane_off[d->k];
    a.k = d->k;
    a.V = d->V;
    a.H = d->H;
    a.B = B;
    a.ldw = d->ldw;
    a.table_bf16 = d->type == SB_BF16;
    a.rows_bf16 = rows_type == SB_BF16;
    a.ids = ids;
    a.scale = scale;
    return a;
}

}  // namespace

extern "C" {

sb_status sb_embed(const sb_table_desc *desc, const int32_t *ids, int32_t B, float scale, void *out,
                   int out_type, int64_t ldo, void *stream)
{
    sb_status st = check(desc);
    if (st != SB_OK || (st = check_rows(desc, ids, B, out, out_type, ldo, scale)) != SB_OK)
        return st;
    if (B == 0 || desc->H == 0)
        return SB_OK;
    sbk::EmbedArgs a = args_of(desc, ids, B, scale, out_type);
    a.out = out;
    a.ldo = ldo;
    return sbk::launch_embed(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SB_OK : SB_ERR_HIP;
}

size_t sb_embed_grad_workspace_bytes(const sb_table_desc *desc, int32_t B, int accumulate, sb_status *status)
{
    const sb_status st = check_grad(desc, B);
    if (status)
        *status = st;
    return st == SB_OK ? layout(desc, B, accumulate != 0).total : 0;
}

sb_status sb_embed_grad(const sb_table_desc *desc, const int32_t *ids, int32_t B, float scale,
                        const void *dout, int dout_type, int64_t lddo, int accumulate, void *ws,
                        size_t ws_bytes, void *stream)
{
    sb_status st = check_grad(desc, B);
    if (st != SB_OK || (st = check_rows(desc, ids, B, dout, dout_type, lddo, scale)) != SB_OK)
        return st;
    const bool add = accumulate != 0;
    const Layout L = layout(desc, B, add);
    if (L.total == 0)
        return SB_OK;
    if (!ws)
        return SB_ERR_NULL;
    if (ws_bytes < L.total)
        return SB_ERR_WORKSPACE;
    if (!aligned(ws, 16))
        return SB_ERR_ALIGN;
    sbk::EmbedArgs a = args_of(desc, ids, B, scale, dout_type);
    char *base = static_cast<char *>(ws);
    a.dout = dout;
    a.lddo = lddo;
    a.add = add;
    a.range = sbk::embed_range(desc->V);
    a.shift = sbk::embed_shift(desc->V);
    a.start = reinterpret_cast<int32_t *>(base + L.start);
    a.order = reinterpret_cast<int32_t *>(base + L.order);
    a.sorted = reinterpret_cast<int32_t *>(base + L.sorted);
    a.part = reinterpret_cast<float *>(base + L.part);
    a.ldpart = L.ldpart;
    a.runs = L.runs;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (sbk::launch_embed_sort(a, s) != hipSuccess || sbk::launch_embed_sums(a, s) != hipSuccess)
        return SB_ERR_HIP;
    return SB_OK;
}

}  // extern "C"
