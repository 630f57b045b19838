// libsb C ABI: the head in 8-bit integers -- argument validation, workspace
// layout and launches.  Everything is checked on the host before the first
// launch, so an error status means nothing was enqueued.
#include <string.h>

#include <algorithm>

#include "../../include/sb.h"
#include "int8.h"

namespace {

constexpr size_t kRegionAlign = 256;
constexpr int32_t kMaxVocab = 1 << 30;
constexpr int64_t kItems = (int64_t)1 << 32;  // work items a launch dimension stays below

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int64_t tiles_of(const int32_t *off, int k, int width)
{
    int64_t n = 0;
    for (int i = 0; i < k; ++i)
        n += ((int64_t)off[i + 1] - off[i] + width - 1) / width;
    return n;
}

sb_status check(const sb_int8_desc *d)
{
    if (!d || !d->lane_off || !d->w || !d->w_scale)
        return SB_ERR_NULL;
    if (d->B < 0 || d->H < 0 || d->V < 1)
        return SB_ERR_SHAPE;
    if (d->k < 1 || d->k > SB_MAX_LANES || d->lane_off[0] != 0 || d->lane_off[d->k] != d->V)
        return SB_ERR_LANES;
    for (int i = 0; i < d->k; ++i)
        if (d->lane_off[i + 1] <= d->lane_off[i])
            return SB_ERR_LANES;
    if (d->B > 0) {
        if (!d->x_scale)
            return SB_ERR_NULL;
        for (int i = 0; i < d->k; ++i)
            if (!d->w_scale[i])
                return SB_ERR_NULL;
        if (d->H > 0) {
            if (!d->x)
                return SB_ERR_NULL;
            for (int i = 0; i < d->k; ++i)
                if (!d->w[i])
                    return SB_ERR_NULL;
        }
    }
    if (d->ldx < d->H || d->ldw < d->H)
        return SB_ERR_SHAPE;
    if (d->B > 0) {
        if (!aligned(d->x_scale, 4))
            return SB_ERR_ALIGN;
        for (int i = 0; i < d->k; ++i)
            if (!aligned(d->w_scale[i], 4))
                return SB_ERR_ALIGN;
        if (d->H > 0) {
            if (!aligned(d->x, 16) || d->ldx % 16 != 0 || d->ldw % 16 != 0)
                return SB_ERR_ALIGN;
            for (int i = 0; i < d->k; ++i)
                if (!aligned(d->w[i], 16))
                    return SB_ERR_ALIGN;
        }
    }
    // exact 32-bit sums; 32-bit offsets over 256 rows and 256 channels
    if (d->V > kMaxVocab || d->H > sbk::kInt8MaxH || sbk::spans_4gib(256, d->ldx, 1) ||
        sbk::spans_4gib(256, d->ldw, 1))
        return SB_ERR_UNSUPPORTED;
    const bool few = sbk::int8_few(d->B, d->V);
    const int64_t tiles = tiles_of(d->lane_off, d->k, sbk::int8_tile(few));
    if (tiles > (1 << 30) / sbk::kInt8SmallTile ||
        sbk::int8_launch_items(few, d->B, tiles, sbk::int8_slices(few, d->B, d->H, (int32_t)tiles)) >= kItems)
        return SB_ERR_UNSUPPORTED;
    return SB_OK;
}

struct Layout {
    int32_t tiles = 0, slices = 1, pairs = 0;
    size_t part = 0, pair = 0, total = 0;
};

Layout layout(const sb_int8_desc *d, bool tokens)
{
    Layout L;
    const bool few = sbk::int8_few(d->B, d->V);
    L.tiles = (int32_t)tiles_of(d->lane_off, d->k, sbk::int8_tile(few));
    if (d->B == 0)
        return L;
    L.slices = sbk::int8_slices(few, d->B, d->H, L.tiles);
    size_t at = 0;
    if (L.slices > 1) {
        L.part = at;
        at = up(at + (size_t)L.slices * d->B * (size_t)L.tiles * sbk::int8_tile(few) * sizeof(int32_t),
                kRegionAlign);
    }
    if (tokens) {
        L.pairs = L.slices > 1 ? (L.tiles * sbk::int8_tile(few) + sbk::kInt8Chunk - 1) / sbk::kInt8Chunk
                               : L.tiles;
        if (L.slices == 1 && !few && sbk::int8_small(d->B, L.tiles))
            L.pairs *= 2;
        L.pair = at;
        at = up(at + (size_t)L.pairs * d->B * sizeof(int2), kRegionAlign);
    }
    L.total = at;
    return L;
}

sb_status check_ws(const Layout &L, void *ws, size_t ws_bytes)
{
    if (L.total == 0)
        return SB_OK;
    if (!ws)
        return SB_ERR_NULL;
    if (ws_bytes < L.total)
        return SB_ERR_WORKSPACE;
    return aligned(ws, 16) ? SB_OK : SB_ERR_ALIGN;
}

void fill(const sb_int8_desc *d, const Layout &L, void *ws, sbk::Int8Args &a)
{
    memset(&a, 0, sizeof a);
    a.few = sbk::int8_few(d->B, d->V);
    const int width = sbk::int8_tile(a.few);
    a.k = d->k;
    int tiles = 0;
    for (int i = 0; i < d->k; ++i) {
        a.w[i] = static_cast<const int8_t *>(d->w[i]);
        a.w_scale[i] = d->w_scale[i];
        a.off[i] = d->lane_off[i];
        a.tile0[i] = tiles;
        tiles += (d->lane_off[i + 1] - d->lane_off[i] + width - 1) / width;
    }
    a.off[d->k] = d->lane_off[d->k];
    a.tile0[d->k] = tiles;
    a.x = static_cast<const int8_t *>(d->x);
    a.x_scale = d->x_scale;
    a.ldx = d->ldx;
    a.ldw = d->ldw;
    a.B = d->B;
    a.H = d->H;
    a.V = d->V;
    a.slices = L.slices;
    a.slice_steps = sbk::int8_slice_steps(d->H, L.slices);
    if (L.slices > 1)
        a.part = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + L.part);
    if (L.pairs) {
        a.pair = reinterpret_cast<int2 *>(static_cast<char *>(ws) + L.pair);
        a.pairs = L.pairs;
    }
}

}  // namespace

extern "C" {

sb_status sb_int8_quantize_rows(const void *x, int64_t ldx, int32_t B, int32_t H, void *q, int64_t ldq,
                                float *scale, void *stream)
{
    if (B < 0 || H < 0 || ldx < H || ldq < H)
        return SB_ERR_SHAPE;
    if (B == 0)
        return SB_OK;
    if (!scale || (H > 0 && (!x || !q)))
        return SB_ERR_NULL;
    if (!aligned(scale, 4) ||
        (H > 0 && (!aligned(x, 16) || !aligned(q, 16) || ldx % 8 != 0 || ldq % 16 != 0)))
        return SB_ERR_ALIGN;
    if ((int64_t)B * 1024 >= kItems || H > sbk::kInt8MaxH)
        return SB_ERR_UNSUPPORTED;
    return sbk::launch_int8_quantize_rows(static_cast<const uint16_t *>(x), ldx, B, H,
                                          static_cast<int8_t *>(q), ldq, scale,
                                          static_cast<hipStream_t>(stream)) == hipSuccess
               ? SB_OK
               : SB_ERR_HIP;
}

sb_status sb_int8_quantize_head(const sb_head_desc *desc, void *const *q, int64_t ldq,
                                float *const *scale, void *stream)
{
    if (!desc || !desc->lane_off || !desc->w || !q || !scale)
        return SB_ERR_NULL;
    // the head's own rules for its weight: no rows of x are looked at
    sb_head_desc d = *desc;
    d.B = 0;
    d.x = nullptr;
    d.ldx = d.H > 0 ? d.H : 0;
    sb_status st = SB_OK;
    sb_workspace_bytes(&d, SB_SURF_TOKENS, &st);
    if (st != SB_OK)
        return st;
    if (ldq < d.H)
        return SB_ERR_SHAPE;
    for (int i = 0; i < d.k; ++i)
        if (!scale[i] || (d.H > 0 && (!q[i] || !d.w[i])))
            return SB_ERR_NULL;
    for (int i = 0; i < d.k; ++i)
        if (!aligned(scale[i], 4) || (d.H > 0 && (!aligned(q[i], 16) || !aligned(d.w[i], 16))))
            return SB_ERR_ALIGN;
    if (d.H > 0 && (ldq % 16 != 0 || d.ldw % 8 != 0))
        return SB_ERR_ALIGN;
    const int64_t tiles = tiles_of(d.lane_off, d.k, sbk::kInt8QuantizeTile);
    if (d.H > sbk::kInt8MaxH || tiles * sbk::kInt8QuantizeThreads >= kItems)
        return SB_ERR_UNSUPPORTED;
    sbk::Int8QuantizeArgs a;
    memset(&a, 0, sizeof a);
    int at = 0;
    for (int i = 0; i < d.k; ++i) {
        a.w[i] = static_cast<const uint16_t *>(d.w[i]);
        a.q[i] = static_cast<int8_t *>(q[i]);
        a.scale[i] = scale[i];
        a.off[i] = d.lane_off[i];
        a.tile0[i] = at;
        at += (d.lane_off[i + 1] - d.lane_off[i] + sbk::kInt8QuantizeTile - 1) / sbk::kInt8QuantizeTile;
    }
    a.off[d.k] = d.lane_off[d.k];
    a.tile0[d.k] = at;
    a.k = d.k;
    a.H = d.H;
    a.ldw = d.ldw;
    a.ldq = ldq;
    return sbk::launch_int8_quantize_head(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SB_OK
                                                                                             : SB_ERR_HIP;
}

size_t sb_int8_workspace_bytes(const sb_int8_desc *desc, int surface, sb_status *status)
{
    sb_status st = check(desc);
    if (st == SB_OK && surface != SB_SURF_TOKENS && surface != SB_SURF_FULL_LOGITS)
        st = SB_ERR_SHAPE;
    if (status)
        *status = st;
    return st == SB_OK ? layout(desc, surface == SB_SURF_TOKENS).total : 0;
}

sb_status sb_int8_project_tokens(const sb_int8_desc *desc, int32_t *ids, void *ws, size_t ws_bytes,
                                 void *stream)
{
    sb_status st = check(desc);
    if (st != SB_OK)
        return st;
    if (desc->B == 0)
        return SB_OK;
    if (!ids)
        return SB_ERR_NULL;
    const Layout L = layout(desc, true);
    if ((st = check_ws(L, ws, ws_bytes)) != SB_OK)
        return st;
    sbk::Int8Args a;
    fill(desc, L, ws, a);
    a.ids = ids;
    return sbk::launch_int8(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SB_OK : SB_ERR_HIP;
}

sb_status sb_int8_logits(const sb_int8_desc *desc, void *out, int dtype, int64_t ldo, void *ws,
                         size_t ws_bytes, void *stream)
{
    sb_status st = check(desc);
    if (st != SB_OK)
        return st;
    if (dtype != SB_FP32 && dtype != SB_BF16)
        return SB_ERR_SHAPE;
    if (desc->B == 0)
        return SB_OK;
    if (!out)
        return SB_ERR_NULL;
    if (ldo < desc->V)
        return SB_ERR_SHAPE;
    if (!aligned(out, 16) || ldo % (dtype == SB_FP32 ? 4 : 8) != 0)
        return SB_ERR_ALIGN;
    const Layout L = layout(desc, false);
    if ((st = check_ws(L, ws, ws_bytes)) != SB_OK)
        return st;
    sbk::Int8Args a;
    fill(desc, L, ws, a);
    a.out = out;
    a.ldo = ldo;
    a.bf16 = dtype == SB_BF16;
    return sbk::launch_int8(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SB_OK : SB_ERR_HIP;
}

}  // extern "C"
