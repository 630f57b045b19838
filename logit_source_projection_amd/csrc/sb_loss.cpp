// libsb C ABI: softmax cross entropy over the head and its gradient --
// argument validation, workspace layout and launches.  Everything is checked
// on the host before the first launch, so an error status means nothing was
// enqueued.
#include <string.h>

#include <algorithm>

#include "../../include/sb.h"
#include "loss.h"

namespace {

constexpr size_t kRegionAlign = 256;
constexpr int64_t kItems = (int64_t)1 << 32;  // work items a launch dimension stays below

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int blocks_of(const sb_head_desc *d)
{
    int n = 0;
    for (int i = 0; i < d->k; ++i)
        n += (d->lane_off[i + 1] - d->lane_off[i] + sbk::kVocabBlock - 1) / sbk::kVocabBlock;
    return n;
}

// dz of a piece is at most this many bytes, the size of the last-level cache:
// its two readers find most of it there (but always one block at least).
constexpr int64_t kPieceBytes = (int64_t)256 << 20;

struct Layout {
    int blocks = 0, piece = 0, splits = 1;
    bool direct = false;  // dx written without partial sums
    int slices = 1;       // K slices of the logits
    size_t zp = 0, mse = 0, zt = 0, rest = 0, dz = 0, xm = 0, dxp = 0, total = 0;
    int64_t ldz = 0, ldxm = 0, ldxp = 0;
};

Layout layout(const sb_head_desc *d, bool grad)
{
    Layout L;
    L.blocks = blocks_of(d);
    if (d->B == 0) {
        L.piece = L.blocks;
        return L;
    }
    const size_t B = (size_t)d->B;
    size_t at = 0;
    const bool few = d->B <= sbk::kLossSmallRows;
    // (a gradient in several pieces has more tiles than are ever split)
    L.slices = sbk::loss_slices(d->B, d->H, L.blocks);
    if (L.slices > 1) {
        L.zp = at;
        at = up(at + (size_t)L.slices * B * L.blocks * sbk::kVocabBlock * sizeof(float), kRegionAlign);
    }
    if (!grad) {
        L.mse = at;
        at = up(at + B * sbk::loss_parts(d->B, L.blocks, L.slices) * sizeof(float2), kRegionAlign);
        L.zt = at;
        at = up(at + B * sizeof(float), kRegionAlign);
        L.total = at;
        return L;
    }
    if (few) {
        // all of dz; dx in partial sums
        L.piece = L.blocks;
        L.splits = sbk::dx_splits(d->B, d->H, L.blocks);
        L.ldz = (int64_t)L.blocks * sbk::kVocabBlock;
        L.ldxp = ((int64_t)d->H + 3) & ~(int64_t)3;
        L.dz = at;
        at = up(at + sbk::dz_parts(d->B) * B * (size_t)L.ldz * 2, kRegionAlign);
        L.dxp = at;
        L.total = up(at + (size_t)L.splits * B * (size_t)L.ldxp * sizeof(float), kRegionAlign);
        return L;
    }
    const int64_t most = kPieceBytes / ((int64_t)d->B * sbk::kVocabBlock * 2);
    L.piece = (int)std::max<int64_t>(1, std::min<int64_t>(L.blocks, most));
    // pieces of nearly equal size
    const int pieces = (L.blocks + L.piece - 1) / L.piece;
    L.piece = (L.blocks + pieces - 1) / pieces;
    L.splits = sbk::dx_splits(d->B, d->H, L.piece);
    L.direct = pieces == 1 && L.splits == 1;
    L.ldz = (int64_t)L.piece * sbk::kVocabBlock;
    L.ldxm = ((int64_t)d->H + 7) & ~(int64_t)7;
    L.ldxp = ((int64_t)d->H + 3) & ~(int64_t)3;
    L.dz = at;
    at = up(at + B * (size_t)L.ldz * 2, kRegionAlign);
    L.xm = at;
    at = up(at + B * (size_t)L.ldxm * 2, kRegionAlign);
    if (L.direct) {
        L.rest = at;
        at = up(at + B * 2, kRegionAlign);
    } else {
        L.dxp = at;
        at = up(at + (size_t)L.splits * B * (size_t)L.ldxp * sizeof(float), kRegionAlign);
    }
    L.total = at;
    return L;
}

// The head's own rules, then the limits of these calls.
sb_status check(const sb_head_desc *d, bool grad)
{
    sb_status st = SB_OK;
    sb_workspace_bytes(d, SB_SURF_TOKENS, &st);
    if (st != SB_OK)
        return st;
    // 32-bit offsets: 256 rows of x; 64 rows of a shard, and 256 in the gradient;
    // there also 256 rows of a piece of dz (all columns with few rows)
    if (sbk::spans_4gib(sbk::kVocabBlock, d->ldx, 2) ||
        sbk::spans_4gib(grad ? sbk::kVocabBlock : 64, d->ldw, 2))
        return SB_ERR_UNSUPPORTED;
    const Layout L = layout(d, grad);
    const int nblk = grad ? L.piece : L.blocks;
    if (grad && (sbk::spans_4gib(sbk::kVocabBlock, L.ldz, 2) || sbk::spans_4gib(64, L.ldxm, 2)))
        return SB_ERR_UNSUPPORTED;
    if (sbk::loss_launch_items(d->B, d->H, nblk, L.splits) >= kItems)
        return SB_ERR_UNSUPPORTED;
    return SB_OK;
}

sb_status check_ws(const Layout &L, void *ws, size_t ws_bytes)
{
    if (L.total == 0)
        return SB_OK;
    if (!ws)
        return SB_ERR_NULL;
    if (ws_bytes < L.total)
        return SB_ERR_WORKSPACE;
    return aligned16(ws) ? SB_OK : SB_ERR_ALIGN;
}

template <typename T>
T *region(void *ws, size_t at)
{
    return reinterpret_cast<T *>(static_cast<char *>(ws) + at);
}

void fill(const sb_head_desc *d, const int32_t *targets, sbk::LossArgs &a)
{
    memset(&a, 0, sizeof a);
    a.vocab.k = d->k;
    int nb = 0;
    for (int i = 0; i < d->k; ++i) {
        a.vocab.w[i] = static_cast<const uint16_t *>(d->w[i]);
        a.vocab.off[i] = d->lane_off[i];
        a.vocab.blk0[i] = nb;
        nb += (d->lane_off[i + 1] - d->lane_off[i] + sbk::kVocabBlock - 1) / sbk::kVocabBlock;
    }
    a.vocab.off[d->k] = d->lane_off[d->k];
    a.vocab.blk0[d->k] = nb;
    a.x = static_cast<const uint16_t *>(d->x);
    a.targets = targets;
    a.ldx = d->ldx;
    a.ldw = d->ldw;
    a.B = d->B;
    a.H = d->H;
    a.V = d->V;
    a.nblk = nb;
    a.splits = 1;
}

// The K slices of a call and their sums.
void set_slices(const sb_head_desc *d, const Layout &L, void *ws, sbk::LossArgs &a)
{
    a.slices = L.slices;
    a.slice_steps = sbk::loss_slice_steps(d->H, L.slices);
    if (L.slices > 1)
        a.zp = region<float>(ws, L.zp);
}

}  // namespace

extern "C" {

size_t sb_cross_entropy_workspace_bytes(const sb_head_desc *desc, int grad, sb_status *status)
{
    const sb_status st = check(desc, grad != 0);
    if (status)
        *status = st;
    return st == SB_OK ? layout(desc, grad != 0).total : 0;
}

sb_status sb_cross_entropy(const sb_head_desc *desc, const int32_t *targets, float *loss, float *lse,
                           void *ws, size_t ws_bytes, void *stream)
{
    sb_status st = check(desc, false);
    if (st != SB_OK)
        return st;
    if (desc->B == 0)
        return SB_OK;
    if (!targets || !loss || !lse)
        return SB_ERR_NULL;
    const Layout L = layout(desc, false);
    if ((st = check_ws(L, ws, ws_bytes)) != SB_OK)
        return st;
    sbk::LossArgs a;
    fill(desc, targets, a);
    set_slices(desc, L, ws, a);
    a.mse = region<float2>(ws, L.mse);
    a.parts = sbk::loss_parts(desc->B, L.blocks, L.slices);
    a.zt = region<float>(ws, L.zt);
    a.loss = loss;
    a.lse = lse;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (sbk::launch_loss_blocks(a, s) != hipSuccess || sbk::launch_loss_combine(a, s) != hipSuccess)
        return SB_ERR_HIP;
    return SB_OK;
}

sb_status sb_cross_entropy_grad(const sb_head_desc *desc, const int32_t *targets, const float *lse,
                                const float *dloss, void *dx, int64_t lddx, void *const *dw,
                                int64_t lddw, void *ws, size_t ws_bytes, void *stream)
{
    sb_status st = check(desc, true);
    if (st != SB_OK)
        return st;
    if (desc->H == 0 || (desc->B == 0 && !dw))
        return SB_OK;  // the gradients asked for are empty
    if (!dx && !dw)
        return SB_ERR_NULL;
    if (desc->B > 0 && (!targets || !lse || !dloss))
        return SB_ERR_NULL;
    if (dx && lddx < desc->H)
        return SB_ERR_SHAPE;
    if (dx && (!aligned16(dx) || lddx % 8 != 0))
        return SB_ERR_ALIGN;
    if (dw) {
        for (int i = 0; i < desc->k; ++i) {
            if (!dw[i])
                return SB_ERR_NULL;
            if (lddw < desc->lane_off[i + 1] - desc->lane_off[i])
                return SB_ERR_SHAPE;
        }
        for (int i = 0; i < desc->k; ++i)
            if (!aligned16(dw[i]) || lddw % 8 != 0)
                return SB_ERR_ALIGN;
    }
    const Layout L = layout(desc, true);
    if ((st = check_ws(L, ws, ws_bytes)) != SB_OK)
        return st;
    sbk::LossArgs a;
    fill(desc, targets, a);
    if (dw)
        for (int i = 0; i < desc->k; ++i)
            a.vocab.dw[i] = static_cast<uint16_t *>(dw[i]);
    a.lse_in = lse;
    a.dloss = dloss;
    a.ldz = L.ldz;
    a.ldxm = L.ldxm;
    a.dx = static_cast<uint16_t *>(dx);
    a.lddx = lddx;
    a.lddw = lddw;
    a.splits = L.splits;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (desc->B == 0)  // dw of no rows is zero
        return sbk::launch_grad(a, false, true, s) == hipSuccess ? SB_OK : SB_ERR_HIP;
    a.dz = region<uint16_t>(ws, L.dz);
    // What rounding takes from the targets' dz is needed until the last product is
    // done.  Where dx is finished by a launch of its own, its first column is free
    // until then; without dx its partial sums' memory is.
    a.rest = L.direct ? region<uint16_t>(ws, L.rest) : dx ? a.dx : region<uint16_t>(ws, L.dxp);
    a.ldrest = L.direct || !dx ? 1 : lddx;
    set_slices(desc, L, ws, a);
    if (desc->B <= sbk::kLossSmallRows) {
        a.dxp = region<float>(ws, L.dxp);
        a.ldxp = L.ldxp;
        if (sbk::launch_dlogits(a, s) != hipSuccess ||
            sbk::launch_grad_rows(a, dx != nullptr, dw != nullptr, s) != hipSuccess ||
            (dx && sbk::launch_dx_finish(a, s) != hipSuccess))
            return SB_ERR_HIP;
        return SB_OK;
    }
    a.xm = region<uint16_t>(ws, L.xm);
    if (!L.direct) {
        a.dxp = region<float>(ws, L.dxp);
        a.ldxp = L.ldxp;
    }
    if (dw && sbk::launch_mask_rows(a, region<uint16_t>(ws, L.xm), s) != hipSuccess)
        return SB_ERR_HIP;
    for (int nb = 0; nb < L.blocks; nb += L.piece) {
        a.nb0 = nb;
        a.nblk = std::min(L.piece, L.blocks - nb);
        a.first = nb == 0;
        a.last = nb + L.piece >= L.blocks;
        if (sbk::launch_dlogits(a, s) != hipSuccess ||
            sbk::launch_grad(a, dx != nullptr, dw != nullptr, s) != hipSuccess)
            return SB_ERR_HIP;
    }
    if (dx && a.dxp && sbk::launch_dx_finish(a, s) != hipSuccess)
        return SB_ERR_HIP;
    return SB_OK;
}

}  // extern "C"
