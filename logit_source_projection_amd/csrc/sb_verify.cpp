// libsb C ABI: verification of drafted tokens -- argument validation, workspace
// layout and launches.  Everything is checked on the host before the first
// launch, so an error status means nothing was enqueued.
#include <string.h>

#include "../../include/sb.h"
#include "values.h"
#include "verify.h"

namespace {

constexpr size_t kRegionAlign = 256;
constexpr int32_t kMaxVocab = 1 << 30;
constexpr int64_t kMostGroups = 1 << 24;  // workgroups that a launch stays below

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }
bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int64_t chunks_of(int32_t V, int columns = sbk::kVerifyChunk) { return ((int64_t)V + columns - 1) / columns; }

sb_status check(const sb_drafts_desc *d)
{
    if (!d)
        return SB_ERR_NULL;
    if (d->N < 0 || d->K < 0 || d->V < 1 || d->drafts < 0 || (d->type != SB_FP32 && d->type != SB_BF16) ||
        d->ldt < d->V || (d->draft && d->ldd < d->V))
        return SB_ERR_SHAPE;
    const int64_t bytes = d->type == SB_BF16 ? 2 : 4, unit = 16 / bytes;
    if (d->N > 0) {
        if (!d->offsets || !d->target || (d->drafts > 0 && !d->tokens))
            return SB_ERR_NULL;
        if (!aligned(d->offsets, 4) || !aligned(d->tokens, 4) || !aligned(d->temperature, 4) ||
            !aligned(d->target, 16) || d->ldt % unit != 0)
            return SB_ERR_ALIGN;
        if (d->draft && (!aligned(d->draft, 16) || d->ldd % unit != 0))
            return SB_ERR_ALIGN;
    }
    if (d->V > kMaxVocab || sbk::spans_addresses((int64_t)d->drafts + d->N, d->ldt, bytes) ||
        (d->draft && sbk::spans_addresses(d->drafts, d->ldd, bytes)))
        return SB_ERR_UNSUPPORTED;
    // (each factor below 2^32, and the first two together below 2^24)
    if ((int64_t)d->N * chunks_of(d->V, sbk::kVerifyDraw) >= kMostGroups ||
        (int64_t)d->N * (2 * (int64_t)d->K + 1) >= kMostGroups ||
        (int64_t)d->N * (2 * (int64_t)d->K + 1) * chunks_of(d->V) >= kMostGroups)
        return SB_ERR_UNSUPPORTED;
    return SB_OK;
}

int64_t slots_of(const sb_drafts_desc *d) { return (d->draft ? 2 : 1) * (int64_t)d->K + 1; }

struct Layout {
    size_t parts = 0, made = 0, rest = 0, done = 0, total = 0;
};

Layout layout(const sb_drafts_desc *d)
{
    Layout L;
    const size_t rows = (size_t)d->N * chunks_of(d->V);
    size_t at = up(rows * (size_t)slots_of(d) * sizeof(sbk::RowPart), kRegionAlign);
    L.made = at;
    at = up(at + (size_t)d->N * sizeof(sbk::Verdict), kRegionAlign);
    L.rest = at;
    at = up(at + (size_t)d->N * chunks_of(d->V, sbk::kVerifyDraw) * 2 * sizeof(double), kRegionAlign);
    L.done = at;
    L.total = up(at + (size_t)d->N * sbk::kVerifyDone * sizeof(uint32_t), kRegionAlign);
    return L;
}

}  // namespace

extern "C" {

size_t sb_verify_workspace_bytes(const sb_drafts_desc *desc, sb_status *status)
{
    const sb_status st = check(desc);
    if (status)
        *status = st;
    return st == SB_OK ? layout(desc).total : 0;
}

sb_status sb_verify_drafts(const sb_drafts_desc *desc, const float *u, const float *u_next, int32_t *out,
                           int64_t ldo, int32_t *accepted, void *ws, size_t ws_bytes, void *stream)
{
    const sb_status st = check(desc);
    if (st != SB_OK)
        return st;
    if (ldo < (int64_t)desc->K + 1)
        return SB_ERR_SHAPE;
    if (desc->N == 0)
        return SB_OK;
    if (!u_next || !out || !accepted || (desc->drafts > 0 && !u))
        return SB_ERR_NULL;
    if (!aligned(u, 4) || !aligned(u_next, 4) || !aligned(out, 4) || !aligned(accepted, 4))
        return SB_ERR_ALIGN;
    if (sbk::spans_addresses(desc->N, ldo, 4))
        return SB_ERR_UNSUPPORTED;
    const Layout L = layout(desc);
    if (!ws)
        return SB_ERR_NULL;
    if (ws_bytes < L.total)
        return SB_ERR_WORKSPACE;
    if (!aligned(ws, 16))
        return SB_ERR_ALIGN;
    char *base = static_cast<char *>(ws);
    sbk::VerifyArgs a;
    memset(&a, 0, sizeof a);
    a.offsets = desc->offsets;
    a.tokens = desc->tokens;
    a.target = desc->target;
    a.draft = desc->draft;
    a.ldt = desc->ldt;
    a.ldd = desc->ldd;
    a.temperature = desc->temperature;
    a.u = u;
    a.u_next = u_next;
    a.N = desc->N;
    a.K = desc->K;
    a.V = desc->V;
    a.drafts = desc->drafts;
    a.slots = (int32_t)slots_of(desc);
    a.chunks = (int32_t)chunks_of(desc->V);
    a.draws = (int32_t)chunks_of(desc->V, sbk::kVerifyDraw);
    a.bf16 = desc->type == SB_BF16;
    a.parts = reinterpret_cast<sbk::RowPart *>(base + L.parts);
    a.made = reinterpret_cast<sbk::Verdict *>(base + L.made);
    a.rest = reinterpret_cast<double *>(base + L.rest);
    a.done = reinterpret_cast<uint32_t *>(base + L.done);
    a.out = out;
    a.ldo = ldo;
    a.accepted = accepted;
    return sbk::launch_verify(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SB_OK : SB_ERR_HIP;
}

}  // extern "C"
