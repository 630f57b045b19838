// Internal launch interface of the loss and gradient kernels (not part of the
// C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace sbk {

// The vocabulary in blocks of kVocabBlock columns: lane i's blocks are
// blk0[i] .. blk0[i + 1] - 1, the last of them possibly short.  No block
// spans two lanes.
constexpr int kVocabBlock = 256;

struct VocabTable {
    const uint16_t *w[kMaxLanes];  // lane i's shard, bf16 [H][ldw]
    uint16_t *dw[kMaxLanes];       // its gradient, bf16 [H][lddw], or NULL
    int32_t off[kMaxLanes + 1];
    int32_t blk0[kMaxLanes + 1];
    int32_t k;
};

struct LossArgs {
    VocabTable vocab;
    const uint16_t *x;       // bf16 [B][ldx]
    const int32_t *targets;  // [B]
    int64_t ldx, ldw;
    int32_t B, H, V;
    int32_t nb0, nblk;       // the blocks of this launch
    // loss
    float2 *mse;             // [blocks][B] {block maximum, sum exp(z - maximum)}
    float *zt;               // [B] the target's logit
    float *loss, *lse;       // [B]
    // gradient
    const float *lse_in;     // [B]
    const float *dloss;      // [B]
    uint16_t *dz;            // bf16 [B][ldz], columns of blocks nb0 ..
    int64_t ldz;
    const uint16_t *xm;      // bf16 [B][ldxm]: x with the ignored rows zeroed
    int64_t ldxm;
    float *dxp;              // fp32 [splits][B][ldxp] partial sums of dx, or NULL
    int64_t ldxp;
    uint16_t *dx;            // bf16 [B][lddx], or NULL
    int64_t lddx, lddw;
    int32_t splits;          // K splits of dx
    int32_t first;           // the first launch on dxp stores, later ones add
};

// Per-block results of the logits of blocks nb0 .. nb0 + nblk - 1.
hipError_t launch_loss_blocks(const LossArgs &a, hipStream_t s);
// loss and lse of every row from the per-block results.
hipError_t launch_loss_combine(const LossArgs &a, hipStream_t s);

// xm = x with the rows of negative targets zeroed.
hipError_t launch_mask_rows(const LossArgs &a, uint16_t *xm, hipStream_t s);
// dz = (exp(z - lse) - onehot(target)) * dloss of blocks nb0 ...
hipError_t launch_dlogits(const LossArgs &a, hipStream_t s);
// dw of blocks nb0 ... and the blocks' part of dx.
hipError_t launch_grad(const LossArgs &a, bool want_dx, bool want_dw, hipStream_t s);
// dx = sum of the splits' partial sums.
hipError_t launch_dx_finish(const LossArgs &a, hipStream_t s);

// Work items of the largest launch of a call of B rows on nblk blocks.
int64_t loss_launch_items(int32_t B, int32_t H, int32_t nblk, int32_t splits);

// K splits of dx for B rows and H columns, so that a tile's chain of K steps
// is no longer than a CU's share of the launch.
int dx_splits(int32_t B, int32_t H, int32_t nblk);

}  // namespace sbk
