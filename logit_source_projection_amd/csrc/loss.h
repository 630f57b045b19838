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
    // K slices of the logits, slice s holding the K steps s * slice_steps .. of
    // kLossStepK, and their sums (with several slices one piece is all blocks)
    int32_t slices, slice_steps;
    float *zp;               // fp32 [slices][B][blocks * kVocabBlock], with two slices or more
    // loss
    float2 *mse;             // {maximum, sum exp(z - maximum)}: [parts][B], or with up to
                             // kLossSmallRows rows or several slices [B][parts]
    int32_t parts;           // runs of columns that the row's sum is made of
    float *zt;               // [B] the target's logit
    float *loss, *lse;       // [B]
    // gradient
    const float *lse_in;     // [B]
    const float *dloss;      // [B]
    uint16_t *dz;            // bf16 [dz_parts(B)][B][ldz], whose sum is dz, columns of
                             // blocks nb0 ..
    int64_t ldz;
    uint16_t *rest;          // bf16 [B], ldrest apart: what rounding took from the target's dz,
    int64_t ldrest;          // relative to what is left, where dz_parts(B) is 1
    const uint16_t *xm;      // bf16 [B][ldxm]: x with the ignored rows zeroed
    int64_t ldxm;
    float *dxp;              // fp32 [splits][B][ldxp] partial sums of dx, or NULL
    int64_t ldxp;
    uint16_t *dx;            // bf16 [B][lddx], or NULL
    int64_t lddx, lddw;
    int32_t splits;          // K splits of dx
    int32_t first, last;     // the first launch on dxp stores, later ones add
};

// Batches of up to kLossSmallRows rows stream the weight past all of them; larger
// ones run MFMA tiles of two sizes (small_logits, small_grad).
constexpr int kLossSmallRows = 64;
constexpr int kLossStepK = 32;        // K rows per MFMA step
constexpr int kLossSmallTile = 128;   // columns per workgroup of the streaming kernel
constexpr int kLossChunk = 1024;      // columns per workgroup that adds slices up
// bf16 parts that dz is held in.  A term that stands alone in a sum would double
// the rounding of the bf16 result.  Up to 32 rows, where any term can, a second
// part holds what the first leaves.  Above, the target's dz is the term that
// stands out in its row of dX and its column of dW, at any batch size: the row's
// others together are as large, but spread over the vocabulary.  What rounding
// took from it is kept (`rest`).  dW adds its products to the accumulators (x is
// read along rows), and so does dX where the weight's tile is in LDS (up to 64
// rows).  Larger batches would have to gather columns of the weight, a cache line
// per value (333 rows of H 1111: 50 us of 160); there dX's rows are multiplied by 1 +
// rest instead, which makes the target's term whole and moves the sum of the others by
// as much as their own roundings may.  Those stay: 2^-8 of each, independent.  The
// results are off by 1.65e-3 of their norm, their own rounding (2.4e-3 without the
// rests), for 4.8 us of 193 at 333 rows of H 1111, V 50257 and 0.19 ms of 15.2 at 4096
// of the dense head; two parts everywhere would be two more products.
constexpr int dz_parts(int B) { return B <= 32 ? 2 : 1; }
// Whether the logits of nblk blocks, and the gradient's two products, run small
// tiles (batches of more than kLossSmallRows rows).  Small tiles read each
// operand twice as often and ran 20 to 30 % longer where big ones fill the card,
// but took 0.66 to 0.91 of their time on fewer tiles than half the CUs (56 to
// 112 tiles; 198 tiles: 1.5), and 0.8 to 0.98 up to 128 rows, where a big tile
// is half empty.  The gradient has many short products: 0.62 to 0.86 up to
// 448 (tiles of dw) x (256-row blocks), 1.15 at 1792.
constexpr int kSmallRows = 128, kSmallLogitsTiles = 128, kSmallGradTiles = 1024;
bool small_logits(int32_t B, int32_t nblk);
bool small_grad(int32_t B, int32_t H, int32_t nblk);
inline int loss_parts(int B, int nblk, int slices)
{
    if (slices > 1)
        return (nblk * kVocabBlock + kLossChunk - 1) / kLossChunk;
    if (B > kLossSmallRows)
        return small_logits(B, nblk) ? 2 * nblk : nblk;
    return nblk * (kVocabBlock / kLossSmallTile);
}
int loss_slices(int32_t B, int32_t H, int32_t nblk);
int loss_slice_steps(int32_t H, int slices);

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
// The same for up to kLossSmallRows rows (all blocks in one launch; reads x, not xm).
hipError_t launch_grad_rows(const LossArgs &a, bool want_dx, bool want_dw, hipStream_t s);
// dx = sum of the splits' partial sums.
hipError_t launch_dx_finish(const LossArgs &a, hipStream_t s);

// Work items of the largest launch of a call of B rows on nblk blocks.
int64_t loss_launch_items(int32_t B, int32_t H, int32_t nblk, int32_t splits);

// K splits of dx for B rows and H columns, so that a tile's chain of K steps
// is no longer than a CU's share of the launch.
int dx_splits(int32_t B, int32_t H, int32_t nblk);

}  // namespace sbk
