// Internal launch interface of the 8-bit head kernels (not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace sbk {

// Largest hidden size: 131071 products of -128 * -128 still fit 32 bits.
constexpr int kInt8MaxH = 131071;

// Batches of up to kInt8SmallRows rows stream the weight once past all of
// them (int8_rows_kernel); larger ones run MFMA tiles, and so do more than
// kInt8FewRows rows on heads of kInt8FewV columns or more: such heads fill half the
// card with tiles or more, whatever their lanes, without the split of K that
// narrower ones need either way (tiles and streaming at B 64, H 4096: V 28672 39
// and 46 us, V 50257 64 and 74 us, V 8192 35 and 35 us; H 8192, V 4096 53 and 35
// us; at B 32, V 50257 63 and 59 us).
constexpr int kInt8SmallRows = 64, kInt8FewRows = 32, kInt8FewV = 16384;
inline bool int8_few(int32_t B, int32_t V)
{
    return B <= (V < kInt8FewV ? kInt8SmallRows : kInt8FewRows);
}
constexpr int kInt8SmallTile = 64;   // channels per workgroup of the streaming kernel
constexpr int kInt8LargeTile = 256;  // channels per tile of the MFMA kernel
constexpr int int8_tile(bool few) { return few ? kInt8SmallTile : kInt8LargeTile; }

struct Int8Args {
    const int8_t *w[kMaxLanes];       // lane i's channels, int8 [V_i][ldw]
    const float *w_scale[kMaxLanes];  // [V_i]
    int32_t off[kMaxLanes + 1];       // vocab offsets
    int32_t tile0[kMaxLanes + 1];     // first tile of lane i (int8_tile(few) channels each)
    int32_t k;
    const int8_t *x;                  // int8 [B][ldx]
    const float *x_scale;             // [B]
    int64_t ldx, ldw;
    int32_t B, H, V;
    bool few;                         // int8_few(B, V): the streaming kernel
    // the product: fp32 or bf16 [B][ldo]
    void *out;
    int64_t ldo;
    int32_t bf16;
    // greedy token IDs: one (value, lowest index) pair per row and tile (or per
    // row and chunk of kInt8Chunk columns of a split product)
    int2 *pair;                       // [B][pairs]
    int32_t pairs;
    int32_t *ids;                     // [B]
    // K slices: slice s holds K steps s * slice_steps ..
    int32_t slices, slice_steps;      // steps of kInt8StepK
    int32_t *part;                    // [slices][B][tiles * int8_tile(few)]
};

// Whether the MFMA kernel runs small tiles (`tiles` of kInt8LargeTile channels):
// 0.8 of the big ones' time up to 128 rows, 0.7 to 0.8 on 56 to 112 tiles, 1.2
// where big tiles fill the card.
constexpr int kInt8TileSmallRows = 128, kInt8SmallTiles = 128;
bool int8_small(int32_t B, int32_t tiles);

constexpr int kInt8StepK = 128;  // a cache line of every channel
constexpr int kInt8Chunk = 1024;

// K slices for `tiles` tiles.
int int8_slices(bool few, int32_t B, int32_t H, int32_t tiles);
int int8_slice_steps(int32_t H, int slices);

hipError_t launch_int8_quantize_rows(const uint16_t *x, int64_t ldx, int32_t B, int32_t H, int8_t *q,
                                     int64_t ldq, float *scale, hipStream_t s);

struct Int8QuantizeArgs {
    const uint16_t *w[kMaxLanes];  // bf16 [H][ldw]
    int8_t *q[kMaxLanes];          // int8 [V_i][ldq]
    float *scale[kMaxLanes];       // [V_i]
    int32_t off[kMaxLanes + 1];
    int32_t tile0[kMaxLanes + 1];  // first tile of kInt8QuantizeTile channels of lane i
    int32_t k, H;
    int64_t ldw, ldq;
};
constexpr int kInt8QuantizeTile = 64, kInt8QuantizeThreads = 512;
hipError_t launch_int8_quantize_head(const Int8QuantizeArgs &a, hipStream_t s);

// The scaled product (a.out) or the pairs and IDs (a.ids).
hipError_t launch_int8(const Int8Args &a, hipStream_t s);

// Work items of the largest launch of a product of B rows on `tiles` tiles.
int64_t int8_launch_items(bool few, int32_t B, int64_t tiles, int32_t slices);

}  // namespace sbk
