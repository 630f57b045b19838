// Internal launch interface of the embedding kernels (not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace sbk {

struct EmbedArgs {
    void *w[kMaxLanes];           // lane i's rows [V_i][ldw], fp32 or bf16
    int32_t off[kMaxLanes + 1];   // vocab offsets
    int32_t k;
    int32_t V, H, B;
    int64_t ldw;
    bool table_bf16, rows_bf16;   // types of the table and of out / dout
    const int32_t *ids;           // [B]
    float scale;
    // lookup
    void *out;                    // [B][ldo]
    int64_t ldo;
    // gradient
    const void *dout;             // [B][lddo]
    int64_t lddo;
    bool add;                     // added to the table's rows instead of replacing all of them
    int32_t shift;                // 2^shift groups of IDs: ID v is number v >> shift of group
                                  // v % 2^shift
    int32_t range;                // IDs of a group
    int32_t *start;               // [range * 2^shift + 1]: where each ID's positions start in
                                  // `order`, group by group (embed_slot); behind the last
                                  // ID, how many there are
    int32_t *order;               // [B] positions sorted by their IDs' places in `start`,
                                  // those of an ID ascending
    int32_t *sorted;              // [B] their IDs
    float *part;                  // fp32 [pieces][2][ldpart]
    int64_t ldpart;
    int32_t runs;
};

// IDs of up to kEmbedLong positions are summed whole, by the workgroup of the run of
// kEmbedRun sorted positions that they start in; those of more in pieces of kEmbedPiece
// sorted positions, whose sums (`part`) are joined.
constexpr int kEmbedRun = 16, kEmbedLong = 32, kEmbedPiece = 32;

// Whether the gradient's launches fit a grid.
bool embed_grad_fits(int32_t B, int32_t H);

// The groups that a table's IDs are sorted in (2 to this), and the IDs of each.
int embed_shift(int32_t V);
inline int embed_range(int32_t V) { return (int)(((int64_t)V + (1 << embed_shift(V)) - 1) >> embed_shift(V)); }

hipError_t launch_embed(const EmbedArgs &a, hipStream_t s);
hipError_t launch_embed_sort(const EmbedArgs &a, hipStream_t s);
hipError_t launch_embed_sums(const EmbedArgs &a, hipStream_t s);

}  // namespace sbk
