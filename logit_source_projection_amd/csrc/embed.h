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
    int32_t *start;               // [V + 1]: where each ID's positions start in `order`
    int32_t *order;               // [B] positions sorted by their IDs, equal ones ascending
    int32_t *sorted;              // [B] their IDs
    float *part;                  // fp32 [runs][2][ldpart]
    int64_t ldpart;
    int32_t runs;
};

// Sorted positions per run: the rows of a run are summed by one workgroup.
constexpr int kEmbedRun = 64;

hipError_t launch_embed(const EmbedArgs &a, hipStream_t s);
hipError_t launch_embed_sort(const EmbedArgs &a, hipStream_t s);
hipError_t launch_embed_sums(const EmbedArgs &a, hipStream_t s);

}  // namespace sbk
