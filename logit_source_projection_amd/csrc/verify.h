// Internal launch interface of the draft verification kernels (not part of the
// C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sbk {

// Columns of a row that one workgroup takes.
constexpr int kVerifyChunk = 8192;

// What a chunk of a row holds.  Sampled rows: the largest logit (NaN where one is
// NaN or +inf) and the sum of exp((z - largest) / temperature).  Greedy rows: the
// best logit and its column.
struct RowPart {
    double sum;
    float most;
    int32_t at;
};

// What became of a sequence: its accepted drafts, and how its next token is drawn.
struct Decision {
    int32_t accepted, how;
};

struct VerifyArgs {
    const int32_t *offsets;      // [N + 1]
    const int32_t *tokens;       // [drafts]
    const void *target, *draft;  // logits [drafts + N][ldt], [drafts][ldd] or NULL
    int64_t ldt, ldd;
    const float *temperature;    // [N] or NULL
    const float *u, *u_next;     // [drafts], [N]
    int32_t N, K, V, drafts;
    int32_t chunks;
    bool bf16;                   // type of the logits, else fp32
    RowPart *parts;              // [N][2 K + 1][chunks]: target rows 0 .. K, draft rows 0 .. K - 1
    double *rest;                // [N][chunks]: sums of what is left of a row
    Decision *made;              // [N]
    int32_t *out;                // [N][ldo]
    int64_t ldo;
    int32_t *accepted;           // [N]
};

hipError_t launch_verify(const VerifyArgs &a, hipStream_t s);

}  // namespace sbk
