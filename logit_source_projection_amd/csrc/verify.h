// Internal launch interface of the draft verification kernels (not part of the
// C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sbk {

// Columns of a row that one workgroup takes: for its maximum and sum, and in the draw.
constexpr int kVerifyChunk = 8192, kVerifyDraw = 2048;

// Words between the sequences' counters: a cache line, as the atomics of a line take turns.
constexpr int kVerifyDone = 32;

// What a chunk of a row holds.  Sampled rows: the largest logit (NaN where one is
// NaN or +inf) and the sum of exp((z - that one) / temperature).
// Greedy rows: the best logit and its column.
struct RowPart {
    double sum;
    float most;
    int32_t at;
};

// A row's softmax: its largest logit (NaN or -inf where the row has no distribution), and
// one over the sum of its powers.
struct Softmax {
    double over;
    float most;
};

// What became of a sequence: its accepted drafts, and how the next token is drawn.
struct Verdict {
    Softmax p, q;
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
    int32_t slots;               // rows of a sequence that are looked at: K + 1, with draft logits 2 K + 1
    int32_t chunks, draws;       // of a row, of kVerifyChunk and kVerifyDraw columns
    bool bf16;                   // type of the logits, else fp32
    RowPart *parts;              // [N][slots][chunks]: target rows 0 .. K, draft rows 0 .. K - 1
    Verdict *made;               // [N]
    double *rest;                // [N][draws][2]: sums of what is left of the row, and of p
    uint32_t *done;              // [N][kVerifyDone], the first: how many of `rest` are written
    int32_t *out;                // [N][ldo]
    int64_t ldo;
    int32_t *accepted;           // [N]
};

hipError_t launch_verify(const VerifyArgs &a, hipStream_t s);

}  // namespace sbk
