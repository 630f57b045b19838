/*
 * sb.h -- C ABI of libsb: source projection of a vocab-sharded output head
 * on one AMD Instinct MI355X (gfx950).
 *
 * The head computes logits z = X . W for hidden rows X [B, H] (bf16) and a
 * head weight W [H, V] (bf16) whose vocabulary is split into k contiguous
 * lanes, lane i holding vocab columns [off_i, off_{i+1}).  Three result
 * surfaces are offered, following the SemBridge paper ("SemBridge: Compiling
 * Consumer Observations into Cross-Stack Communication Plans"):
 *
 *  - token-only (sb_project_tokens): section 2.3 and section 5.2 -- a
 *    deterministic token request applies the sampler (argmax) at the source
 *    and ships int32 token IDs; section 6 / Figure 1 -- one result per lane
 *    ("argmax x k"), and all plans deliver the same token ID;
 *  - log-probability (sb_project_logprobs): section 3.2 / 3.4 -- the surface
 *    keeps the complete logits plus token IDs; here the logsumexp per row, the
 *    selected-token log-probability and, on request, the complete fp32
 *    log-probabilities;
 *  - full-logit plan (sb_full_logits): section 5.2 / section 6 -- the logits
 *    are sliced by lane, the shards reconstructed into the complete tensor
 *    (the destination-local AllGather, here a device-local copy), then argmax.
 *
 * Semantics common to every call
 *  - Token IDs are int32 GLOBAL vocabulary indices.  The registered projection
 *    is greedy argmax over the fp32 logits; among equal maxima the LOWEST
 *    global index wins (section 3.1: a projection operator declares
 *    deterministic tie-breaking).
 *  - Logits are fp32 sums of exact bf16 x bf16 products.  The order in which
 *    each logit is accumulated depends only on (B, H, V), never on the
 *    surface, the lane split or the column position, so the three calls
 *    return bit-identical logits and IDs for the same inputs.
 *  - lse is an online sum over 128-column tiles.  A lane's tile grid starts on
 *    the cache line that holds the lane's first column, so lse (and sel_lp and
 *    the complete log-probs) can differ in the last bits between shard
 *    placements that differ modulo 128 bytes; for the same placement it is
 *    reproduced exactly.
 *  - Non-finite values: the argmax puts a NaN above every number (all NaNs
 *    equal, so the lowest-index NaN wins, as numpy's and torch's argmax do)
 *    and +inf above every finite value, so every ID, and every lane's ID, is
 *    one of the row's columns whatever the inputs.  NaN and infinities in x
 *    or w reach the fp32 logits by IEEE rules (NaN * anything and 0 * inf
 *    give NaN).  lse, sel_lp and the complete log-probs of a row holding a
 *    NaN or +inf logit are NaN; of a row of -inf only, unspecified.  Finite
 *    inputs whose sums overflow fp32 are outside the contract
 *    (|logit| < FLT_MAX).
 *
 * Ownership and threading
 *  - The caller allocates every device buffer.  The library allocates no
 *    device memory and is thread-safe.  The only things it keeps between
 *    calls are a per-device note of the kernels whose LDS limit it has
 *    raised (hipFuncSetAttribute, once per device and kernel) and, for
 *    sb_project_tokens_static, each device's address of its static array.
 *  - All work is enqueued asynchronously on `stream` (a hipStream_t; NULL is
 *    the default stream).  Inputs are read-only.  Every device pointer of a
 *    call must be memory the stream's device can access (its own, or a
 *    peer's with peer access enabled); the library does not check this, as
 *    a per-call pointer query would cost more than a decode call's launch.
 *    Outputs must not overlap inputs, the workspace or each other.  A row of
 *    an input may be read up to the end of the 16 bytes that hold its last
 *    value (a row starts at, and its stride is, a multiple of 16); what is
 *    read behind the last value has no effect.
 *  - The workspace is scratch owned by the call until its work completes on
 *    the stream: its contents on entry do not matter, and nothing in it is
 *    valid afterwards.  The workspaces of calls on a head start with the same
 *    fixed region (8,192 bytes) of per-tile counters for heads split into K
 *    slices (see below); a call that counts clears its counters on `stream`
 *    before its head kernel runs (by a small clearing launch, or by the
 *    hidden-row copy for 33 <= B <= 64), so a workspace sized for the
 *    largest call serves calls of any shape, surface or entry point in any
 *    order.  Two calls that use one workspace at the same time (on different
 *    streams without ordering) race and give undefined results.
 *  - A head of fewer than 128 vocabulary tiles of 128 columns (B <= 64) splits
 *    each tile's hidden sum into up to 8 slices that run as separate
 *    workgroups, and one of 257 to 352 tiles (B <= 16, H >= 4065) into 2;
 *    the slice partials are added in slice order.  The split depends on
 *    (B, H, V) only, so the guarantees above still hold.
 *
 * Errors
 *  - Validation is synchronous: on any error status nothing is enqueued and
 *    no output is touched (missing facts select no silent fallback; section
 *    3.4's rule that an unavailable fact selects the materialising plan is
 *    left to the caller, who may call sb_full_logits).
 *  - SB_ERR_HIP reports a failed kernel launch (hipGetLastError); work may
 *    then be partially enqueued.
 */
#ifndef SB_H
#define SB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum sb_status {
    SB_OK = 0,
    SB_ERR_NULL = -1,        /* a required pointer is NULL                     */
    SB_ERR_SHAPE = -2,       /* B < 0, H < 0, V < 1, or a leading dim too small */
    SB_ERR_LANES = -3,       /* k < 1, k > SB_MAX_LANES, or lane offsets not
                                strictly increasing from 0 to V               */
    SB_ERR_ALIGN = -4,       /* x, w[i], an fp32 output or the workspace not
                                16-byte aligned; ldx, ldw not multiples of 8;
                                a logits / log-probs leading dim not a
                                multiple of 4                                  */
    SB_ERR_WORKSPACE = -5,   /* workspace smaller than sb_workspace_bytes()   */
    SB_ERR_UNSUPPORTED = -6, /* V > 2^30; or 40 shard rows or 64 rows of x
                                span 4 GiB or more; or, for 65 <= B <= 128,
                                128 rows of x
                                do; or, for B >= 129, 72 shard rows or 256
                                rows of x do; or a launch of the call would
                                need 2^32 work items or more in one grid
                                dimension (B >= 2^24 always does; for
                                B >= 129 roughly B * V >= 5.5e11)          */
    SB_ERR_HIP = -7,         /* a HIP launch failed                            */
    /* not a status: widens the enumeration to every 32-bit int, so that
       sb_status_string() may be given any value a caller holds */
    SB_STATUS_RANGE_MAX_ = 0x7FFFFFFF
} sb_status;

#define SB_MAX_LANES 64

/* Result surfaces, used to size the workspace. */
typedef enum sb_surface {
    SB_SURF_TOKENS = 0,         /* sb_project_tokens                          */
    SB_SURF_LOGPROBS = 1,       /* sb_project_logprobs, logprobs == NULL      */
    SB_SURF_LOGPROBS_FULL = 2,  /* sb_project_logprobs, logprobs != NULL      */
    SB_SURF_FULL_LOGITS = 3     /* sb_full_logits (includes the lane shards)  */
} sb_surface;

/*
 * The head.  All shapes in elements.
 *   B        rows (decode batch / prefill tokens); B == 0 is a valid no-op
 *   H        hidden size (K of the product); H == 0 gives all-zero logits
 *   V        vocabulary size, >= 1
 *   k        number of vocab lanes, 1..SB_MAX_LANES
 *   lane_off HOST array of k+1 int32: 0 = off_0 < off_1 < ... < off_k = V
 *   x        DEVICE pointer, bf16 [B][ldx] row-major, 16-byte aligned
 *   ldx      row stride of x, >= H, multiple of 8
 *   w        HOST array of k DEVICE pointers; w[i] is lane i's shard, bf16
 *            [H][ldw] row-major, column j of the shard = vocab column
 *            off_i + j; 16-byte aligned.  A single [H][V] allocation is
 *            passed as w[i] = base + off_i with ldw = V (then every off_i
 *            must be a multiple of 8).
 *   ldw      row stride of every shard, >= max_i (off_{i+1} - off_i),
 *            multiple of 8
 */
typedef struct sb_head_desc {
    int32_t B, H, V, k;
    const int32_t *lane_off;
    const void *x;
    int64_t ldx;
    const void *const *w;
    int64_t ldw;
} sb_head_desc;

/*
 * Bytes of device workspace a call on `desc` with the given surface needs
 * (0 if none).  Returns 0 and sets *status (if not NULL) to an error code when
 * the descriptor is invalid.  Host-only; enqueues nothing.
 */
size_t sb_workspace_bytes(const sb_head_desc *desc, int surface, sb_status *status);

/*
 * Token-only surface (source projection, SemBridge section 5.2 / section 6):
 * ids[b] = lowest global index of max_v z[b][v].  Each lane reduces to one
 * (max, lowest-index) result per row inside the GEMM epilogue; the per-lane
 * results are combined in ascending lane order.  The full logits are never
 * written to memory.  Launches: the head kernel, which writes one (max,
 * lowest index) pair per (row, 128-column tile) into the workspace, then a
 * combine kernel (one workgroup per row) that folds them, lane by lane; for
 * 33 <= B <= 64 the head kernel is preceded by a copy of x into the
 * workspace in fragment order, and a head split into K slices by the
 * clearing of its slice counters (done by that copy where there is one).
 *   ids  DEVICE int32 [B]
 *   ws   DEVICE workspace of >= sb_workspace_bytes(desc, SB_SURF_TOKENS)
 *        bytes, 16-byte aligned
 */
sb_status sb_project_tokens(const sb_head_desc *desc, int32_t *ids,
                            void *ws, size_t ws_bytes, void *stream);

/*
 * sb_project_tokens for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same launches and bit-identical ids, with the workspace
 * taken from a static device array inside the library instead of an
 * argument.  The array holds SB_STATIC_SCRATCH_BYTES bytes on every device
 * the library runs on and stays allocated until the process ends; this call
 * allocates nothing.  Its address is looked up once per device, on the first
 * call there.
 *   ids     DEVICE int32 [B]
 *   stream  as for every call; the array used is the one of the stream's
 *           device
 * Returns SB_ERR_WORKSPACE when the call needs more than
 * SB_STATIC_SCRATCH_BYTES of workspace (sb_workspace_bytes(desc,
 * SB_SURF_TOKENS); for example B = 2048 rows at V = 151936 need about 20 MB).
 * Every call on a device shares that device's array and leaves its last
 * contents there: calls on one device whose work overlaps in time (two
 * streams, or two threads, without ordering between them) race and give
 * undefined results.
 */
#define SB_STATIC_SCRATCH_BYTES ((size_t)32 << 20)
sb_status sb_project_tokens_static(const sb_head_desc *desc, int32_t *ids, void *stream);

/*
 * Token surface plus each lane's own result (SemBridge Figure 1 caption and
 * section 5.2: under source projection every lane ships one int32 result per
 * row).  Same launches and same ids as sb_project_tokens; in addition
 *   lane_ids[b][i] = lowest global index of the maximum of z[b][v] over lane
 *                    i's columns (DEVICE int32 [B][k], or NULL)
 *   lane_max[b][i] = that maximum (DEVICE fp32 [B][k], or NULL; -0 is
 *                    reported as +0)
 * ids[b] is lane_ids[b][j] for the first lane j whose lane_max is largest.
 *   ws  >= sb_workspace_bytes(desc, SB_SURF_TOKENS)
 */
sb_status sb_project_lane_results(const sb_head_desc *desc, int32_t *ids,
                                  int32_t *lane_ids, float *lane_max,
                                  void *ws, size_t ws_bytes, void *stream);

/*
 * Log-probability surface (SemBridge section 3.2 / 3.4: complete logits plus
 * token IDs), computed with an online per-lane logsumexp:
 *   ids[b]         as sb_project_tokens (bit-identical)
 *   lse[b]         = log sum_v exp(z[b][v])                       (fp32)
 *   sel_lp[b]      = z[b][ids[b]] - lse[b]   (optional, may be NULL)
 *   logprobs[b][v] = z[b][v] - lse[b]        (optional, may be NULL; fp32
 *                    [B][ldlp], ldlp >= V and a multiple of 4, 16-byte
 *                    aligned)
 *   ws  >= sb_workspace_bytes(desc, logprobs ? SB_SURF_LOGPROBS_FULL
 *                                            : SB_SURF_LOGPROBS)
 */
sb_status sb_project_logprobs(const sb_head_desc *desc, int32_t *ids,
                              float *lse, float *sel_lp, float *logprobs,
                              int64_t ldlp, void *ws, size_t ws_bytes,
                              void *stream);

/*
 * Full-logit plan (SemBridge section 5.2 / section 6, the layout-directed
 * baseline): every lane writes its fp32 logit shard [B][V_i] into the
 * workspace, the shards are reconstructed into logits [B][ldl] (the
 * destination-local AllGather, a device-local copy here), then, if ids is not
 * NULL, a row argmax (lowest index on ties) yields the token IDs.
 *   logits DEVICE fp32 [B][ldl], ldl >= V and a multiple of 4, 16-byte aligned
 *   ids    DEVICE int32 [B] or NULL
 *   ws     >= sb_workspace_bytes(desc, SB_SURF_FULL_LOGITS)
 */
sb_status sb_full_logits(const sb_head_desc *desc, float *logits, int64_t ldl,
                         int32_t *ids, void *ws, size_t ws_bytes, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Partial completion (SemBridge section 6.4, Exact Shards and Partial
 * Completion; section 3.6, reduction obligations).  The MLP down projection is
 * row parallel: lane i holds a distinct activation shard X_i [B][K_i] and the
 * matching weight rows W_i [K_i][N], and produces the incomplete full-width
 * partial P_i = X_i . W_i (fp32 sums of exact bf16 x bf16 products).  The
 * registered elementwise operator completes the partials before the output
 * is exposed:  out = op(...op(op(P_0, P_1), P_2)..., P_{k-1})  (ascending
 * lane order).  Each P_i is accumulated in an order fixed by the shapes
 * alone (1024-row chunks summed in a fixed order), so repeated calls give
 * bit-identical outputs.  SB_RED_MIN and SB_RED_MAX propagate NaN (IEEE
 * 754-2019 minimum and maximum, as numpy's and torch's elementwise ones):
 * an output is NaN when any lane's partial there is NaN.
 * ---------------------------------------------------------------------------
 */
typedef enum sb_reduce_op {
    SB_RED_SUM = 0,
    SB_RED_PROD = 1,
    SB_RED_MIN = 2,
    SB_RED_MAX = 3
} sb_reduce_op;

/*
 *   B       rows (tokens); B == 0 is a valid no-op; the chunked GEMM's
 *           launch of about ceil(K_i / 1024) * ceil(N / 128) * ceil(B / 64)
 *           workgroups of 256 work items, summed over lanes, must hold fewer
 *           than 2^32 work items (else SB_ERR_UNSUPPORTED)
 *   N       output width (the model's hidden size), >= 1
 *   k       lanes, 1..SB_MAX_LANES
 *   lane_k  HOST array of k+1 int32 offsets of the reduction dimension:
 *           0 = lane_k[0] < lane_k[1] < ... < lane_k[k]; K_i = lane_k[i+1] -
 *           lane_k[i]
 *   x       HOST array of k DEVICE pointers; x[i] is bf16 [B][ldx], columns
 *           [0, K_i) used; 16-byte aligned
 *   ldx     row stride of every x[i], >= max K_i, multiple of 8
 *   w       HOST array of k DEVICE pointers; w[i] is bf16 [K_i][ldw], columns
 *           [0, N) used; 16-byte aligned
 *   ldw     row stride of every w[i], >= N, multiple of 8
 */
typedef struct sb_partial_desc {
    int32_t B, N, k;
    const int32_t *lane_k;
    const void *const *x;
    int64_t ldx;
    const void *const *w;
    int64_t ldw;
} sb_partial_desc;

/*
 * Bytes of device workspace sb_partial_complete needs on `desc`: the head
 * calls' fixed counter region, which this call leaves untouched, then the
 * fp32 chunk partials.  0 for B == 0.
 * Returns 0 and sets *status on an invalid descriptor (statuses as for the
 * head; SB_ERR_LANES for bad lane_k).
 */
size_t sb_partial_workspace_bytes(const sb_partial_desc *desc, sb_status *status);

/*
 * out[b][n] = op over lanes (ascending) of P_i[b][n].
 *   op   one of sb_reduce_op (anything else: SB_ERR_SHAPE)
 *   out  DEVICE fp32 [B][ldo], ldo >= N and a multiple of 4, 16-byte aligned
 *   ws   >= sb_partial_workspace_bytes(desc) bytes, 16-byte aligned
 * Two kernel launches: the chunked partial GEMM and the lane reduction.
 */
sb_status sb_partial_complete(const sb_partial_desc *desc, int op, float *out, int64_t ldo,
                              void *ws, size_t ws_bytes, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Training surface: softmax cross entropy over the whole vocabulary and its
 * gradient.  The logits are not kept (few tiles of them split their hidden sum into
 * slices, whose sums pass through the workspace).
 *   lse[b]  = log sum_v exp(z[b][v])
 *   loss[b] = lse[b] - z[b][targets[b]], taken as (max z - z target) + log sum
 *             exp(z - max z): a small loss keeps its digits beside large logits
 *   dz[b][v] = (exp(z[b][v] - lse[b]) - [v == targets[b]]) * dloss[b]
 *   dx = dz . W^T (bf16 [B][lddx]),  dw = x^T . dz (bf16, lane by lane)
 *  - A negative target marks an ignored row (padding): its loss is 0, its row
 *    of dx is 0 wherever W is finite, and it adds nothing to dw, whatever its
 *    x holds.  Its lse is computed like any other, and it costs as much.  A
 *    target >= V makes the row's loss, its row of dx and all of dw NaN.
 *  - Logits are fp32 sums of exact bf16 x bf16 products, and lse an online sum, in
 *    orders fixed by B, H, V and the lane offsets: the same call repeated gives
 *    the same bits, while the same row in another batch size, under another lane
 *    split or in a projection call can differ in the last ones.  The gradient
 *    computes the logits again, in pieces of the vocabulary, rounds dz to bf16
 *    and accumulates dx and dw in fp32; each is rounded once.  Up to 32 rows two
 *    bf16 numbers hold a dz (off by at most 2^-16 of its value); above, the
 *    target's dz is as exact and the others are off by at most 2^-8 of theirs
 *    (in dx above 64 rows their sum by 2^-8 more).
 *  - Non-finite logits follow IEEE rules: a row with a NaN or +inf logit has a
 *    NaN lse; -inf logits count as probability 0, also in a row of nothing else:
 *    its lse is -inf, its loss +inf and its dz -dloss at the target, 0 elsewhere.
 *    Products with a non-finite x or W in dx and dw are NaN where dz is 0.
 * The head descriptor and its limits are the projection calls'.  Also (else
 * SB_ERR_UNSUPPORTED) 256 rows of x must span less than 4 GiB, and so must 64
 * shard rows, 256 of them in the gradient; the gradient of up to 64 rows takes
 * fewer than 2^23 columns, every lane rounded up to 256.  H == 0 gives all-zero
 * logits; the gradients are then empty and the call does nothing.
 * ---------------------------------------------------------------------------
 */

/*
 * Bytes of device workspace of sb_cross_entropy (grad == 0) or
 * sb_cross_entropy_grad (grad != 0); 0 for B == 0.  On an invalid descriptor
 * returns 0 and sets *status (if not NULL).
 */
size_t sb_cross_entropy_workspace_bytes(const sb_head_desc *desc, int grad, sb_status *status);

/*
 *   targets  DEVICE int32 [B]
 *   loss     DEVICE fp32 [B]
 *   lse      DEVICE fp32 [B]
 *   ws       >= sb_cross_entropy_workspace_bytes(desc, 0), 16-byte aligned
 */
sb_status sb_cross_entropy(const sb_head_desc *desc, const int32_t *targets, float *loss, float *lse,
                           void *ws, size_t ws_bytes, void *stream);

/*
 *   targets  DEVICE int32 [B]
 *   lse      DEVICE fp32 [B], as sb_cross_entropy returned it
 *   dloss    DEVICE fp32 [B], the gradient of each row's loss (1 / rows for
 *            a mean)
 *   dx       DEVICE bf16 [B][lddx] or NULL; lddx >= H, a multiple of 8;
 *            16-byte aligned
 *   dw       HOST array of k DEVICE pointers or NULL; dw[i] is lane i's
 *            gradient, bf16 [H][lddw], laid out as w[i]; lddw >= every lane's
 *            width, a multiple of 8; 16-byte aligned
 *   ws       >= sb_cross_entropy_workspace_bytes(desc, 1), 16-byte aligned
 * At least one of dx and dw is required (of gradients that are not empty).
 * Both are overwritten, not added to (B == 0 zeroes dw).  Columns past H in dx and past a lane's width in dw are
 * left as they were.
 */
sb_status sb_cross_entropy_grad(const sb_head_desc *desc, const int32_t *targets, const float *lse,
                                const float *dloss, void *dx, int64_t lddx, void *const *dw,
                                int64_t lddw, void *ws, size_t ws_bytes, void *stream);

/*
 * ---------------------------------------------------------------------------
 * The head in 8-bit integers: rows quantised with one scale each, weights
 * held as one channel per vocabulary column with one scale each.
 *   z[b][v] = (float(sum_h x[b][h] * w[v][h]) * x_scale[b]) * w_scale[v]
 * The integer sums are exact (H <= 131071), so z is the same whatever the
 * batch, the lane split or the call: three fp32 roundings (the sum's, and
 * one for each scale).  sb_int8_project_tokens ranks these fp32 z as the
 * projection calls rank theirs: NaN above every number, the lowest global
 * index among equals.
 *
 * Codes and scales (of a row of x, or of a column of the head weight):
 *   scale = max |value| / 127,  code = rint(value / scale)
 * both in fp32, ties to even, codes in -127 .. 127.  A row or column of zeros
 * has scale 0; one that holds a NaN or an infinity has the scale NaN or
 * infinity, which makes its z NaN; the codes of both are 0.
 * ---------------------------------------------------------------------------
 */

/* Element types of an output. */
typedef enum sb_dtype {
    SB_FP32 = 0,
    SB_BF16 = 1
} sb_dtype;

/*
 *   B, V, k, lane_off   as in sb_head_desc
 *   H        hidden size, <= 131071 (SB_ERR_UNSUPPORTED)
 *   x        DEVICE int8 [B][ldx], 16-byte aligned; -128 is allowed
 *   ldx      row stride of x, >= H, multiple of 16
 *   x_scale  DEVICE fp32 [B]
 *   w        HOST array of k DEVICE pointers; w[i] is lane i's channels,
 *            int8 [V_i][ldw]: row j is vocab column off_i + j; 16-byte
 *            aligned.  A single [V][ldw] allocation is passed as w[i] =
 *            base + off_i * ldw.
 *   ldw      channel stride, >= H, multiple of 16
 *   w_scale  HOST array of k DEVICE pointers; w_scale[i] is fp32 [V_i]
 * 256 rows of x and 256 channels must span less than 4 GiB, and B is below
 * 2^22 (SB_ERR_UNSUPPORTED).  Bytes past H in a row or channel may hold
 * anything.
 */
typedef struct sb_int8_desc {
    int32_t B, H, V, k;
    const int32_t *lane_off;
    const void *x;
    int64_t ldx;
    const float *x_scale;
    const void *const *w;
    int64_t ldw;
    const float *const *w_scale;
} sb_int8_desc;

/*
 * Codes and scales of B rows.
 *   x      DEVICE bf16 [B][ldx], 16-byte aligned, ldx >= H, multiple of 8
 *   q      DEVICE int8 [B][ldq], 16-byte aligned, ldq >= H, multiple of 16;
 *          bytes past H are left as they were
 *   scale  DEVICE fp32 [B]
 */
sb_status sb_int8_quantize_rows(const void *x, int64_t ldx, int32_t B, int32_t H, void *q, int64_t ldq,
                                float *scale, void *stream);

/*
 * Codes and scales of a bf16 head's weight, turned round into channels.  Only
 * the weight fields of `desc` are read (H, V, k, lane_off, w, ldw).
 *   q      HOST array of k DEVICE pointers; q[i] is int8 [V_i][ldq], 16-byte
 *          aligned, ldq >= H, multiple of 16; bytes past H are left as they were
 *   scale  HOST array of k DEVICE pointers; scale[i] is fp32 [V_i]
 */
sb_status sb_int8_quantize_head(const sb_head_desc *desc, void *const *q, int64_t ldq,
                                float *const *scale, void *stream);

/*
 * Bytes of device workspace of sb_int8_project_tokens (SB_SURF_TOKENS) or
 * sb_int8_logits (SB_SURF_FULL_LOGITS; often 0).  On an invalid descriptor or
 * another surface returns 0 and sets *status (if not NULL).
 */
size_t sb_int8_workspace_bytes(const sb_int8_desc *desc, int surface, sb_status *status);

/* ids[b] = lowest global index of max_v z[b][v]  (DEVICE int32 [B]). */
sb_status sb_int8_project_tokens(const sb_int8_desc *desc, int32_t *ids, void *ws, size_t ws_bytes,
                                 void *stream);

/*
 * out[b][v] = z[b][v], rounded once more for SB_BF16.
 *   dtype  sb_dtype of out (anything else: SB_ERR_SHAPE)
 *   out    DEVICE [B][ldo], 16-byte aligned; ldo >= V, a multiple of 4 (fp32)
 *          or 8 (bf16)
 */
sb_status sb_int8_logits(const sb_int8_desc *desc, void *out, int dtype, int64_t ldo, void *ws,
                         size_t ws_bytes, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Layer norm: the step between a model's rows and the head, and its gradient.
 *   mean[b] = sum_h x[b][h] / H
 *   rstd[b] = 1 / sqrt(sum_h (x[b][h] - mean[b])^2 / H + eps)
 *   xh      = (x - mean) * rstd,   y = xh * weight + bias
 *   g = dy * weight,  dx = rstd * (g - sum_h g / H - xh * sum_h (g * xh) / H)
 *   dweight = sum_b dy * xh,   dbias = sum_b dy
 * Sums are fp32, in orders fixed by B, H and the types; every result is rounded
 * once to its type.  NaN and infinities follow IEEE rules: a row of x that holds
 * one is NaN in y, rstd and dx, and makes all of dweight NaN; one in dy leaves
 * nothing finite in its row of dx, and in dweight and dbias stays in its column.
 * Other rows of y and dx are not touched by either.  A row whose values are all
 * the same has y = bias for eps > 0 (rounding of the mean aside) and NaN for
 * eps = 0.  Finite rows whose sums or squares overflow fp32 are outside the
 * contract (values up to 10^15 are safe).
 * ---------------------------------------------------------------------------
 */

/*
 *   B        rows; B == 0 is a valid no-op (it zeroes dweight and dbias)
 *   H        columns, 1 .. 2^24 (SB_ERR_UNSUPPORTED beyond)
 *   x        DEVICE [B][ldx], 16-byte aligned
 *   x_type   sb_dtype of x (anything else: SB_ERR_SHAPE, as for every type)
 *   ldx      row stride of x, >= H, a multiple of 4 (fp32) or 8 (bf16)
 *   weight   DEVICE [H], 16-byte aligned, or NULL (1)
 *   bias     DEVICE [H], 16-byte aligned, or NULL (0)
 *   param_type  sb_dtype of weight and bias, and of their gradients
 *   eps      >= 0 and finite (SB_ERR_SHAPE)
 * Every matrix of these calls spans less than 2^47 bytes (SB_ERR_UNSUPPORTED).
 */
typedef struct sb_norm_desc {
    int32_t B, H;
    const void *x;
    int x_type;
    int64_t ldx;
    const void *weight, *bias;
    int param_type;
    float eps;
} sb_norm_desc;

/*
 *   y       DEVICE [B][ldy], 16-byte aligned; ldy >= H, a multiple of 4 (fp32)
 *           or 8 (bf16); columns past H are left as they were
 *   y_type  sb_dtype of y; any pair of types of x and y
 *   mean, rstd  DEVICE fp32 [B] each, or NULL
 */
sb_status sb_layer_norm(const sb_norm_desc *desc, void *y, int y_type, int64_t ldy, float *mean,
                        float *rstd, void *stream);

/*
 * Bytes of device workspace of sb_layer_norm_grad, for its parameter gradients
 * (a call without them needs none); 0 for few rows.  On an invalid descriptor
 * returns 0 and sets *status (if not NULL).
 */
size_t sb_layer_norm_grad_workspace_bytes(const sb_norm_desc *desc, sb_status *status);

/*
 *   dy       DEVICE [B][lddy], laid out as y, of dy_type (an sb_dtype)
 *   mean, rstd  DEVICE fp32 [B], as sb_layer_norm returned them
 *   dx       DEVICE [B][lddx] of x's type, laid out as x, or NULL; columns past
 *            H are left as they were
 *   dweight, dbias  DEVICE [H] of param_type, 16-byte aligned, or NULL; also
 *            where the weight or bias itself is NULL
 *   ws       >= sb_layer_norm_grad_workspace_bytes(desc), 16-byte aligned;
 *            only with dweight or dbias, and where it is not 0
 * At least one of dx, dweight and dbias is required.  All are overwritten, not
 * added to.
 */
sb_status sb_layer_norm_grad(const sb_norm_desc *desc, const void *dy, int dy_type, int64_t lddy,
                             const float *mean, const float *rstd, void *dx, int64_t lddx,
                             void *dweight, void *dbias, void *ws, size_t ws_bytes, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Embedding: the vocabulary's other table, rows looked up by token IDs and
 * scaled, and the gradient of that lookup.
 *   out[b]    = scale * table[ids[b]]
 *   dtable[v] = scale * sum over b with ids[b] == v of dout[b]
 *  - A negative ID marks padding: its row of out is 0, and it adds nothing to
 *    the gradient, whatever its row of dout holds.  An ID >= V makes the row of
 *    out NaN and adds nothing to the gradient.
 *  - The gradient's sums are fp32 and run over the positions of an ID in
 *    ascending order, in runs that depend on the IDs alone: the same call
 *    repeated gives the same bits.  Each result is rounded once.
 * ---------------------------------------------------------------------------
 */

/*
 *   V        rows of the table, >= 1
 *   H        columns; H == 0 is a valid no-op
 *   k, lane_off  vocabulary lanes, as in sb_head_desc (any offsets)
 *   w        HOST array of k DEVICE pointers; w[i] is lane i's rows, [V_i][ldw]:
 *            row j is vocab row off_i + j; 16-byte aligned.  A single [V][ldw]
 *            allocation is passed as w[i] = base + off_i * ldw.
 *   ldw      row stride, >= H, a multiple of 4 (fp32) or 8 (bf16)
 *   type     sb_dtype of the table (anything else: SB_ERR_SHAPE, as for every type)
 * H <= 2^24 and V <= 2^30; in the gradient H < 2^24 - 256, V <= 2^24, B <= 2^24 and
 * about B * H < 2^37; every matrix of these calls spans less than 2^47 bytes
 * (SB_ERR_UNSUPPORTED).
 */
typedef struct sb_table_desc {
    int32_t V, H, k;
    const int32_t *lane_off;
    void *const *w;
    int64_t ldw;
    int type;
} sb_table_desc;

/*
 *   ids       DEVICE int32 [B]
 *   B         rows; B == 0 is a valid no-op
 *   scale     finite (SB_ERR_SHAPE)
 *   out       DEVICE [B][ldo], 16-byte aligned; ldo >= H, a multiple of 4 (fp32)
 *             or 8 (bf16); columns past H are left as they were
 *   out_type  sb_dtype of out; any pair of types of table and out
 */
sb_status sb_embed(const sb_table_desc *desc, const int32_t *ids, int32_t B, float scale, void *out,
                   int out_type, int64_t ldo, void *stream);

/*
 * Bytes of device workspace of sb_embed_grad on B rows; 0 where the call does
 * nothing.  On an invalid descriptor returns 0 and sets *status (if not NULL).
 */
size_t sb_embed_grad_workspace_bytes(const sb_table_desc *desc, int32_t B, int accumulate, sb_status *status);

/*
 *   desc        the gradient's table, laid out as the table; it is written
 *   ids, B, scale  as in sb_embed
 *   dout        DEVICE [B][lddo], laid out as out, of dout_type (an sb_dtype)
 *   accumulate  0: every row of the gradient is overwritten, with zeros where no
 *               ID names it (B == 0 zeroes all).  Otherwise the sums are added to
 *               the rows that IDs name and the others are not touched.
 *   ws          >= sb_embed_grad_workspace_bytes(desc, B, accumulate), 16-byte
 *               aligned
 * Columns past H are left as they were.
 */
sb_status sb_embed_grad(const sb_table_desc *desc, const int32_t *ids, int32_t B, float scale,
                        const void *dout, int dout_type, int64_t lddo, int accumulate, void *ws,
                        size_t ws_bytes, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Verification of drafted tokens: a draft model (or a lookup) proposes tokens
 * for a sequence, the head computes the logits of all their positions in one
 * batch, and given random numbers decide how many of them the target keeps.
 * For sequence i with n drafts x_0 .. x_(n-1), target logits z_0 .. z_n, draft
 * logits y_0 .. y_(n-1) and temperature t > 0:
 *   p_j = softmax(z_j / t),  q_j = softmax(y_j / t)
 *   draft j is accepted if every one before it is and u_j * q_j(x_j) < p_j(x_j)
 *   the next token is drawn from max(p_j - q_j, 0) of the first rejected draft
 *   j, or from p_n if all are accepted: the lowest column whose cumulative sum
 *   passes u_next times the whole
 * Over uniform random numbers accepted drafts and next token follow the target's
 * distribution, whatever the draft's is.
 *  - Without draft logits a draft counts as certain: q_j(x_j) = 1.
 *  - Where max(p_j - q_j, 0) is 0 everywhere the token is drawn from p_j.
 *  - A temperature that is not > 0 (0, negative, NaN) is greedy: draft j is
 *    accepted if it is the argmax of z_j, and the next token is the argmax (the
 *    projection calls' order: NaN above every number, the lowest index among
 *    equals).  Draft logits and random numbers are not used.
 *  - A logit of -inf is a token that cannot be drawn.  A row that holds a NaN or
 *    +inf logit, or nothing but -inf, has no distribution: as p_j its draft is
 *    rejected and the next token is -1; as q_j its draft is rejected and the
 *    next token is drawn from p_j.
 *  - A drafted token outside 0 .. V - 1 is rejected (without draft logits the
 *    next token is then drawn from p_j).  u_j of 0 accepts any draft with
 *    p_j(x_j) > 0, NaN none; u_next below 0 or NaN counts as 0, and from 1 up
 *    it draws the last token that can be drawn.
 *  - Everything behind the logits is computed in 64 bits, in an order fixed by
 *    V alone: the same logits and numbers give the same tokens in any batch.  An
 *    exponential is within 5 * 10^-14 of itself (below 10^-20: 2 * 10^-13) and
 *    exactly 1 of the largest logit: 2^n equal logits alone have shares of 2^-n.
 *    One below 2^-1074 is 0, as that of -inf.
 * ---------------------------------------------------------------------------
 */

/*
 *   N        sequences; N == 0 is a valid no-op
 *   K        the most drafts of a sequence, >= 0 (0: every call draws one token
 *            per sequence)
 *   V        vocabulary size, 1 .. 2^30 (SB_ERR_UNSUPPORTED beyond)
 *   drafts   drafted tokens of all sequences together
 *   offsets  DEVICE int32 [N + 1]: sequence i's drafts are offsets[i] ..
 *            offsets[i + 1] - 1.  Drafts past the K-th of a sequence are ignored.
 *            Offsets outside 0 .. drafts or falling ones are taken as the nearest
 *            that fit: never read out of range.
 *   tokens   DEVICE int32 [drafts]
 *   target   DEVICE [drafts + N][ldt] logits, 16-byte aligned: sequence i's rows
 *            are offsets[i] + i .. offsets[i + 1] + i, one for each draft and one
 *            behind the last
 *   ldt      row stride, >= V, a multiple of 4 (fp32) or 8 (bf16)
 *   draft    DEVICE [drafts][ldd] logits, laid out as target, or NULL
 *   type     sb_dtype of target and draft (anything else: SB_ERR_SHAPE)
 *   temperature  DEVICE fp32 [N], or NULL (1)
 * N * ceil(V / 2048) and N * (2 K + 1) * ceil(V / 8192) are below 2^24, and every
 * matrix spans less than 2^47 bytes (SB_ERR_UNSUPPORTED).
 */
typedef struct sb_drafts_desc {
    int32_t N, K, V, drafts;
    const int32_t *offsets;
    const int32_t *tokens;
    const void *target;
    int64_t ldt;
    const void *draft;
    int64_t ldd;
    int type;
    const float *temperature;
} sb_drafts_desc;

/*
 * Bytes of device workspace of sb_verify_drafts; 0 for N == 0.  On an invalid
 * descriptor returns 0 and sets *status (if not NULL).
 */
size_t sb_verify_workspace_bytes(const sb_drafts_desc *desc, sb_status *status);

/*
 *   u         DEVICE fp32 [drafts], numbers drawn from [0, 1)
 *   u_next    DEVICE fp32 [N], numbers drawn from [0, 1)
 *   out       DEVICE int32 [N][ldo], ldo >= K + 1: the accepted drafts, the next
 *             token, then -1 up to column K; columns past K are left as they were
 *   accepted  DEVICE int32 [N]: how many drafts are accepted
 *   ws        >= sb_verify_workspace_bytes(desc), 16-byte aligned
 */
sb_status sb_verify_drafts(const sb_drafts_desc *desc, const float *u, const float *u_next, int32_t *out,
                           int64_t ldo, int32_t *accepted, void *ws, size_t ws_bytes, void *stream);

/* Static, NUL-terminated description of a status code. */
const char *sb_status_string(sb_status status);

#ifdef __cplusplus
}
#endif

#endif /* SB_H */
