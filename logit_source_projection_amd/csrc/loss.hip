// Softmax cross entropy of the output head and its gradient (gfx950).
//
//   z = X . W            lse_b = log sum_v exp(z_bv)
//   loss_b = lse_b - z_b,t(b)                     (0 where t(b) < 0)
//   dz_bv = (exp(z_bv - lse_b) - [v = t(b)]) g_b  (0 where t(b) < 0)
//   dX = dz . W^T        dW = X^T . dz
//
// The logits are not kept.  The forward pass reduces each tile of them to (maximum,
// sum of exponentials) per row, in the accumulators or, where few tiles split K,
// when the slices' fp32 sums are added up; the backward pass computes them again,
// piece by piece of the vocabulary, writes the piece's dz in bf16 and multiplies
// it both ways.
#include "loss.h"

#include <limits.h>
#include <math.h>

#include <algorithm>

#include "tile_gemm.h"

namespace sbk {
namespace {

static_assert(kVocabBlock == BigTile::kN && kVocabBlock % SmallTile::kN == 0, "no tile spans two blocks");

__device__ __forceinline__ int block_lane(const VocabTable &t, int nb)
{
    int lane = 0;
    while (lane + 1 < t.k && t.blk0[lane + 1] <= nb)
        ++lane;
    return lane;
}

// (m, s) <- the merge of two (maximum, sum exp(z - maximum)) pairs; an empty
// pair is (-inf, 0).  A NaN sum stays NaN.
__device__ __forceinline__ void merge_ms(float &m, float &s, float m2, float s2)
{
    const float top = fmaxf(m, m2);
    const float at = top == -INFINITY ? 0.f : top;
    s = s * __expf(m - at) + s2 * __expf(m2 - at);
    m = top;
}

// Four floats rounded to bf16 (nearest, ties to even) and stored; the first n.
__device__ __forceinline__ void store_bf16x4(uint16_t *p, const float (&v)[4], int n)
{
    bf16x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        h[e] = (__bf16)v[e];
    if (n >= 4) {
        *reinterpret_cast<uint2 *>(p) = __builtin_bit_cast(uint2, h);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n)
                p[e] = __builtin_bit_cast(uint16_t, (__bf16)v[e]);
    }
}

__device__ __forceinline__ float bf16_value(uint16_t bits) { return __uint_as_float((uint32_t)bits << 16); }

// What the rounding of the target's dz v to h took, relative to h, in bf16: h * (1 +
// that) is off by at most 2^-16.  (0 where v is not finite, 0 or below bf16's range.)
__device__ __forceinline__ void store_rest(const LossArgs &a, int64_t b, float v)
{
    const float h = (float)(__bf16)v, r = (v - h) / h;
    a.rest[b * a.ldrest] = __builtin_bit_cast(uint16_t, (__bf16)(fabsf(r) <= 0.0078125f ? r : 0.f));
}
__device__ __forceinline__ float rest_of(const LossArgs &a, int64_t b) { return bf16_value(a.rest[b * a.ldrest]); }

// sum + rest * v, unless that is no number (then v, or the term that the rest was
// taken from, is none either and the sum holds it).
__device__ __forceinline__ float add_rest(float sum, float rest, float v)
{
    const float c = rest * v;
    return fabsf(c) < INFINITY ? sum + c : sum;
}

// lse and loss of a row from its logits' maximum and sum exp(z - maximum).  The
// target's logit is taken from the maximum: what the two leave is exact where they
// are close, while lse - z would round a small loss to the step of a large logit.
// A row of -inf only (no sum) has probability 0 at its target: an infinite loss.
__device__ __forceinline__ void store_loss(const LossArgs &a, int64_t b, float m, float s)
{
    const float logs = logf(s);
    const int t = a.targets[b];
    a.lse[b] = m + logs;
    const float loss = m == -INFINITY && s == 0.f ? INFINITY : m - a.zt[b] + logs;
    a.loss[b] = t < 0 ? 0.f : (t >= a.V ? NAN : loss);
}

// The lse that the gradient's probabilities exp(z - lse) are formed with: a row of
// -inf only has probability 0 everywhere, not exp(-inf + inf).
__device__ __forceinline__ float grad_lse(float lse) { return lse == -INFINITY ? 0.f : lse; }

enum LogitsUse { kUseLoss, kUseGrad };

// Z tile = rows of X times a block of W.
struct LogitsSrc {
    const uint8_t *x, *w;
    int64_t xbytes, wbytes, ldw_bytes;
    int H;
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t a(int st) const
    {
        const int64_t at = (int64_t)st * kStageBytes;
        return buffer_of(x + at, st * kStageK < H ? xbytes - at : 0);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t b(int st) const
    {
        const int64_t at = (int64_t)st * kStageK * ldw_bytes;
        return buffer_of(w + at, wbytes - at);  // rows past H read as zeros
    }
    __device__ __forceinline__ int tail(int st) const { return min((H - st * kStageK) * 2, kStageBytes); }
    __device__ __forceinline__ void meanwhile() const {}
};

// More than 64 rows: a tile of the logits per workgroup, reduced (loss) or
// turned into dz (gradient) in its registers; where tiles are few, K is split
// (loss_slices), the slices' fp32 logits are stored and join_kernel does the rest
// (SPLIT, which only small tiles have, and where USE does not matter).
//
// Bound by MFMA at the clock that power allows: 2048 rows of the dense head (H
// 5120, V 151936) take 2.39 ms (1.33 PFLOP/s), the pieces of a 4096-row gradient
// 1.02 ms each (1.25 PFLOP/s, 252 MB of dz written).  With a short H the ends of
// a tile count: 257 rows of H 1111, V 50257 take 67 us, 18 stages a tile, and half
// the tile rows hold one row.
template <class C, int USE, bool SPLIT>
__global__ __launch_bounds__(C::kThreads, C::kPerCu) void logits_kernel(const LossArgs a, const TileGrid grid)
{
    constexpr int kM = C::kM, kN = C::kN, kWN = C::kWN, kRB = C::kRB, kCB = C::kCB;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tiles = grid.mt * grid.nt, number = xcd_tile(blockIdx.x, SPLIT ? tiles * a.slices : tiles);
    if (number < 0)
        return;
    const int slice = SPLIT ? number / tiles : 0;
    int mt, nt;
    tile_of(grid, number - slice * tiles, mt, nt);
    const int nb = a.nb0 + nt / (kVocabBlock / kN);
    const int lane = block_lane(a.vocab, nb);
    // first column inside the lane (a block's later tiles can lie past it)
    const int c0 = (nb - a.vocab.blk0[lane]) * kVocabBlock + nt % (kVocabBlock / kN) * kN;
    const int nvalid = max(0, min(kN, a.vocab.off[lane + 1] - a.vocab.off[lane] - c0));
    const int m0 = mt * kM;
    const int rows = min(a.B - m0, kM);
    // the slice's part of K: H rows of the weight from k0
    const int k0 = SPLIT ? slice * a.slice_steps * kLossStepK : 0;
    const int H = SPLIT ? min(a.H - k0, a.slice_steps * kLossStepK) : a.H;

    LogitsSrc src;
    src.x = reinterpret_cast<const uint8_t *>(a.x + (int64_t)m0 * a.ldx + k0);
    src.w = reinterpret_cast<const uint8_t *>(a.vocab.w[lane] + (int64_t)k0 * a.ldw + c0);
    src.ldw_bytes = a.ldw * 2;
    src.xbytes = ((int64_t)(rows - 1) * a.ldx + ((a.H + 7) & ~7) - k0) * 2;
    src.wbytes = nvalid > 0 ? ((int64_t)(H - 1) * a.ldw + ((nvalid + 7) & ~7)) * 2 : 0;
    src.H = H;
    WaveTile<C, f32x4> t;
    t.init();
    t.template run<kAlongK, kAcrossK, true, false>(smem, (H + kStageK - 1) / kStageK, a.ldx * 2, a.ldw * 2,
                                          src);

    if (SPLIT) {
        const int64_t ld = (int64_t)a.nblk * kVocabBlock;
        float *p = a.zp + ((int64_t)slice * a.B + m0) * ld + (int64_t)nt * kN + t.col0 + 4 * (t.L >> 4);
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb) {
            const int r = t.row0 + 16 * rb + (t.L & 15);
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb)
                if (r < rows)
                    *reinterpret_cast<f32x4 *>(p + r * ld + 16 * cb) = t.acc[rb][cb];
        }
        return;
    }
    // The epilogue is VALU work that nothing overlaps: 128 values per lane of a
    // big tile.  Ragged blocks and the rows whose target falls among a wave's
    // columns take branches of their own (uniform over the wave), so that the
    // others pay no comparison per value.
    const int n = t.L & 15, g = t.L >> 4;
    const int tcol0 = a.vocab.off[lane] + c0 + t.col0 + 4 * g;  // the lane's first column
    const bool ragged = nvalid < t.col0 + 16 * kCB;
    if (USE == kUseLoss) {
        float2 *part = reinterpret_cast<float2 *>(smem);  // [kM][column waves]
        if (ragged) {
#pragma unroll
            for (int rb = 0; rb < kRB; ++rb)
#pragma unroll
                for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (t.col0 + 16 * cb + 4 * g + e >= nvalid)
                            t.acc[rb][cb][e] = -INFINITY;
        }
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb) {
            const int r = t.row0 + 16 * rb + n;
            // the target's place among the lane's columns 16 cb + e
            const int at = r < rows ? (int)((uint32_t)a.targets[m0 + r] - (uint32_t)tcol0) : -1;
            const bool mine = (uint32_t)at < 16u * kCB && (at & 15) < 4 && t.col0 + 4 * g + at < nvalid;
            if (__builtin_amdgcn_ballot_w64(mine) != 0) {
#pragma unroll
                for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (mine && at == 16 * cb + e)
                            a.zt[m0 + r] = t.acc[rb][cb][e];
            }
            float m = -INFINITY;
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    m = fmaxf(m, t.acc[rb][cb][e]);
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            const float ref = m == -INFINITY ? 0.f : m;
            float s = 0.f;
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s += __expf(t.acc[rb][cb][e] - ref);
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            if (g == 0)
                part[r * kWN + t.wave % kWN] = make_float2(m, s);
        }
        __syncthreads();
        const int r = threadIdx.x;
        if (r < rows) {
            float2 p = part[r * kWN];
#pragma unroll
            for (int w = 1; w < kWN; ++w)
                merge_ms(p.x, p.y, part[r * kWN + w].x, part[r * kWN + w].y);
            a.mse[(int64_t)nt * a.B + m0 + r] = p;
        }
    } else {
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb) {
            const int r = t.row0 + 16 * rb + n;
            const int tgt = r < rows ? a.targets[m0 + r] : -1;
            const float l = r < rows ? grad_lse(a.lse_in[m0 + r]) : 0.f;
            // a target past the vocabulary has no gradient: NaN, not a guess
            const float scale = r >= rows ? 0.f : (tgt >= a.V ? NAN : a.dloss[m0 + r]);
            const uint32_t keep = tgt < 0 ? 0u : 0xFFFFFFFFu;  // ignored rows: 0, whatever z is
            const int at = (int)((uint32_t)tgt - (uint32_t)tcol0);  // its place among the lane's columns
            const bool mine = (uint32_t)at < 16u * kCB;
            const bool plain = !ragged && __builtin_amdgcn_ballot_w64(mine) == 0;
            float term = 0.f;  // the target's dz
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = __expf(t.acc[rb][cb][e] - l);
                if (!plain) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] -= at == 16 * cb + e ? 1.f : 0.f;
                        if (t.col0 + 16 * cb + 4 * g + e >= nvalid)
                            v[e] = 0.f;
                    }
                }
                bf16x4 h;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    h[e] = (__bf16)(v[e] * scale);
                if (!plain) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (at == 16 * cb + e)
                            term = v[e] * scale;
                }
                uint2 bits = __builtin_bit_cast(uint2, h);
                bits.x &= keep;
                bits.y &= keep;
                t.put(smem, rb, cb, bits);
            }
            if (!plain && mine && (at & 15) < 4 && t.col0 + 4 * g + at < nvalid)
                store_rest(a, m0 + r, term);
        }
        uint16_t *const out = a.dz + (int64_t)m0 * a.ldz + (int64_t)nt * kN;
        t.flush(smem, [&](int r, int c, u32x4 v) {
            if (r < rows)
                *reinterpret_cast<u32x4 *>(out + (int64_t)r * a.ldz + c) = v;
        });
    }
}

// One workgroup = 16 rows; thread (row, j) merges parts j, j + 64, ... in
// ascending order, then the 64 runs are merged: 4 in a wave, 16 waves in order.
constexpr int kCombineRows = 16, kCombineRuns = 64;
__global__ __launch_bounds__(kCombineRows * kCombineRuns) void loss_combine_kernel(const LossArgs a)
{
    __shared__ float2 part[kCombineRuns / 4][kCombineRows];
    const int row = threadIdx.x % kCombineRows, run = threadIdx.x / kCombineRows;
    const int64_t b = (int64_t)blockIdx.x * kCombineRows + row;
    float m = -INFINITY, s = 0.f;
    if (b < a.B)
#pragma unroll 4
        for (int i = run; i < a.parts; i += kCombineRuns) {
            const float2 p = a.mse[(int64_t)i * a.B + b];
            merge_ms(m, s, p.x, p.y);
        }
#pragma unroll
    for (int d = 16; d < 64; d <<= 1) {
        const float m2 = __shfl_xor(m, d), s2 = __shfl_xor(s, d);
        merge_ms(m, s, m2, s2);
    }
    if ((threadIdx.x & 63) < kCombineRows)
        part[threadIdx.x >> 6][row] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x >= kCombineRows || b >= a.B)
        return;
#pragma unroll
    for (int w = 1; w < kCombineRuns / 4; ++w)
        merge_ms(m, s, part[w][row].x, part[w][row].y);
    store_loss(a, b, m, s);
}

// ---------------------------------------------------------------------------
// Up to 64 rows: the weight streams from memory once past all of them.  One
// workgroup = 4 waves = 128 columns; wave w takes the K steps w, w + 4, ... of
// its slice (32 rows of W each).  A lane loads 8 rows x 8 columns (16 lanes
// read 256 contiguous bytes of a row) and turns them round in registers: MFMA c
// of a step covers the columns 8 n + c, n = 0 .. 15.  The four partial tiles
// are added in wave order through LDS; K slices, where the tiles alone cannot
// fill the card, are added in slice order by join_kernel.  Neighbouring tiles
// run on one XCD, so that a line that two of them share (rows need not start on
// lines) is fetched into one L2: 8 to 13 % at V 50257, H 4096.
//
// Bound by the weight's bytes: 16 rows of H 4096, V 151936 take 192 us in all
// (6.5 TB/s), one row of H 5120, V 37984 72 us (5.4 TB/s; in one slice
// instead of three 14 us more).
// ---------------------------------------------------------------------------
constexpr int kRowsWaves = 4, kRowsThreads = kRowsWaves * 64;

template <int MB>
struct RowFrags {
    u32x4 w[8], x[MB];
};

// loss: {maximum, sum of exponentials} of n values (the 16 lanes of a row
// hold its columns) and the target's logit.
__device__ __forceinline__ float2 part_of(const float *y, int n, int lanes)
{
    float m = -INFINITY;
    for (int e = 0; e < n; ++e)
        m = fmaxf(m, y[e]);
    for (int d = 1; d < lanes; d <<= 1)
        m = fmaxf(m, __shfl_xor(m, d));
    const float at = m == -INFINITY ? 0.f : m;
    float s = 0.f;
    for (int e = 0; e < n; ++e)
        s += __expf(y[e] - at);
    for (int d = 1; d < lanes; d <<= 1)
        s += __shfl_xor(s, d);
    return make_float2(m, s);
}

// dz of one logit: what its row needs, read once per row.
struct RowGrad {
    float lse, scale;
    int target;
    __device__ __forceinline__ RowGrad(const LossArgs &a, int64_t b)
    {
        target = a.targets[b];
        lse = grad_lse(a.lse_in[b]);
        // a target past the vocabulary has no gradient: NaN, not a guess
        scale = target >= a.V ? NAN : a.dloss[b];
    }
    __device__ __forceinline__ float dz(float z, int col) const
    {
        const float p = __expf(z - lse) - (col == target ? 1.f : 0.f);
        return target < 0 ? 0.f : p * scale;
    }
    // what rounding takes from the target's dz, where it is among the n values v of columns col ..
    template <int N>
    __device__ __forceinline__ void keep_rest(const LossArgs &a, int64_t b, const float (&v)[N], int col,
                                              int n) const
    {
        const uint32_t at = (uint32_t)target - (uint32_t)col;
        if (at >= (uint32_t)min(max(n, 0), N))
            return;
        float term = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e)
            term += at == (uint32_t)e ? v[e] : 0.f;
        store_rest(a, b, term);
    }
};

// dz in bf16, and where lo is not NULL the rest of it too: as the sum of two
// bf16 numbers it is off by at most 2^-16.
template <int N>
__device__ __forceinline__ void store_split(uint16_t *hi, uint16_t *lo, const float (&v)[N])
{
    typedef __bf16 vec __attribute__((ext_vector_type(N)));
    vec h, l;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        h[e] = (__bf16)v[e];
        l[e] = (__bf16)(v[e] - (float)h[e]);
    }
    *reinterpret_cast<vec *>(hi) = h;
    if (lo)
        *reinterpret_cast<vec *>(lo) = l;
}

template <int MB, int USE>
__global__ __launch_bounds__(kRowsThreads, MB == 4 ? 2 : (MB == 2 ? 3 : 4)) void logits_rows_kernel(const LossArgs a)
{
    __shared__ float red[kRowsWaves][16][kLossSmallTile + 4];
    const int number = xcd_tile(blockIdx.x, a.nblk * (kVocabBlock / kLossSmallTile) * a.slices);
    if (number < 0)
        return;
    const int tile = number / a.slices, slice = number - tile * a.slices;
    const int nb = tile / (kVocabBlock / kLossSmallTile);
    const int lane = block_lane(a.vocab, nb);
    const int c0 = (nb - a.vocab.blk0[lane]) * kVocabBlock + tile % (kVocabBlock / kLossSmallTile) * kLossSmallTile;
    const int nvalid = max(0, min(kLossSmallTile, a.vocab.off[lane + 1] - a.vocab.off[lane] - c0));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int L = threadIdx.x & 63, n = L & 15, g = L >> 4;
    const int H = a.H;
    const uint16_t *wbase = a.vocab.w[lane] + c0;
    const int64_t wbytes = H > 0 && nvalid > 0 ? ((int64_t)(H - 1) * a.ldw + ((nvalid + 7) & ~7)) * 2 : 0;
    const int64_t xbytes = H > 0 ? ((int64_t)(a.B - 1) * a.ldx + ((H + 7) & ~7)) * 2 : 0;
    uint32_t wo[8], xo[MB];
#pragma unroll
    for (int r = 0; r < 8; ++r)
        wo[r] = (uint32_t)(((int64_t)(8 * g + r) * a.ldw + 8 * n) * 2);
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
        xo[mb] = (uint32_t)(((int64_t)(16 * mb + n) * a.ldx + 8 * g) * 2);
    f32x4 acc[MB][8];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int c = 0; c < 8; ++c)
            acc[mb][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int steps = (H + kLossStepK - 1) / kLossStepK;
    const int s0 = slice * a.slice_steps, s1 = min(s0 + a.slice_steps, steps);
    auto load = [&](RowFrags<MB> &f, int st) {  // (at or past s1: zeros)
        const int64_t wat = (int64_t)st * kLossStepK * a.ldw * 2, xat = (int64_t)st * kLossStepK * 2;
        const __amdgpu_buffer_rsrc_t rw =
            buffer_of(reinterpret_cast<const uint8_t *>(wbase) + wat, st < s1 ? wbytes - wat : 0);
        const __amdgpu_buffer_rsrc_t rx =
            buffer_of(reinterpret_cast<const uint8_t *>(a.x) + xat, st < s1 ? xbytes - xat : 0);
#pragma unroll
        for (int r = 0; r < 8; ++r)  // non-temporal: the launch reads each weight byte once
            f.w[r] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, wo[r], 0, 2));
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
            f.x[mb] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, xo[mb], 0, 0));
    };
    auto mma = [&](RowFrags<MB> &f, int st) {
        if (__builtin_expect(st * kLossStepK + kLossStepK > H, 0)) {
            // values of x at and past H: a row's padding, or the next row
            const int left = H - st * kLossStepK - 8 * g;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    f.x[mb][d] &= (left > 2 * d ? 0x0000FFFFu : 0u) | (left > 2 * d + 1 ? 0xFFFF0000u : 0u);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            u32x4 col;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                col[q] = __builtin_amdgcn_perm(f.w[2 * q + 1][c >> 1], f.w[2 * q][c >> 1],
                                               c & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                acc[mb][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, f.x[mb]), __builtin_bit_cast(bf16x8, col), acc[mb][c], 0, 0, 0);
        }
    };
    RowFrags<MB> fa, fb;
    load(fa, s0 + wave);
    for (int st = s0 + wave; st < s1; st += 2 * kRowsWaves) {
        load(fb, st + kRowsWaves);
        mma(fa, st);
        load(fa, st + 2 * kRowsWaves);
        mma(fb, st + kRowsWaves);
    }

    // thread: row threadIdx.x / 16 of a block, columns 8 * (threadIdx.x % 16) ..
    const int er = threadIdx.x >> 4, ec = 8 * (threadIdx.x & 15);
    const int gcol = a.vocab.off[lane] + c0 + ec;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        if (16 * mb >= a.B)
            break;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            *reinterpret_cast<f32x4 *>(&red[wave][4 * g + r][8 * n]) =
                f32x4{acc[mb][0][r], acc[mb][1][r], acc[mb][2][r], acc[mb][3][r]};
            *reinterpret_cast<f32x4 *>(&red[wave][4 * g + r][8 * n + 4]) =
                f32x4{acc[mb][4][r], acc[mb][5][r], acc[mb][6][r], acc[mb][7][r]};
        }
        __syncthreads();
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            f32x4 s = *reinterpret_cast<const f32x4 *>(&red[0][er][ec + e]);
#pragma unroll
            for (int w = 1; w < kRowsWaves; ++w)
                s += *reinterpret_cast<const f32x4 *>(&red[w][er][ec + e]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[e + i] = s[i];
        }
        const int b = 16 * mb + er;
        if (a.slices > 1) {
            if (b < a.B) {
                float *p = a.zp + ((int64_t)slice * a.B + b) * ((int64_t)a.nblk * kVocabBlock) +
                           (int64_t)tile * kLossSmallTile + ec;
                *reinterpret_cast<f32x4 *>(p) = f32x4{y[0], y[1], y[2], y[3]};
                *reinterpret_cast<f32x4 *>(p + 4) = f32x4{y[4], y[5], y[6], y[7]};
            }
            continue;
        }
        if (USE == kUseLoss) {
            const int tgt = b < a.B ? a.targets[b] : -1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (ec + e >= nvalid)
                    y[e] = -INFINITY;
                else if (gcol + e == tgt)
                    a.zt[b] = y[e];
            }
            const float2 p = part_of(y, 8, 16);
            if (ec == 0 && b < a.B)
                a.mse[(int64_t)b * a.parts + tile] = p;
        } else if (b < a.B) {
            const RowGrad row(a, b);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = ec + e < nvalid ? row.dz(y[e], gcol + e) : 0.f;
            uint16_t *p = a.dz + (int64_t)b * a.ldz + (int64_t)tile * kLossSmallTile + ec;
            store_split(p, dz_parts(a.B) > 1 ? p + (int64_t)a.B * a.ldz : nullptr, v);
            if (MB == 4)  // one part
                row.keep_rest(a, b, v, gcol, nvalid - ec);
        }
    }
}

// The slices of the logits added up: one workgroup = kLossChunk columns of a row.
template <int USE>
__global__ __launch_bounds__(256) void join_kernel(const LossArgs a)
{
    __shared__ float2 part[4];
    const int b = blockIdx.y;
    const int64_t ld = (int64_t)a.nblk * kVocabBlock;
    const int64_t col = (int64_t)blockIdx.x * kLossChunk + 4 * threadIdx.x;
    float y[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (col < ld) {
        const int nb = (int)(col / kVocabBlock);
        const int lane = block_lane(a.vocab, nb);
        const int c = (nb - a.vocab.blk0[lane]) * kVocabBlock + (int)(col % kVocabBlock);
        const int left = a.vocab.off[lane + 1] - a.vocab.off[lane] - c;
        const int gcol = a.vocab.off[lane] + c;
        const float *p = a.zp + (int64_t)b * ld + col;
        f32x4 s = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll 4
        for (int i = 1; i < a.slices; ++i)
            s += *reinterpret_cast<const f32x4 *>(p + (int64_t)i * a.B * ld);
        if (USE == kUseLoss) {
            const int tgt = a.targets[b];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left) {
                    y[e] = s[e];
                    if (gcol + e == tgt)
                        a.zt[b] = s[e];
                }
        } else {
            const RowGrad row(a, b);
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = e < left ? row.dz(s[e], gcol + e) : 0.f;
            uint16_t *q = a.dz + (int64_t)b * a.ldz + col;
            store_split(q, dz_parts(a.B) > 1 ? q + (int64_t)a.B * a.ldz : nullptr, v);
            if (dz_parts(a.B) == 1)
                row.keep_rest(a, b, v, gcol, left);
        }
    }
    if (USE == kUseLoss) {
        float2 p = part_of(y, 4, 64);
        if ((threadIdx.x & 63) == 0)
            part[threadIdx.x >> 6] = p;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < 4; ++w)
                merge_ms(p.x, p.y, part[w].x, part[w].y);
            a.mse[(int64_t)b * a.parts + blockIdx.x] = p;
        }
    }
}

// Few rows or K slices: one workgroup per row, its parts spread over the threads.
__global__ __launch_bounds__(256) void loss_rows_combine_kernel(const LossArgs a)
{
    __shared__ float2 part[4];
    const int b = blockIdx.x;
    float m = -INFINITY, s = 0.f;
    for (int i = threadIdx.x; i < a.parts; i += 256) {
        const float2 p = a.mse[(int64_t)b * a.parts + i];
        merge_ms(m, s, p.x, p.y);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const float m2 = __shfl_xor(m, d), s2 = __shfl_xor(s, d);
        merge_ms(m, s, m2, s2);
    }
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x != 0)
        return;
    for (int w = 1; w < 4; ++w)
        merge_ms(m, s, part[w].x, part[w].y);
    store_loss(a, b, m, s);
}

// Copies x in 16-byte units, the rows of negative targets as zeros: an
// ignored row adds nothing to dw whatever its x holds (0 * NaN would).
__global__ __launch_bounds__(256) void mask_rows_kernel(const LossArgs a, uint16_t *xm)
{
    const int64_t units = a.ldxm / 8;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t b = at / units, u = at - b * units;
    if (b >= a.B)
        return;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (a.targets[b] >= 0)
        v = *reinterpret_cast<const u32x4 *>(a.x + b * a.ldx + 8 * u);
    *reinterpret_cast<u32x4 *>(xm + b * a.ldxm + 8 * u) = v;
}

// dX tile = rows of dz times the block columns of W rows (k = vocabulary).
template <typename Meanwhile>
struct DxSrc {
    const LossArgs &args;
    const uint8_t *dz;    // the tile's rows, from the split's first block on
    int64_t dzbytes;
    int nb_first, nb_end; // the split's blocks
    int h0, hrows;
    // the lane that holds the stage being loaded
    int lane, lane_end;
    // valid K bytes of the last two stages loaded
    int tail0, tail1;
    Meanwhile meanwhile;
    __device__ __forceinline__ DxSrc(const LossArgs &a_, Meanwhile m) : args(a_), meanwhile(m) {}
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t a(int st) const
    {
        const int64_t at = (int64_t)st * kStageBytes;
        return buffer_of(dz + at, st < (nb_end - nb_first) * (kVocabBlock / kStageK) ? dzbytes - at : 0);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t b(int st)
    {
        const int nb = nb_first + st / (kVocabBlock / kStageK);
        if (nb >= nb_end)
            return buffer_of(args.vocab.w[lane], 0);
        while (nb >= lane_end) {
            ++lane;
            lane_end = args.vocab.blk0[lane + 1];
        }
        const int c = (nb - args.vocab.blk0[lane]) * kVocabBlock + st % (kVocabBlock / kStageK) * kStageK;
        const int width = args.vocab.off[lane + 1] - args.vocab.off[lane];
        const int cols = max(0, min(kStageK, width - c));
        (st & 1 ? tail1 : tail0) = cols * 2;
        const int64_t first = (int64_t)h0 * args.ldw + c;
        return buffer_of(args.vocab.w[lane] + first,
                         cols > 0 ? ((int64_t)(hrows - 1) * args.ldw + ((cols + 7) & ~7)) * 2 : 0);
    }
    __device__ __forceinline__ int tail(int st) const { return st & 1 ? tail1 : tail0; }
};

// The rows whose target is one of n columns from col on, up to 64 of them in ascending
// order, one to a lane; next is the first row not looked at.
struct TargetRows {
    static constexpr int kAhead = 8;  // loads in flight, 64 rows each
    int col, n;
    int row, count, next;
    int at;  // the target's place among the columns
    int t[kAhead];
    // Targets of rows next ..  No lane branches: the ballots below need all of them,
    // and a branch here was merged into their loop.
    __device__ __forceinline__ void load(const LossArgs &a)
    {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int b = next + 64 * j + (threadIdx.x & 63), v = a.targets[min(b, a.B - 1)];
            t[j] = b < a.B ? v : -1;
        }
    }
    // (after load)
    __device__ __forceinline__ void find(const LossArgs &a)
    {
        const int L = threadIdx.x & 63;
        count = 0;
        for (;;) {
            int done = 64 * kAhead;  // rows of the loaded ones that are looked at
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const uint32_t c = (uint32_t)t[j] - (uint32_t)col;
                uint64_t hits = __builtin_amdgcn_ballot_w64(c < (uint32_t)n);
                if (__builtin_expect(hits == 0 || done < 64 * kAhead, 1))
                    continue;
                if (count + __builtin_popcountll(hits) > 64) {
                    done = 64 * j;
                    continue;
                }
                for (; hits != 0; hits &= hits - 1, ++count) {
                    const int l = __builtin_ctzll(hits), hit = __builtin_amdgcn_readlane((int)c, l);
                    if (L == count) {
                        row = next + 64 * j + l;
                        at = hit;
                    }
                }
            }
            next += done;
            if (next >= a.B || done < 64 * kAhead)
                return;
            load(a);
        }
    }
};

// dW tile = X^T rows times a block of dz (k = batch rows).
template <typename Meanwhile>
struct DwSrc {
    const uint8_t *x, *dz;
    int64_t xbytes, zbytes, ldx_bytes, ldz_bytes;
    Meanwhile meanwhile;
    __device__ __forceinline__ DwSrc(Meanwhile m) : meanwhile(m) {}
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t a(int st) const
    {
        const int64_t at = (int64_t)st * kStageK * ldx_bytes;
        return buffer_of(x + at, xbytes - at);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t b(int st) const
    {
        const int64_t at = (int64_t)st * kStageK * ldz_bytes;
        return buffer_of(dz + at, zbytes - at);
    }
    __device__ __forceinline__ int tail(int) const { return kStageBytes; }
};

// The two products of a piece share one launch: dX has few tiles with a long
// K (the piece's columns), dW many with a short one (the rows), and each has
// half the work, so the dX tiles go first and the dW tiles fill the CUs that
// are left over.  Bound by MFMA: a piece of 4096 rows, H 5120 and 30464 columns
// takes 2.0 ms (1.28 PFLOP/s; one XCD with a few long dX tiles more than the
// others made it 2.76).  The targets' rests (see dz_parts) are 1 to 2 % of it.
template <class C>
__global__ __launch_bounds__(C::kThreads, C::kPerCu) void grad_kernel(const LossArgs a, const TileGrid gx,
                                                                      const int dx_ids, const TileGrid gw)
{
    constexpr int kM = C::kM, kN = C::kN, kRB = C::kRB, kCB = C::kCB;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int n = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    WaveTile<C, f32x4> t;
    int mt, nt;
    if ((int)blockIdx.x < dx_ids) {
        const int tiles = gx.mt * gx.nt;
        const int number = xcd_tile(blockIdx.x, tiles * a.splits);
        if (number < 0)
            return;
        const int split = number / tiles;
        tile_of(gx, number - split * tiles, mt, nt);
        const int per = (a.nblk + a.splits - 1) / a.splits;
        const int b0 = min(split * per, a.nblk), b1 = min(b0 + per, a.nblk);
        const int m0 = mt * kM, rows = min(a.B - m0, kM);
        // the last piece's launch makes the targets' terms whole (see dz_parts)
        int target[kRB];
        uint16_t rest[kRB];
        auto meanwhile = [&]() {
#pragma unroll
            for (int rb = 0; rb < kRB; ++rb) {
                const int64_t b = m0 + min(t.row0 + 16 * rb + n, rows - 1);
                target[rb] = a.targets[b];
                rest[rb] = a.rest[b * a.ldrest];
            }
        };
        DxSrc<decltype(meanwhile)> src(a, meanwhile);
        src.dz = reinterpret_cast<const uint8_t *>(a.dz + (int64_t)m0 * a.ldz + (int64_t)b0 * kVocabBlock);
        src.dzbytes = ((int64_t)(rows - 1) * a.ldz + (int64_t)(b1 - b0) * kVocabBlock) * 2;
        src.nb_first = a.nb0 + b0;
        src.nb_end = a.nb0 + b1;
        src.h0 = nt * kN;
        src.hrows = min(a.H - src.h0, kN);
        src.lane = block_lane(a.vocab, src.nb_first);
        src.lane_end = a.vocab.blk0[src.lane + 1];
        src.tail0 = src.tail1 = kStageBytes;
        t.init();
        t.template run<kAlongK, kAlongK, false, true>(smem, (b1 - b0) * (kVocabBlock / kStageK), a.ldz * 2,
                                             a.ldw * 2, src);
        if (b1 == b0)  // (an empty split has not run)
            meanwhile();
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb) {
            const int r = t.row0 + 16 * rb + n;
            if (r >= rows)
                continue;
            const float whole = a.last && (uint32_t)target[rb] < (uint32_t)a.V ? 1.f + bf16_value(rest[rb]) : 1.f;
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb) {
                const int c = src.h0 + t.col0 + 16 * cb + 4 * g;
                if (c >= a.H)
                    continue;
                if (a.dxp) {
                    f32x4 *p = reinterpret_cast<f32x4 *>(
                        a.dxp + ((int64_t)split * a.B + m0 + r) * a.ldxp + c);
                    const f32x4 sum = a.first ? t.acc[rb][cb] : *p + t.acc[rb][cb];
                    *p = sum * whole;
                } else {
                    const f32x4 sum = t.acc[rb][cb] * whole;
                    const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
                    store_bf16x4(a.dx + (int64_t)(m0 + r) * a.lddx + c, v, a.H - c);
                }
            }
        }
        return;
    }
    const int number = xcd_tile(blockIdx.x - dx_ids, gw.mt * gw.nt);
    if (number < 0)
        return;
    tile_of(gw, number, mt, nt);
    const int nb = a.nb0 + nt / (kVocabBlock / kN);
    const int lane = block_lane(a.vocab, nb);
    const int c0 = (nb - a.vocab.blk0[lane]) * kVocabBlock + nt % (kVocabBlock / kN) * kN;
    const int nvalid = min(kN, a.vocab.off[lane + 1] - a.vocab.off[lane] - c0);
    if (nvalid <= 0)
        return;
    const int h0 = mt * kM, hrows = min(a.H - h0, kM);
    t.init();
    // What rounding took from the dz of the targets among the wave's columns, times
    // their rows of x, goes on top of the product, four rows at a time: a step of MFMAs
    // whose k = 8 g is the list's row i + g and whose other k are zeros.  The rows are
    // found, and the first four's x fetched, while the tile's first stages are on
    // their way; each next four's are fetched ahead.
    TargetRows hits;
    hits.col = a.vocab.off[lane] + c0 + t.col0;
    hits.n = max(0, min(16 * kCB, nvalid - t.col0));
    hits.next = hits.count = hits.row = hits.at = 0;
    uint16_t high = 0, rest = 0;  // of lane i's row: its dz and what rounding took, relative to it
    uint16_t ahead[kRB];          // x of the next four rows
    auto fetch = [&](int i) {
        const uint16_t *row = a.xm + (int64_t)__shfl(hits.row, i + g) * a.ldxm + h0;
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb)
            ahead[rb] = row[min(t.row0 + 16 * rb + n, hrows - 1)];
    };
    auto find = [&]() {
        hits.find(a);
        high = a.dz[(int64_t)hits.row * a.ldz + (int64_t)nt * kN + t.col0 + hits.at];
        rest = a.rest[hits.row * a.ldrest];
        if (hits.count > 0)
            fetch(0);
    };
    if (a.B > 0)
        hits.load(a);
    DwSrc<decltype(find)> src(find);
    src.x = reinterpret_cast<const uint8_t *>(a.xm + h0);
    src.dz = reinterpret_cast<const uint8_t *>(a.dz + (int64_t)nt * kN);
    src.ldx_bytes = a.ldxm * 2;
    src.ldz_bytes = a.ldz * 2;
    src.xbytes = ((int64_t)(a.B - 1) * a.ldxm + ((hrows + 7) & ~7)) * 2;
    src.zbytes = ((int64_t)(a.B - 1) * a.ldz + kN) * 2;
    t.template run<kAcrossK, kAcrossK, false, false>(smem, (a.B + kStageK - 1) / kStageK, a.ldxm * 2,
                                            a.ldz * 2, src);
    while (hits.count > 0) {
        const float took = bf16_value(high) * bf16_value(rest);  // (NaN of an infinite dz)
        const int left = __builtin_bit_cast(uint16_t, (__bf16)(fabsf(took) < INFINITY ? took : 0.f));
        for (int i = 0; i < hits.count; i += 4) {
            const bool ok = i + g < hits.count;
            const int at = __shfl(hits.at, i + g), z = __shfl(left, i + g);
            uint32_t x[kRB];
#pragma unroll
            for (int rb = 0; rb < kRB; ++rb)
                x[rb] = ok ? ahead[rb] : 0u;
            fetch(min(i + 4, 60));
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb) {
                const u32x4 zf = {ok && at == 16 * cb + n ? (uint32_t)z : 0u, 0u, 0u, 0u};
#pragma unroll
                for (int rb = 0; rb < kRB; ++rb)
                    block_mma(t.acc[rb][cb], u32x4{x[rb], 0u, 0u, 0u}, zf);
            }
        }
        if (hits.next >= a.B)
            break;
        hits.load(a);
        find();
    }
#pragma unroll
    for (int rb = 0; rb < kRB; ++rb)
#pragma unroll
        for (int cb = 0; cb < kCB; ++cb) {
            bf16x4 h;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                h[e] = (__bf16)t.acc[rb][cb][e];
            t.put(smem, rb, cb, __builtin_bit_cast(uint2, h));
        }
    uint16_t *const out = a.vocab.dw[lane] + (int64_t)h0 * a.lddw + c0;
    t.flush(smem, [&](int r, int c, u32x4 v) {
        if (r >= hrows || c >= nvalid)
            return;
        uint16_t *p = out + (int64_t)r * a.lddw + c;
        if (c + 8 <= nvalid) {
            *reinterpret_cast<u32x4 *>(p) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < nvalid)
                    p[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
    });
}

// ---------------------------------------------------------------------------
// Up to 64 rows: dX and dW in one pass over the weight, which both are bound
// by (W is read, dW written).  A workgroup has 64 rows h of W and a run of
// 64-column steps, which its waves take in turn, so that the lines of W and dW
// that straddle two steps (row strides need not be multiples of a line) are
// read and written by neighbours at the same time.  At 16 rows, H 5120, V 37984
// (rows of 593.5 lines) the whole gradient took 365 us with 256 rows and one
// step at a time per workgroup, 330 us with two steps, 296 us with four.
// A wave streams its tiles of W and of dz through a private LDS ring of whole
// lines and shares nothing.  dz's tile is [rows][64 columns]: rows b of its
// high part, then (up to 32 rows) of its low part.
//   dX[b][h] += sum_v W[h][v] dz[b][v]   (k = columns, along both)
//   dW[h][v]  = sum_b x[b][h] dz[b][v]   (k = dz rows, read across)
// There it reads and writes 838 MB in 200 us (4.2 TB/s; a copy runs at 4.85).
// ---------------------------------------------------------------------------
constexpr int kFewH = 64, kFewSlots = 2, kFewStep = 64;
constexpr int kFewWaves = 4, kFewThreads = kFewWaves * 64;
constexpr int kFewWBytes = kFewH * kFewStep * 2;  // a step's tile of W

template <int MB>
struct FewShape {
    static constexpr int kBp = 16 * MB;                        // rows b, padded
    static constexpr int kRows = dz_parts(kBp) * kBp;          // dz rows: 32, 64 or 64
    static constexpr int kSlot = kFewWBytes + kRows * kFewStep * 2;
    static constexpr int kLds = kFewWaves * kFewSlots * kSlot;
};

// A step's columns: its lane, the first column there and how many.
struct Cols {
    int lane, c, n;
};

template <int MB>
__global__ __launch_bounds__(kFewThreads, 1) void grad_rows_kernel(const LossArgs a, const int htiles,
                                                                                const int per, const int want_dx,
                                                                                const int want_dw)
{
    // the shape as local constants (usable in device code as values)
    constexpr int kBp = FewShape<MB>::kBp, kRows = FewShape<MB>::kRows, kSlot = FewShape<MB>::kSlot;
    constexpr int kParts = kRows / kBp;
    constexpr int kKc = kRows / 32;          // 32-row K steps of dW
    constexpr int kXc = MB == 4 ? 2 : 1;     // of which x has this many of its own
    constexpr int kZ = kRows / 8;            // loads of dz per step (8 rows each)
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int split = blockIdx.x / htiles, hw = (blockIdx.x - split * htiles) * kFewH;
    const int steps = a.nblk * (kVocabBlock / kFewStep);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int L = threadIdx.x & 63, n = L & 15, g = L >> 4;
    // the wave's steps: s0, s0 + kFewWaves, ... below s1
    const int s0 = min(split * per, steps) + wave, s1 = min((split + 1) * per, steps);
    const int hrows = min(kFewH, a.H - hw);
    uint8_t *const ring = smem + wave * (kFewSlots * kSlot);

    // x's fragments: lane holds x[b][h] of h = 16 hb + n, b = 8 g .. 8 g + 7 of
    // each 32 dz rows; ignored rows, and rows past B or H, are zeros
    u32x4 xf[4][kXc];
    if (want_dw) {
        const __amdgpu_buffer_rsrc_t rt = buffer_of(a.targets, (int64_t)a.B * 4);
        const __amdgpu_buffer_rsrc_t rx =
            buffer_of(a.x, ((int64_t)(a.B - 1) * a.ldx + ((a.H + 7) & ~7)) * 2);
        int tgt[kXc][8];
#pragma unroll
        for (int kc = 0; kc < kXc; ++kc)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                tgt[kc][j] = (int)__builtin_amdgcn_raw_buffer_load_b32(
                    rt, 4 * ((32 * kc + 8 * g + j) % kBp), 0, 0);
#pragma unroll
        for (int kc = 0; kc < kXc; ++kc)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int b = (32 * kc + 8 * g + j) % kBp;
#pragma unroll
                for (int hb = 0; hb < 4; ++hb) {
                    const int h = hw + 16 * hb + n;
                    // past the buffer's end where the value is to be zero
                    const uint32_t at = b < a.B && tgt[kc][j] >= 0 && h < a.H
                                            ? (uint32_t)(((int64_t)b * a.ldx + h) * 2) : 0xFFFFFFF0u;
                    const uint32_t v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rx, at, 0, 0);
                    if (j & 1)
                        xf[hb][kc][j >> 1] |= v << 16;
                    else
                        xf[hb][kc][j >> 1] = v;
                }
            }
    }

    uint32_t wo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 8 * i + (L >> 3);
        wo[i] = (uint32_t)((int64_t)r * a.ldw * 2 + 16 * ((L & 7) ^ ((r >> 1) & 7)));
    }
    uint32_t zo[kZ];
#pragma unroll
    for (int i = 0; i < kZ; ++i) {
        const int r = 8 * i + (L >> 3);
        zo[i] = (uint32_t)((int64_t)(r % kBp) * a.ldz * 2 + 16 * ((L & 7) ^ ((r >> 1) & 7)));
    }
    int lane = block_lane(a.vocab, min(s0, steps - 1) / (kVocabBlock / kFewStep));
    int lane_end = a.vocab.blk0[lane + 1];
    auto cols_of = [&](int st) {
        const int nb = st / (kVocabBlock / kFewStep);
        while (nb >= lane_end) {
            ++lane;
            lane_end = a.vocab.blk0[lane + 1];
        }
        const int c = (nb - a.vocab.blk0[lane]) * kVocabBlock + st % (kVocabBlock / kFewStep) * kFewStep;
        return Cols{lane, c, max(0, min(kFewStep, a.vocab.off[lane + 1] - a.vocab.off[lane] - c))};
    };
    // of row L, where its dz is in one part: its target, and what rounding took from its
    // dz there (relative to that)
    int target = -1;
    float rest = 0.f;
    if (kParts == 1) {
        const int b = min(L, a.B - 1), v = a.targets[b];
        target = L < a.B ? v : -1;
        rest = rest_of(a, b);
    }
    const int64_t zplane = (int64_t)a.B * a.ldz;
    const int64_t zbytes = ((int64_t)(a.B - 1) * a.ldz + kFewStep) * 2;
    auto load = [&](int slot, int st) -> Cols {  // (at or past s1: zeros)
        Cols k = {lane, 0, 0};
        if (st < s1)
            k = cols_of(st);
        uint8_t *const to = ring + slot * kSlot;
        if (want_dx) {
            const __amdgpu_buffer_rsrc_t rw =
                buffer_of(a.vocab.w[k.lane] + (int64_t)hw * a.ldw + k.c,
                          k.n > 0 ? ((int64_t)(hrows - 1) * a.ldw + ((k.n + 7) & ~7)) * 2 : 0);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                load_to_lds(to + i * 1024, rw, wo[i]);
        }
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
            const __amdgpu_buffer_rsrc_t rz =
                buffer_of(a.dz + part * zplane + (int64_t)st * kFewStep, st < s1 ? zbytes : 0);
#pragma unroll
            for (int i = part * (kZ / kParts); i < (part + 1) * (kZ / kParts); ++i)
                load_to_lds(to + kFewWBytes + i * 1024, rz, zo[i]);
        }
        return k;
    };

    f32x4 dxa[4][MB];
#pragma unroll
    for (int hb = 0; hb < 4; ++hb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
            dxa[hb][mb] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint32_t fo = (uint32_t)(n * 128 + ((g ^ ((n >> 1) & 7)) * 16));  // row n, piece g
    Cols cur = load(0, s0), next = load(1, s0 + kFewWaves);
    // The wave's last memory operations are the next step's loads (kZ of dz, 8
    // of W) and then kW stores of dw, where the last step stored whole tiles;
    // a ragged one may have stored more or fewer, and counts as none.
    constexpr int kW = 8;
    bool stored = false;
    int slot = 0;
    for (int st = s0; st < s1; st += kFewWaves, slot ^= 1) {
        // this step's tiles have landed (the next step's loads stay in flight)
        asm volatile("" ::: "memory");
        if (want_dx) {
            if (stored)
                __builtin_amdgcn_s_waitcnt(vmcnt_only(kZ + 8 + kW));
            else
                __builtin_amdgcn_s_waitcnt(vmcnt_only(kZ + 8));
        } else if (stored) {
            __builtin_amdgcn_s_waitcnt(vmcnt_only(kZ + kW));
        } else {
            __builtin_amdgcn_s_waitcnt(vmcnt_only(kZ));
        }
        asm volatile("" ::: "memory");
        const uint8_t *wt = ring + slot * kSlot, *zt = wt + kFewWBytes;
        f32x4 dwa[4][4];
#pragma unroll
        for (int hb = 0; hb < 4; ++hb)
#pragma unroll
            for (int vb = 0; vb < 4; ++vb)
                dwa[hb][vb] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (want_dx) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                u32x4 wf[4];
#pragma unroll
                for (int hb = 0; hb < 4; ++hb) {
                    wf[hb] = *reinterpret_cast<const u32x4 *>(wt + (fo ^ (uint32_t)(64 * ks)) + hb * 16 * 128);
                    if (__builtin_expect(cur.n < kFewStep, 0)) {
                        // columns past the lane: its padding, or another row
                        const int left = cur.n - 32 * ks - 8 * g;
#pragma unroll
                        for (int d = 0; d < 4; ++d)
                            wf[hb][d] &= (left > 2 * d ? 0x0000FFFFu : 0u) | (left > 2 * d + 1 ? 0xFFFF0000u : 0u);
                    }
                }
#pragma unroll
                for (int part = 0; part < kParts; ++part)
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb) {
                        const u32x4 zf = *reinterpret_cast<const u32x4 *>(
                            zt + (fo ^ (uint32_t)(64 * ks)) + (part * kBp + 16 * mb) * 128);
#pragma unroll
                        for (int hb = 0; hb < 4; ++hb)
                            dxa[hb][mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8, wf[hb]), __builtin_bit_cast(bf16x8, zf),
                                dxa[hb][mb], 0, 0, 0);
                    }
            }
        }
        if (want_dw) {
#pragma unroll
            for (int kc = 0; kc < kKc; ++kc)
#pragma unroll
                for (int vb = 0; vb < 4; ++vb) {
                    // dz across: row 32 kc + 8 g + i / 4 (+ 4), columns 32 (vb / 2)
                    // + 8 (i % 4) + 4 (vb % 2) .. + 3: the MFMAs vb and vb + 1 leave
                    // 8 consecutive columns in a lane
                    const int r = 32 * kc + 8 * g + (n >> 2);
                    const int q = 4 * (vb >> 1) + (n & 3);
                    const uint8_t *p0 = zt + r * 128 + ((q ^ ((r >> 1) & 7)) * 16) + 8 * (vb & 1);
                    const uint8_t *p1 = zt + (r + 4) * 128 + ((q ^ (((r + 4) >> 1) & 7)) * 16) + 8 * (vb & 1);
                    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                    const u32x2 lo = __builtin_bit_cast(u32x2, read_across((lds_s16x4)p0));
                    const u32x2 hi = __builtin_bit_cast(u32x2, read_across((lds_s16x4)p1));
                    const u32x4 zf = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
                    for (int hb = 0; hb < 4; ++hb)
                        dwa[hb][vb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, zf), __builtin_bit_cast(bf16x8, xf[hb][kc % kXc]),
                            dwa[hb][vb], 0, 0, 0);
                }
        }
        if (kParts == 1) {
            const uint32_t c = (uint32_t)target - (uint32_t)(a.vocab.off[cur.lane] + cur.c);
            const bool hit = c < (uint32_t)cur.n;
            const uint64_t hits = __builtin_amdgcn_ballot_w64(hit);
            if (__builtin_expect(hits != 0, 0)) {
                // row L: the target's place among the step's columns, and what rounding took there
                const int at = hit ? (int)c : 0;
                const float took = rest * bf16_value(*reinterpret_cast<const uint16_t *>(
                                              zt + L * 128 + (((at >> 3) ^ ((L >> 1) & 7)) * 16) + 2 * (at & 7)));
                const float left = hit && fabsf(took) < INFINITY ? took : 0.f;
                if (want_dx)
                    for (uint64_t m = hits; m != 0; m &= m - 1) {
                        const int b = __builtin_ctzll(m), col = __builtin_amdgcn_readlane(at, b);
                        const float of_b = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(left), b));
                        const float mine = n == (b & 15) ? of_b : 0.f;
                        float v[4][4];
#pragma unroll
                        for (int hb = 0; hb < 4; ++hb)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int r = 16 * hb + 4 * g + e;
                                v[hb][e] = bf16_value(*reinterpret_cast<const uint16_t *>(
                                    wt + r * 128 + (((col >> 3) ^ ((r >> 1) & 7)) * 16) + 2 * (col & 7)));
                            }
#pragma unroll
                        for (int mb = 0; mb < MB; ++mb)
                            if (b >> 4 == mb)
#pragma unroll
                                for (int hb = 0; hb < 4; ++hb)
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        dxa[hb][mb][e] = add_rest(dxa[hb][mb][e], mine, v[hb][e]);
                    }
                if (want_dw) {
                    // another step of dW's product, with these in place of dz
                    const int packed = at << 16 | __builtin_bit_cast(uint16_t, (__bf16)left);
#pragma unroll
                    for (int kc = 0; kc < kXc; ++kc) {
                        if ((uint32_t)(hits >> (32 * kc)) == 0u)
                            continue;
                        u32x4 zf[4] = {};
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t of_b = (uint32_t)__shfl(packed, 32 * kc + 8 * g + j);
#pragma unroll
                            for (int vb = 0; vb < 4; ++vb)
                                if ((int)(of_b >> 16) == 32 * (vb >> 1) + 8 * (n >> 2) + 4 * (vb & 1) + (n & 3))
                                    zf[vb][j >> 1] |= (of_b & 0xFFFFu) << (16 * (j & 1));
                        }
#pragma unroll
                        for (int vb = 0; vb < 4; ++vb)
#pragma unroll
                            for (int hb = 0; hb < 4; ++hb)
                                block_mma(dwa[hb][vb], xf[hb][kc], zf[vb]);
                    }
                }
            }
        }
        wait_lds();  // the tiles are read: their slot can be filled again
        const Cols done = cur;
        cur = next;
        next = load(slot, st + 2 * kFewWaves);
        asm volatile("" ::: "memory");  // the stores below stay behind these loads
        stored = want_dw && done.n == kFewStep && hrows == kFewH;
        if (want_dw) {
#pragma unroll
            for (int hb = 0; hb < 4; ++hb) {
                const int h = hw + 16 * hb + n;
                if (h >= a.H)
                    continue;
                uint16_t *row = a.vocab.dw[done.lane] + (int64_t)h * a.lddw + done.c;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int c = 32 * half + 8 * g;
                    bf16x8 v;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = (__bf16)dwa[hb][2 * half + (e >> 2)][e & 3];
                    if (c + 8 <= done.n) {
                        *reinterpret_cast<bf16x8 *>(row + c) = v;
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (c + e < done.n)
                                row[c + e] = __builtin_bit_cast(uint16_t, (__bf16)v[e]);
                    }
                }
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(0x0f70);  // the ring's last (empty) loads
    if (want_dx)
#pragma unroll
        for (int hb = 0; hb < 4; ++hb) {
            const int h = hw + 16 * hb + 4 * g;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                const int b = 16 * mb + n;
                if (b < a.B && h < a.H)
                    *reinterpret_cast<f32x4 *>(a.dxp + ((int64_t)(split * kFewWaves + wave) * a.B + b) * a.ldxp + h) =
                        dxa[hb][mb];
            }
        }
}

// Four columns per thread; PARTS threads share a sum (splits p, p + PARTS, ..
// in ascending order each, then the parts in order).
template <int PARTS>
__global__ __launch_bounds__(256) void dx_finish_kernel(const LossArgs a)
{
    __shared__ f32x4 sums[PARTS][256 / PARTS];
    const int64_t quads = a.ldxp / 4;
    const int q = threadIdx.x % (256 / PARTS), part = threadIdx.x / (256 / PARTS);
    const int64_t at = (int64_t)blockIdx.x * (256 / PARTS) + q;
    const int64_t b = at / quads;
    const int c = (int)(at - b * quads) * 4;
    const bool ok = b < a.B;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (ok) {
        const float *p = a.dxp + b * a.ldxp + c;
#pragma unroll 4
        for (int i = part; i < a.splits; i += PARTS)
            s += *reinterpret_cast<const f32x4 *>(p + (int64_t)i * a.B * a.ldxp);
    }
    if (PARTS > 1) {
        sums[part][q] = s;
        __syncthreads();
        if (part > 0)
            return;
#pragma unroll
        for (int i = 1; i < PARTS; ++i)
            s += sums[i][q];
    }
    if (!ok)
        return;
    const float v[4] = {s[0], s[1], s[2], s[3]};
    store_bf16x4(a.dx + b * a.lddx + c, v, a.H - c);
}

// The slices' sums added up.
template <int USE>
hipError_t launch_join(const LossArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(join_kernel<USE>, dim3((unsigned)loss_parts(a.B, a.nblk, a.slices), a.B), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <class C, int USE, bool SPLIT>
hipError_t launch_logits_tiles(const LossArgs &a, hipStream_t s)
{
    const TileGrid g = tile_grid<C>(a.B, (int64_t)a.nblk * kVocabBlock);
    static std::atomic<uint64_t> lds_done{0};
    const hipError_t e = allow_lds((const void *)logits_kernel<C, USE, SPLIT>, C::kLds, lds_done);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((logits_kernel<C, USE, SPLIT>), dim3((unsigned)xcd_ids(tile_count(g) * a.slices)),
                       dim3(C::kThreads), C::kLds, s, a, g);
    return hipGetLastError();
}

template <int USE>
hipError_t launch_logits(const LossArgs &a, hipStream_t s)
{
    if (!small_logits(a.B, a.nblk))
        return launch_logits_tiles<BigTile, USE, false>(a, s);
    if (a.slices == 1)
        return launch_logits_tiles<SmallTile, USE, false>(a, s);
    const hipError_t e = launch_logits_tiles<SmallTile, kUseLoss, true>(a, s);
    return e != hipSuccess ? e : launch_join<USE>(a, s);
}

template <class C>
hipError_t launch_grad_tiles(const LossArgs &a, bool want_dx, bool want_dw, hipStream_t s)
{
    const TileGrid gx = tile_grid<C>(a.B, a.H), gw = tile_grid<C>(a.H, (int64_t)a.nblk * kVocabBlock);
    const int64_t dx_ids = want_dx ? xcd_ids(tile_count(gx) * a.splits) : 0;
    const int64_t ids = dx_ids + (want_dw ? xcd_ids(tile_count(gw)) : 0);
    if (ids <= 0)
        return hipSuccess;
    static std::atomic<uint64_t> lds_done{0};
    const hipError_t e = allow_lds((const void *)grad_kernel<C>, C::kLds, lds_done);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(grad_kernel<C>, dim3((unsigned)ids), dim3(C::kThreads), C::kLds, s, a, gx, (int)dx_ids, gw);
    return hipGetLastError();
}

template <int USE>
hipError_t launch_logits_rows(const LossArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)xcd_ids((int64_t)a.nblk * (kVocabBlock / kLossSmallTile) * a.slices));
    if (a.B <= 16)
        hipLaunchKernelGGL((logits_rows_kernel<1, USE>), grid, dim3(kRowsThreads), 0, s, a);
    else if (a.B <= 32)
        hipLaunchKernelGGL((logits_rows_kernel<2, USE>), grid, dim3(kRowsThreads), 0, s, a);
    else
        hipLaunchKernelGGL((logits_rows_kernel<4, USE>), grid, dim3(kRowsThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || a.slices == 1 ? e : launch_join<USE>(a, s);
}

// Steps of a workgroup where `splits` of them share the blocks.
inline int few_steps(int nblk, int splits)
{
    const int steps = nblk * (kVocabBlock / kFewStep);
    return ((steps + splits - 1) / splits + kFewWaves - 1) / kFewWaves * kFewWaves;
}

template <int MB>
hipError_t launch_few(const LossArgs &a, bool want_dx, bool want_dw, hipStream_t s)
{
    static std::atomic<uint64_t> lds_done{0};
    const hipError_t e = allow_lds((const void *)grad_rows_kernel<MB>, FewShape<MB>::kLds, lds_done);
    if (e != hipSuccess)
        return e;
    const int htiles = (a.H + kFewH - 1) / kFewH;
    const int splits = a.splits / kFewWaves;
    hipLaunchKernelGGL(grad_rows_kernel<MB>, dim3((unsigned)((int64_t)htiles * splits)), dim3(kFewThreads),
                       FewShape<MB>::kLds, s, a, htiles, few_steps(a.nblk, splits), (int)want_dx, (int)want_dw);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_loss_blocks(const LossArgs &a, hipStream_t s)
{
    return a.B <= kLossSmallRows ? launch_logits_rows<kUseLoss>(a, s) : launch_logits<kUseLoss>(a, s);
}

hipError_t launch_dlogits(const LossArgs &a, hipStream_t s)
{
    return a.B <= kLossSmallRows ? launch_logits_rows<kUseGrad>(a, s) : launch_logits<kUseGrad>(a, s);
}

hipError_t launch_loss_combine(const LossArgs &a, hipStream_t s)
{
    if (a.B <= kLossSmallRows || a.slices > 1) {
        hipLaunchKernelGGL(loss_rows_combine_kernel, dim3(a.B), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(loss_combine_kernel, dim3((unsigned)(((int64_t)a.B + kCombineRows - 1) / kCombineRows)),
                       dim3(kCombineRows * kCombineRuns), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_mask_rows(const LossArgs &a, uint16_t *xm, hipStream_t s)
{
    const int64_t items = (int64_t)a.B * (a.ldxm / 8);
    if (items <= 0)
        return hipSuccess;
    hipLaunchKernelGGL(mask_rows_kernel, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, s, a, xm);
    return hipGetLastError();
}

hipError_t launch_grad(const LossArgs &a, bool want_dx, bool want_dw, hipStream_t s)
{
    return small_grad(a.B, a.H, a.nblk) ? launch_grad_tiles<SmallTile>(a, want_dx, want_dw, s)
                                        : launch_grad_tiles<BigTile>(a, want_dx, want_dw, s);
}

hipError_t launch_grad_rows(const LossArgs &a, bool want_dx, bool want_dw, hipStream_t s)
{
    if (a.B <= 16)
        return launch_few<1>(a, want_dx, want_dw, s);
    if (a.B <= 32)
        return launch_few<2>(a, want_dx, want_dw, s);
    return launch_few<4>(a, want_dx, want_dw, s);
}

hipError_t launch_dx_finish(const LossArgs &a, hipStream_t s)
{
    const int64_t items = (int64_t)a.B * (a.ldxp / 4);
    if (items <= 0)
        return hipSuccess;
    if (a.B <= kLossSmallRows)
        hipLaunchKernelGGL(dx_finish_kernel<8>, dim3((unsigned)((items + 31) / 32)), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL(dx_finish_kernel<1>, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

int loss_slices(int32_t B, int32_t H, int32_t nblk)
{
    const int tiles = nblk * (kVocabBlock / kLossSmallTile);
    if (B <= 0 || tiles <= 0)
        return 1;
    // The slices fill the workgroups that the card holds at a time once (4, 3
    // or 2 on a CU, as the kernel's registers allow), with at least 16 K steps
    // each: a slice's sums are written and read again, and a second, partial
    // round costs a whole one (1024 places at every B: 132 us at B 64, H 4096,
    // V 65536, 104 us with 512).
    const int steps = (H + kLossStepK - 1) / kLossStepK;
    int64_t fit = 1;
    if (B <= kLossSmallRows)
        fit = (B <= 16 ? 1024 : B <= 32 ? 768 : 512) / tiles;
    else if (small_logits(B, nblk) && steps >= 64)
        // a small tile for every CU (V 4096 at B 128: 83 us whole and 30 us split
        // at H 8192, 30 and 25 us at H 2048, 21 and 24 us at H 1024)
        fit = 256 / tile_count(tile_grid<SmallTile>(B, (int64_t)nblk * kVocabBlock));
    const int s = (int)std::max<int64_t>(1, std::min<int64_t>(fit, steps / 16));
    const int per = loss_slice_steps(H, s);
    return per > 0 ? std::max(1, (steps + per - 1) / per) : 1;
}

int loss_slice_steps(int32_t H, int slices)
{
    const int steps = (H + kLossStepK - 1) / kLossStepK;
    return ((steps + slices - 1) / slices + kRowsWaves - 1) / kRowsWaves * kRowsWaves;
}

bool small_logits(int32_t B, int32_t nblk)
{
    return B <= kSmallRows ||
           tile_count(tile_grid<BigTile>(B, (int64_t)nblk * kVocabBlock)) <= kSmallLogitsTiles;
}

bool small_grad(int32_t B, int32_t H, int32_t nblk)
{
    const int64_t dw = tile_count(tile_grid<BigTile>(H, (int64_t)nblk * kVocabBlock));
    return B <= kSmallRows || dw * ((B + BigTile::kM - 1) / BigTile::kM) <= kSmallGradTiles;
}

int dx_splits(int32_t B, int32_t H, int32_t nblk)
{
    if (B <= kLossSmallRows) {
        // one workgroup of the streaming kernel to a CU (its LDS allows no
        // more); each of its waves has a partial sum of its own
        const int htiles = std::max(1, (H + kFewH - 1) / kFewH);
        const int steps = nblk * (kVocabBlock / kFewStep);
        const int s = std::max(1, std::min(256 / htiles, steps / kFewWaves));
        const int per = few_steps(nblk, s);
        return (steps + per - 1) / per * kFewWaves;
    }
    const bool small = small_grad(B, H, nblk);
    const int64_t tiles = small ? tile_count(tile_grid<SmallTile>(B, H)) : tile_count(tile_grid<BigTile>(B, H));
    if (tiles <= 0)
        return 1;
    // half of the launch's work is dX: with a tile for half of the CUs'
    // workgroups or more a tile's chain is within a CU's share
    const int64_t most = small ? 256 : 128;
    const int64_t s = (most + tiles - 1) / tiles;
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(s, 32), nblk));
}

int64_t loss_launch_items(int32_t B, int32_t H, int32_t nblk, int32_t splits)
{
    // the small tiles' launches hold twice the work items of the big ones'
    const int64_t logits = tile_count(tile_grid<SmallTile>(B, (int64_t)nblk * kVocabBlock)) *
                           loss_slices(B, H, nblk);
    const int64_t grad = tile_count(tile_grid<SmallTile>(B, H)) * splits +
                         tile_count(tile_grid<SmallTile>(H, (int64_t)nblk * kVocabBlock));
    int64_t items = (std::max(logits, grad) + 16) * SmallTile::kThreads;
    if (B <= kLossSmallRows) {
        const int64_t rows = xcd_ids((int64_t)nblk * (kVocabBlock / kLossSmallTile) * loss_slices(B, H, nblk));
        const int64_t few = ((int64_t)H + kFewH - 1) / kFewH * (splits / kFewWaves);
        items = std::max(std::max(rows * kRowsThreads, few * kFewThreads), (int64_t)loss_parts(1, nblk, 2) * 256);
    }
    items = std::max(items, ((int64_t)B + kCombineRows - 1) / kCombineRows * kCombineRows * kCombineRuns);
    return std::max(items, ((int64_t)B * (((int64_t)H + 7) / 8 * 8) / 4 + 255) / 256 * 256);
}

}  // namespace sbk
