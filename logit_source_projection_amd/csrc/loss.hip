// Softmax cross entropy of the output head and its gradient (gfx950).
//
//   z = X . W            lse_b = log sum_v exp(z_bv)
//   loss_b = lse_b - z_b,t(b)                     (0 where t(b) < 0)
//   dz_bv = (exp(z_bv - lse_b) - [v = t(b)]) g_b  (0 where t(b) < 0)
//   dX = dz . W^T        dW = X^T . dz
//
// The logits exist only in accumulators.  The forward pass reduces each 256 x
// 256 tile of them to (maximum, sum of exponentials) per row; the backward
// pass computes them again, piece by piece of the vocabulary, writes the
// piece's dz in bf16 and multiplies it both ways.
#include "loss.h"

#include <math.h>

#include <algorithm>

#include "tile_gemm.h"

namespace sbk {
namespace {

static_assert(kVocabBlock == kTile, "a vocabulary block is one tile wide");

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
};

enum LogitsUse { kUseLoss, kUseGrad };

template <int USE>
__global__ __launch_bounds__(kTileThreads, 1) void logits_kernel(const LossArgs a, const TileGrid grid)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int number = xcd_tile(blockIdx.x, grid.mt * grid.nt);
    if (number < 0)
        return;
    int mt, nt;
    tile_of(grid, number, mt, nt);
    const int nb = a.nb0 + nt;
    const int lane = block_lane(a.vocab, nb);
    const int c0 = (nb - a.vocab.blk0[lane]) * kTile;  // first column inside the lane
    const int nvalid = min(kTile, a.vocab.off[lane + 1] - a.vocab.off[lane] - c0);
    const int m0 = mt * kTile;
    const int rows = min(a.B - m0, kTile);
    const int H = a.H;

    LogitsSrc src;
    src.x = reinterpret_cast<const uint8_t *>(a.x + (int64_t)m0 * a.ldx);
    src.w = reinterpret_cast<const uint8_t *>(a.vocab.w[lane] + c0);
    src.ldw_bytes = a.ldw * 2;
    src.xbytes = ((int64_t)(rows - 1) * a.ldx + ((H + 7) & ~7)) * 2;
    src.wbytes = ((int64_t)(H - 1) * a.ldw + ((nvalid + 7) & ~7)) * 2;
    src.H = H;
    WaveTile<f32x4> t;
    t.init();
    t.run<kAlongK, kAcrossK, true, false>(smem, (H + kStageK - 1) / kStageK, a.ldx * 2, a.ldw * 2,
                                          src);

    const int n = t.L & 15, g = t.L >> 4;
    const int gcol0 = a.vocab.off[lane] + c0;
    if (USE == kUseLoss) {
        float2 *part = reinterpret_cast<float2 *>(smem);  // [kTile][4 column waves]
#pragma unroll
        for (int rb = 0; rb < kRowBlocks; ++rb) {
            const int r = t.row0 + 16 * rb + n;
            const int tgt = r < rows ? a.targets[m0 + r] - gcol0 : -1;  // target's column in the tile
            float m = -INFINITY;
#pragma unroll
            for (int cb = 0; cb < kColBlocks; ++cb)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = t.col0 + 16 * cb + 4 * g + e;
                    if (c < nvalid) {
                        m = fmaxf(m, t.acc[rb][cb][e]);
                        if (c == tgt)
                            a.zt[m0 + r] = t.acc[rb][cb][e];
                    }
                }
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            const float at = m == -INFINITY ? 0.f : m;
            float s = 0.f;
#pragma unroll
            for (int cb = 0; cb < kColBlocks; ++cb)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t.col0 + 16 * cb + 4 * g + e < nvalid)
                        s += __expf(t.acc[rb][cb][e] - at);
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            if (g == 0)
                part[r * 4 + (t.wave & 3)] = make_float2(m, s);
        }
        __syncthreads();
        const int r = threadIdx.x;
        if (r < rows) {
            float2 p = part[r * 4];
#pragma unroll
            for (int w = 1; w < 4; ++w)
                merge_ms(p.x, p.y, part[r * 4 + w].x, part[r * 4 + w].y);
            a.mse[(int64_t)nb * a.B + m0 + r] = p;
        }
    } else {
#pragma unroll
        for (int rb = 0; rb < kRowBlocks; ++rb) {
            const int r = t.row0 + 16 * rb + n;
            if (r >= rows)
                continue;
            const int tgt = a.targets[m0 + r];
            const float l = a.lse_in[m0 + r];
            // a target past the vocabulary has no gradient: NaN, not a guess
            const float scale = tgt >= a.V ? NAN : a.dloss[m0 + r];
            uint16_t *out = a.dz + (int64_t)(m0 + r) * a.ldz + (int64_t)nt * kTile;
#pragma unroll
            for (int cb = 0; cb < kColBlocks; ++cb) {
                const int c = t.col0 + 16 * cb + 4 * g;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = __expf(t.acc[rb][cb][e] - l) - (c + e == tgt - gcol0 ? 1.f : 0.f);
                    v[e] = tgt < 0 || c + e >= nvalid ? 0.f : p * scale;
                }
                store_bf16x4(out + c, v, 4);
            }
        }
    }
}

// One row per lane; wave w merges blocks w, w + 16, ... in ascending order and
// the waves are merged in wave order.
constexpr int kCombineWaves = 16;
__global__ __launch_bounds__(kCombineWaves * 64) void loss_combine_kernel(const LossArgs a)
{
    __shared__ float2 part[kCombineWaves][64];
    const int L = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t b = (int64_t)blockIdx.x * 64 + L;
    float m = -INFINITY, s = 0.f;
    if (b < a.B)
        for (int nb = wave; nb < a.nblk; nb += kCombineWaves) {
            const float2 p = a.mse[(int64_t)nb * a.B + b];
            merge_ms(m, s, p.x, p.y);
        }
    part[wave][L] = make_float2(m, s);
    __syncthreads();
    if (wave != 0 || b >= a.B)
        return;
    for (int w = 1; w < kCombineWaves; ++w)
        merge_ms(m, s, part[w][L].x, part[w][L].y);
    const float l = m + __logf(s);
    const int t = a.targets[b];
    a.lse[b] = l;
    a.loss[b] = t < 0 ? 0.f : (t >= a.V ? NAN : l - a.zt[b]);
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
    __device__ __forceinline__ DxSrc(const LossArgs &a_) : args(a_) {}
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t a(int st) const
    {
        const int64_t at = (int64_t)st * kStageBytes;
        return buffer_of(dz + at, st < (nb_end - nb_first) * (kTile / kStageK) ? dzbytes - at : 0);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t b(int st)
    {
        const int nb = nb_first + st / (kTile / kStageK);
        if (nb >= nb_end)
            return buffer_of(args.vocab.w[lane], 0);
        while (nb >= lane_end) {
            ++lane;
            lane_end = args.vocab.blk0[lane + 1];
        }
        const int c = (nb - args.vocab.blk0[lane]) * kTile + st % (kTile / kStageK) * kStageK;
        const int width = args.vocab.off[lane + 1] - args.vocab.off[lane];
        const int cols = max(0, min(kStageK, width - c));
        (st & 1 ? tail1 : tail0) = cols * 2;
        const int64_t first = (int64_t)h0 * args.ldw + c;
        return buffer_of(args.vocab.w[lane] + first,
                         cols > 0 ? ((int64_t)(hrows - 1) * args.ldw + ((cols + 7) & ~7)) * 2 : 0);
    }
    __device__ __forceinline__ int tail(int st) const { return st & 1 ? tail1 : tail0; }
};

// dW tile = X^T rows times a block of dz (k = batch rows).
struct DwSrc {
    const uint8_t *x, *dz;
    int64_t xbytes, zbytes, ldx_bytes, ldz_bytes;
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
// are left over.
__global__ __launch_bounds__(kTileThreads, 1) void grad_kernel(const LossArgs a, const TileGrid gx,
                                                               const int dx_ids, const TileGrid gw)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int n = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    WaveTile<f32x4> t;
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
        const int m0 = mt * kTile, rows = min(a.B - m0, kTile);
        DxSrc src(a);
        src.dz = reinterpret_cast<const uint8_t *>(a.dz + (int64_t)m0 * a.ldz + (int64_t)b0 * kTile);
        src.dzbytes = ((int64_t)(rows - 1) * a.ldz + (int64_t)(b1 - b0) * kTile) * 2;
        src.nb_first = a.nb0 + b0;
        src.nb_end = a.nb0 + b1;
        src.h0 = nt * kTile;
        src.hrows = min(a.H - src.h0, kTile);
        src.lane = block_lane(a.vocab, src.nb_first);
        src.lane_end = a.vocab.blk0[src.lane + 1];
        src.tail0 = src.tail1 = kStageBytes;
        t.init();
        t.run<kAlongK, kAlongK, false, true>(smem, (b1 - b0) * (kTile / kStageK), a.ldz * 2,
                                             a.ldw * 2, src);
#pragma unroll
        for (int rb = 0; rb < kRowBlocks; ++rb) {
            const int r = t.row0 + 16 * rb + n;
            if (r >= rows)
                continue;
#pragma unroll
            for (int cb = 0; cb < kColBlocks; ++cb) {
                const int c = src.h0 + t.col0 + 16 * cb + 4 * g;
                if (c >= a.H)
                    continue;
                if (a.dxp) {
                    f32x4 *p = reinterpret_cast<f32x4 *>(
                        a.dxp + ((int64_t)split * a.B + m0 + r) * a.ldxp + c);
                    *p = a.first ? t.acc[rb][cb] : *p + t.acc[rb][cb];
                } else {
                    const float v[4] = {t.acc[rb][cb][0], t.acc[rb][cb][1], t.acc[rb][cb][2],
                                        t.acc[rb][cb][3]};
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
    const int nb = a.nb0 + nt;
    const int lane = block_lane(a.vocab, nb);
    const int c0 = (nb - a.vocab.blk0[lane]) * kTile;
    const int nvalid = min(kTile, a.vocab.off[lane + 1] - a.vocab.off[lane] - c0);
    const int h0 = mt * kTile, hrows = min(a.H - h0, kTile);
    DwSrc src;
    src.x = reinterpret_cast<const uint8_t *>(a.xm + h0);
    src.dz = reinterpret_cast<const uint8_t *>(a.dz + (int64_t)nt * kTile);
    src.ldx_bytes = a.ldxm * 2;
    src.ldz_bytes = a.ldz * 2;
    src.xbytes = ((int64_t)(a.B - 1) * a.ldxm + ((hrows + 7) & ~7)) * 2;
    src.zbytes = ((int64_t)(a.B - 1) * a.ldz + kTile) * 2;
    t.init();
    t.run<kAcrossK, kAcrossK, false, false>(smem, (a.B + kStageK - 1) / kStageK, a.ldxm * 2,
                                            a.ldz * 2, src);
#pragma unroll
    for (int rb = 0; rb < kRowBlocks; ++rb) {
        const int r = t.row0 + 16 * rb + n;
        if (r >= hrows)
            continue;
        uint16_t *out = a.vocab.dw[lane] + (int64_t)(h0 + r) * a.lddw + c0;
#pragma unroll
        for (int cb = 0; cb < kColBlocks; ++cb) {
            const int c = t.col0 + 16 * cb + 4 * g;
            const float v[4] = {t.acc[rb][cb][0], t.acc[rb][cb][1], t.acc[rb][cb][2],
                                t.acc[rb][cb][3]};
            if (c < nvalid)
                store_bf16x4(out + c, v, nvalid - c);
        }
    }
}

// Four columns per thread; the splits are added in ascending order.
__global__ __launch_bounds__(256) void dx_finish_kernel(const LossArgs a)
{
    const int64_t quads = a.ldxp / 4;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t b = at / quads;
    const int c = (int)(at - b * quads) * 4;
    if (b >= a.B || c >= a.H)
        return;
    const float *p = a.dxp + b * a.ldxp + c;
    f32x4 s = *reinterpret_cast<const f32x4 *>(p);
    for (int i = 1; i < a.splits; ++i)
        s += *reinterpret_cast<const f32x4 *>(p + (int64_t)i * a.B * a.ldxp);
    const float v[4] = {s[0], s[1], s[2], s[3]};
    store_bf16x4(a.dx + b * a.lddx + c, v, a.H - c);
}

template <int USE>
hipError_t launch_logits(const LossArgs &a, hipStream_t s)
{
    const TileGrid g = tile_grid(a.B, (int64_t)a.nblk * kTile);
    static std::atomic<uint64_t> lds_done{0};
    const hipError_t e = allow_lds((const void *)logits_kernel<USE>, kTileLdsBytes, lds_done);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(logits_kernel<USE>, dim3((unsigned)xcd_ids(tile_count(g))),
                       dim3(kTileThreads), kTileLdsBytes, s, a, g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_loss_blocks(const LossArgs &a, hipStream_t s) { return launch_logits<kUseLoss>(a, s); }

hipError_t launch_dlogits(const LossArgs &a, hipStream_t s) { return launch_logits<kUseGrad>(a, s); }

hipError_t launch_loss_combine(const LossArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(loss_combine_kernel, dim3((unsigned)(((int64_t)a.B + 63) / 64)),
                       dim3(kCombineWaves * 64), 0, s, a);
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
    const TileGrid gx = tile_grid(a.B, a.H), gw = tile_grid(a.H, (int64_t)a.nblk * kTile);
    const int64_t dx_ids = want_dx ? xcd_ids(tile_count(gx) * a.splits) : 0;
    const int64_t ids = dx_ids + (want_dw ? xcd_ids(tile_count(gw)) : 0);
    if (ids <= 0)
        return hipSuccess;
    static std::atomic<uint64_t> lds_done{0};
    const hipError_t e = allow_lds((const void *)grad_kernel, kTileLdsBytes, lds_done);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(grad_kernel, dim3((unsigned)ids), dim3(kTileThreads), kTileLdsBytes, s, a, gx,
                       (int)dx_ids, gw);
    return hipGetLastError();
}

hipError_t launch_dx_finish(const LossArgs &a, hipStream_t s)
{
    const int64_t items = (int64_t)a.B * (a.ldxp / 4);
    if (items <= 0)
        return hipSuccess;
    hipLaunchKernelGGL(dx_finish_kernel, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

int dx_splits(int32_t B, int32_t H, int32_t nblk)
{
    const int64_t tiles = (int64_t)((B + kTile - 1) / kTile) * ((H + kTile - 1) / kTile);
    if (tiles <= 0)
        return 1;
    // half of the launch's work is dX: with 128 tiles or more a tile's chain
    // is within a CU's share
    const int64_t s = (128 + tiles - 1) / tiles;
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(s, 32), nblk));
}

int64_t loss_launch_items(int32_t B, int32_t H, int32_t nblk, int32_t splits)
{
    const int64_t logits = tile_count(tile_grid(B, (int64_t)nblk * kTile));
    const int64_t grad = tile_count(tile_grid(B, H)) * splits +
                         tile_count(tile_grid(H, (int64_t)nblk * kTile));
    int64_t items = (std::max(logits, grad) + 16) * kTileThreads;
    items = std::max(items, ((int64_t)B + 63) / 64 * 64 * kCombineWaves);
    return std::max(items, ((int64_t)B * (((int64_t)H + 7) / 8 * 8) / 4 + 255) / 256 * 256);
}

}  // namespace sbk
