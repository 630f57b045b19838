// The output head in 8-bit integers (gfx950).
//
//   x_scale_b = max_h |x_bh| / 127          q_bh = rint(x_bh / x_scale_b)
//   z_bv = float(sum_h q_bh w_vh) * x_scale_b * w_scale_v
//
// Integer sums are exact, so neither the order of a sum nor its split changes
// a bit; the three fp32 roundings of z are applied once, at the end.
#include "int8.h"

#include <limits.h>
#include <math.h>

#include <algorithm>

#include "tile_gemm.h"

namespace sbk {
namespace {

static_assert(kInt8LargeTile == BigTile::kN && kInt8LargeTile % SmallTile::kN == 0, "no tile spans two lanes");

// The order of the argmax: NaN above every number, then larger values, then
// lower indices (the projection calls' order).
__device__ __forceinline__ bool better(float v1, int i1, float v2, int i2)
{
    const bool n1 = v1 != v1, n2 = v2 != v2;
    if (n1 || n2)
        return n1 && (!n2 || i1 < i2);
    return v1 > v2 || (v1 == v2 && i1 < i2);
}

__device__ __forceinline__ void take_better(float &v, int &i, float v2, int i2)
{
    if (better(v2, i2, v, i)) {
        v = v2;
        i = i2;
    }
}

__device__ __forceinline__ int tile_lane(const Int8Args &a, int tile)
{
    int lane = 0;
    while (lane + 1 < a.k && a.tile0[lane + 1] <= tile)
        ++lane;
    return lane;
}

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

// ---------------------------------------------------------------------------
// Quantisation of rows: one workgroup per row.  The first kRowUnits 8-value
// units of every thread stay in registers between the maximum and the codes
// (rows of up to 32768 values are read once); longer rows are read again.
// ---------------------------------------------------------------------------
constexpr int kRowUnits = 4;
// Threads per row: enough that a unit or two per thread covers the row.
inline int row_threads(int H) { return H <= 2048 ? 256 : 1024; }

// The code of one value: the fp32 quotient rounded to the nearest, ties to even.
__device__ __forceinline__ int row_code(uint32_t bits, float scale)
{
    const float q = rintf(bf16_value(bits) / scale);
    return (int)fminf(fmaxf(q, -127.f), 127.f);
}

__device__ __forceinline__ uint2 unit_codes(const u32x4 &v, float scale)
{
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t bits = e & 1 ? v[e >> 1] >> 16 : v[e >> 1] & 0xFFFFu;
        w[e >> 2] |= ((uint32_t)row_code(bits, scale) & 0xFFu) << (8 * (e & 3));
    }
    return make_uint2(w[0], w[1]);
}

// |max| of a unit as bf16 bits: without the sign, larger bits are larger
// values, infinity above every number and NaN above infinity.
__device__ __forceinline__ uint32_t unit_max(const u32x4 &v, uint32_t m)
{
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        m = max(m, v[d] & 0x7FFFu);
        m = max(m, (v[d] >> 16) & 0x7FFFu);
    }
    return m;
}

// The scale of codes whose largest magnitude has these bf16 bits; 0 and
// non-finite maxima quantise to codes of 0 (see codes_of_zero).
__device__ __forceinline__ float code_scale(uint32_t maxbits) { return bf16_value(maxbits) / 127.f; }
__device__ __forceinline__ bool codes_of_zero(uint32_t maxbits) { return maxbits == 0 || maxbits >= 0x7F80u; }

template <int kRowThreads>
__global__ __launch_bounds__(kRowThreads) void quantize_rows_kernel(const uint16_t *x, int64_t ldx,
                                                                    int H, int8_t *q, int64_t ldq,
                                                                    float *scale)
{
    __shared__ uint32_t wave_max[kRowThreads / 64];
    const int64_t b = blockIdx.x;
    const uint16_t *row = x + b * ldx;
    int8_t *out = q + b * ldq;
    const int units = H / 8;  // whole units; the last H % 8 values are taken one by one
    u32x4 v[kRowUnits];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kRowUnits; ++i) {
        const int u = threadIdx.x + i * kRowThreads;
        v[i] = u < units ? *reinterpret_cast<const u32x4 *>(row + 8 * u) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < kRowUnits; ++i)
        m = unit_max(v[i], m);
    for (int u = threadIdx.x + kRowUnits * kRowThreads; u < units; u += kRowThreads)
        m = unit_max(*reinterpret_cast<const u32x4 *>(row + 8 * u), m);
    const int tail = 8 * units + threadIdx.x;  // < H for at most 7 threads
    if (tail < H)
        m = max(m, (uint32_t)row[tail] & 0x7FFFu);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        m = max(m, (uint32_t)__shfl_xor((int)m, d));
    if ((threadIdx.x & 63) == 0)
        wave_max[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRowThreads / 64; ++w)
        m = max(m, wave_max[w]);
    const float s = code_scale(m);
    if (threadIdx.x == 0)
        scale[b] = s;
    const bool zero = codes_of_zero(m);
#pragma unroll
    for (int i = 0; i < kRowUnits; ++i) {
        const int u = threadIdx.x + i * kRowThreads;
        if (u < units)
            *reinterpret_cast<uint2 *>(out + 8 * u) = zero ? make_uint2(0u, 0u) : unit_codes(v[i], s);
    }
    for (int u = threadIdx.x + kRowUnits * kRowThreads; u < units; u += kRowThreads)
        *reinterpret_cast<uint2 *>(out + 8 * u) =
            zero ? make_uint2(0u, 0u) : unit_codes(*reinterpret_cast<const u32x4 *>(row + 8 * u), s);
    if (tail < H)
        out[tail] = zero ? (int8_t)0 : (int8_t)row_code(row[tail], s);
}

// ---------------------------------------------------------------------------
// Quantisation of a bf16 head [H][V] into channels [V][H] with one scale each.
// One workgroup = 64 channels: a first pass over H for the channels' maxima, a
// second that turns blocks of 256 rows x 64 channels round through LDS.  Both
// read 16 bytes (8 channels of a row) per thread, several at once; the second
// finds much of its 2 HV bytes in the caches.  Bound by those bytes and the
// divisions: 263 us at H 5120, V 37984 (2.2 TB/s counting the weight once; one
// channel per thread and 2-byte loads took 1226 us).
// ---------------------------------------------------------------------------
typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));
constexpr int kHeadThreads = kInt8QuantizeThreads, kHeadRows = 256;
constexpr int kHeadPitch = kHeadRows + 4;  // bytes of a turned channel: 65 words, an odd number of banks

__global__ __launch_bounds__(kHeadThreads) void quantize_head_kernel(const Int8QuantizeArgs a)
{
    static_assert(kInt8QuantizeTile == 64, "8 threads of 8 channels per row");
    __shared__ u16x8 cmax[kHeadThreads / 8][8];
    __shared__ float cscale[64];
    __shared__ uint32_t czero[64];
    __shared__ uint32_t turn[64 * kHeadPitch / 4];
    int lane = 0;
    while (lane + 1 < a.k && a.tile0[lane + 1] <= (int)blockIdx.x)
        ++lane;
    const int c0 = (blockIdx.x - a.tile0[lane]) * 64;
    const int width = min(64, a.off[lane + 1] - a.off[lane] - c0);
    const int c8 = threadIdx.x & 7, r = threadIdx.x >> 3;
    const bool ok = 8 * c8 < width;  // the unit holds a channel (rows are whole 16-byte units)
    const uint16_t *w = a.w[lane] + c0 + 8 * c8;
    u16x8 m = {0, 0, 0, 0, 0, 0, 0, 0};
    if (ok)
#pragma unroll 8
        for (int h = r; h < a.H; h += kHeadThreads / 8)
            m = __builtin_elementwise_max(m, *reinterpret_cast<const u16x8 *>(w + (int64_t)h * a.ldw) &
                                                 (unsigned short)0x7FFF);
    cmax[r][c8] = m;
    __syncthreads();
    if (threadIdx.x < 64) {
        const int c = threadIdx.x;
        uint32_t top = 0;
        for (int i = 0; i < kHeadThreads / 8; ++i)
            top = max(top, (uint32_t)cmax[i][c >> 3][c & 7]);
        const float s = code_scale(top);
        cscale[c] = s;
        czero[c] = codes_of_zero(top);
        if (c < width)
            a.scale[lane][c0 + c] = s;
    }
    __syncthreads();
    for (int h0 = 0; h0 < a.H; h0 += kHeadRows) {
        // four rows 4 r .. 4 r + 3 of a unit: a word of codes per channel
        u16x8 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int h = h0 + 4 * r + i;
            v[i] = ok && h < a.H ? *reinterpret_cast<const u16x8 *>(w + (int64_t)h * a.ldw)
                                 : u16x8{0, 0, 0, 0, 0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = 8 * c8 + j;
            uint32_t word = 0;
            if (!czero[c]) {
                const float s = cscale[c];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    word |= ((uint32_t)row_code(v[i][j], s) & 0xFFu) << (8 * i);
            }
            turn[c * (kHeadPitch / 4) + r] = word;
        }
        __syncthreads();
        // 16 codes per thread and turn: 16 threads store 256 bytes of a channel
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int c = (threadIdx.x >> 4) + 32 * t, q = 4 * (threadIdx.x & 15);
            const uint32_t *p = turn + c * (kHeadPitch / 4) + q;
            const u32x4 codes = {p[0], p[1], p[2], p[3]};
            const int h = h0 + 4 * q;
            if (c < width && h < a.H) {
                int8_t *out = a.q[lane] + (int64_t)(c0 + c) * a.ldq + h;
                if (h + 16 <= a.H) {
                    *reinterpret_cast<u32x4 *>(out) = codes;
                } else {
                    for (int e = 0; h + e < a.H; ++e)
                        out[e] = (int8_t)(codes[e >> 2] >> (8 * (e & 3)));
                }
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Epilogue of four consecutive channels of one row.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void scaled(const i32x4 &acc, float xs, const float *ws, int n, float (&z)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e)
        z[e] = e < n ? ((float)acc[e] * xs) * ws[e] : 0.f;
}

// z to columns gcol .. of row b, the first n of them.
__device__ __forceinline__ void store_logits(const Int8Args &a, int64_t b, int gcol, const float (&z)[4], int n)
{
    if (a.bf16) {
        uint16_t *p = static_cast<uint16_t *>(a.out) + b * a.ldo + gcol;
        if (n >= 4 && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
            bf16x4 h;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                h[e] = (__bf16)z[e];
            *reinterpret_cast<uint2 *>(p) = __builtin_bit_cast(uint2, h);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n)
                    p[e] = __builtin_bit_cast(uint16_t, (__bf16)z[e]);
        }
    } else {
        float *p = static_cast<float *>(a.out) + b * a.ldo + gcol;
        if (n >= 4 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
            *reinterpret_cast<f32x4 *>(p) = f32x4{z[0], z[1], z[2], z[3]};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n)
                    p[e] = z[e];
        }
    }
}

// ---------------------------------------------------------------------------
// Large batches: MFMA tiles, both operands along K.  Bound by MFMA: 2048 rows of
// H 5120, V 151936 take 1.46 ms with 1.24 GB of fp32 logits written (2.18 POP/s),
// the IDs of 1024 rows 0.69 ms (2.3 POP/s, what one large library product gets).
// Few tiles split K (int8_slices): a slice stores its 32-bit sums, which
// int8_join_kernel adds up; integer sums do not depend on the split.  (The split as
// a template argument: 128 rows, H 1024, V 14000 12.6 -> 12.8 us.)
// ---------------------------------------------------------------------------
struct Int8Src {
    const uint8_t *x, *w;
    int64_t xbytes, wbytes;
    int H;
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t a(int st) const
    {
        const int64_t at = (int64_t)st * kStageBytes;
        return buffer_of(x + at, at < H ? xbytes - at : 0);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t b(int st) const
    {
        const int64_t at = (int64_t)st * kStageBytes;
        return buffer_of(w + at, at < H ? wbytes - at : 0);
    }
    __device__ __forceinline__ int tail(int st) const { return min(H - st * kStageBytes, kStageBytes); }
    __device__ __forceinline__ void meanwhile() const {}
};

template <class C, bool TOKENS>
__global__ __launch_bounds__(C::kThreads, C::kPerCu) void int8_tile_kernel(const Int8Args a, const TileGrid grid)
{
    constexpr int kM = C::kM, kN = C::kN, kWN = C::kWN, kRB = C::kRB, kCB = C::kCB;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    // only small tiles split K; big ones have no register to spare for it
    const int slices = C::kPerCu > 1 ? a.slices : 1;
    const int tiles = grid.mt * grid.nt, number = xcd_tile(blockIdx.x, tiles * slices);
    if (number < 0)
        return;
    const int slice = number / tiles;
    int mt, nt;
    tile_of(grid, number - slice * tiles, mt, nt);
    const int block = nt / (kInt8LargeTile / kN);
    const int lane = tile_lane(a, block);
    // first channel inside the lane (a block's later tiles can lie past it)
    const int c0 = (block - a.tile0[lane]) * kInt8LargeTile + nt % (kInt8LargeTile / kN) * kN;
    const int nvalid = max(0, min(kN, a.off[lane + 1] - a.off[lane] - c0));
    const int m0 = mt * kM, rows = min(a.B - m0, kM);
    // the slice's part of K: H bytes from k0
    const int k0 = slice * a.slice_steps * kInt8StepK;
    const int H = slices > 1 ? min(a.H - k0, a.slice_steps * kInt8StepK) : a.H;
    const int padded = ((a.H + 15) & ~15) - k0;
    Int8Src src;
    src.x = reinterpret_cast<const uint8_t *>(a.x + (int64_t)m0 * a.ldx + k0);
    src.w = reinterpret_cast<const uint8_t *>(a.w[lane] + (int64_t)c0 * a.ldw + k0);
    src.xbytes = (int64_t)(rows - 1) * a.ldx + padded;
    src.wbytes = nvalid > 0 ? (int64_t)(nvalid - 1) * a.ldw + padded : 0;
    src.H = H;
    WaveTile<C, i32x4> t;
    t.init();
    // a ragged H: x zeroed past it makes the products there 0
    t.template run<kAlongK, kAlongK, true, false>(smem, (H + kStageBytes - 1) / kStageBytes, a.ldx, a.ldw, src);

    const int n = t.L & 15, g = t.L >> 4;
    if (slices > 1) {
        const int64_t ld = (int64_t)a.tile0[a.k] * kInt8LargeTile;
        int32_t *p = a.part + ((int64_t)slice * a.B + m0) * ld + (int64_t)nt * kN + t.col0 + 4 * g;
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb) {
            const int r = t.row0 + 16 * rb + n;
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb)
                if (r < rows)
                    *reinterpret_cast<i32x4 *>(p + r * ld + 16 * cb) = t.acc[rb][cb];
        }
        return;
    }
    const int gcol0 = a.off[lane] + c0;
    float2 *part = reinterpret_cast<float2 *>(smem);  // [kM][column waves]
    float ws[kCB][4];
#pragma unroll
    for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = t.col0 + 16 * cb + 4 * g + e;
            ws[cb][e] = c < nvalid ? a.w_scale[lane][c0 + c] : 0.f;
        }
    const bool ragged = nvalid < t.col0 + 16 * kCB;
    const int lcol0 = gcol0 + t.col0 + 4 * g;  // the lane's first column
#pragma unroll
    for (int rb = 0; rb < kRB; ++rb) {
        const int r = t.row0 + 16 * rb + n;
        const float xs = r < rows ? a.x_scale[m0 + r] : 0.f;
        float z[kCB][4];
#pragma unroll
        for (int cb = 0; cb < kCB; ++cb)
            scaled(t.acc[rb][cb], xs, ws[cb], 4, z[cb]);
        if (!TOKENS) {
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb) {
                const int c = t.col0 + 16 * cb + 4 * g;
                if (r < rows && c < nvalid)
                    store_logits(a, m0 + r, gcol0 + c, z[cb], nvalid - c);
            }
            continue;
        }
        // The NaN-propagating maximum of the lane's values tells whether the
        // wave needs the full order; else the row's maximum comes first and
        // then the lowest column that equals it, two instructions per value.
        float bv = z[0][0];
#pragma unroll
        for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                bv = __builtin_elementwise_maximum(bv, z[cb][e]);
        int bi = INT_MAX;
        if (!ragged && __builtin_amdgcn_ballot_w64(bv != bv) == 0) {
            bv = fmaxf(bv, __shfl_xor(bv, 16));
            bv = fmaxf(bv, __shfl_xor(bv, 32));
#pragma unroll
            for (int cb = kCB - 1; cb >= 0; --cb)
#pragma unroll
                for (int e = 3; e >= 0; --e)
                    if (z[cb][e] == bv)
                        bi = 16 * cb + e;
            bi = bi == INT_MAX ? bi : lcol0 + bi;
            bi = min(bi, __shfl_xor(bi, 16));
            bi = min(bi, __shfl_xor(bi, 32));
        } else {
            bv = -INFINITY;
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t.col0 + 16 * cb + 4 * g + e < nvalid)
                        take_better(bv, bi, z[cb][e], lcol0 + 16 * cb + e);
            take_better(bv, bi, __shfl_xor(bv, 16), __shfl_xor(bi, 16));
            take_better(bv, bi, __shfl_xor(bv, 32), __shfl_xor(bi, 32));
        }
        if (g == 0)
            part[r * kWN + t.wave % kWN] = make_float2(bv, __int_as_float(bi));
    }
    if (TOKENS) {
        __syncthreads();
        const int r = threadIdx.x;
        if (r < rows) {
            float v = part[r * kWN].x;
            int i = __float_as_int(part[r * kWN].y);
#pragma unroll
            for (int w = 1; w < kWN; ++w)
                take_better(v, i, part[r * kWN + w].x, __float_as_int(part[r * kWN + w].y));
            a.pair[(int64_t)(m0 + r) * a.pairs + nt] = make_int2(__float_as_int(v), i);
        }
    }
}

// ---------------------------------------------------------------------------
// Up to 64 rows (int8_few): the weight streams from memory once.  One workgroup
// = 4 waves = 64 channels of one lane; wave w takes the K steps w, w + 4, ... of its
// slice (128 bytes each), and the four partial tiles meet in LDS.
//
// Bound by the weight's bytes.  MFMA wants 16 bytes of 16 channels per load,
// half a cache line of each: loaded straight into registers, the second half
// of every line was fetched again (non-temporal: 198 us at 16 rows, H 5120, V
// 151936) or cost L1 look-ups (158 us).  So every wave fills a private LDS ring
// of kSlots steps with direct-to-LDS loads of 8 whole lines and reads its
// fragments from there; nothing is shared before the end, so there is no
// barrier in the loop, only the wave's own load counter.
// ---------------------------------------------------------------------------
constexpr int kRowsWaves = 4, kRowsThreads = kRowsWaves * 64;
constexpr int kRowsBlocks = kInt8SmallTile / 16;  // 16-channel blocks per tile
constexpr int kRowsSlots = 2;
constexpr int kRowsSlotBytes = kInt8SmallTile * kInt8StepK;
constexpr int kRowsLoads = kRowsSlotBytes / 1024;
constexpr int kRowsLdsBytes = kRowsWaves * kRowsSlots * kRowsSlotBytes;
constexpr int kRedStride = kInt8SmallTile / 4 + 1;  // quads per row of a partial tile, one of padding
static_assert(kRowsWaves * 16 * kRedStride * 16 <= kRowsLdsBytes, "the partial tiles reuse the ring");

template <int MB, bool TOKENS>
__global__ __launch_bounds__(kRowsThreads) void int8_rows_kernel(const Int8Args a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tile = blockIdx.x / a.slices, slice = blockIdx.x - tile * a.slices;
    const int lane = tile_lane(a, tile);
    const int c0 = (tile - a.tile0[lane]) * kInt8SmallTile;
    const int nvalid = min(kInt8SmallTile, a.off[lane + 1] - a.off[lane] - c0);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int L = threadIdx.x & 63, n = L & 15, g = L >> 4;
    const int H = a.H;
    const int64_t hb = (H + 15) & ~15;
    // buffers end with the last row's and channel's last unit; what lies past H
    // inside a unit is masked out of x
    const uint8_t *xp = reinterpret_cast<const uint8_t *>(a.x);
    const uint8_t *wp = reinterpret_cast<const uint8_t *>(a.w[lane] + (int64_t)c0 * a.ldw);
    const int64_t xbytes = H > 0 ? (int64_t)(a.B - 1) * a.ldx + hb : 0;
    const int64_t wbytes = H > 0 ? (int64_t)(nvalid - 1) * a.ldw + hb : 0;
    uint32_t xo[MB], wo[kRowsLoads];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
        xo[mb] = (uint32_t)((int64_t)(16 * mb + n) * a.ldx + 16 * g);
    // load i brings channels 8 i .. 8 i + 7; piece p of channel c sits in slot
    // p ^ ((c / 2) & 7) of its line
#pragma unroll
    for (int i = 0; i < kRowsLoads; ++i) {
        const int c = 8 * i + (L >> 3);
        wo[i] = (uint32_t)((int64_t)c * a.ldw + 16 * ((L & 7) ^ ((c >> 1) & 7)));
    }
    uint8_t *const ring = smem + wave * (kRowsSlots * kRowsSlotBytes);
    const uint32_t fo = (uint32_t)(n * kInt8StepK + ((g ^ ((n >> 1) & 7)) * 16));
    i32x4 acc[MB][kRowsBlocks];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int cb = 0; cb < kRowsBlocks; ++cb)
            acc[mb][cb] = i32x4{0, 0, 0, 0};
    const int steps = (H + kInt8StepK - 1) / kInt8StepK;
    const int s0 = slice * a.slice_steps, s1 = min(s0 + a.slice_steps, steps);
    u32x4 fx[kRowsSlots][2][MB];
    // (at or past s1: zeros)
    auto load = [&](int j, int st) {
        const int64_t at = (int64_t)st * kInt8StepK;
        const __amdgpu_buffer_rsrc_t rw = buffer_of(wp + at, st < s1 ? wbytes - at : 0);
        const __amdgpu_buffer_rsrc_t rx = buffer_of(xp + at, st < s1 ? xbytes - at : 0);
#pragma unroll
        for (int i = 0; i < kRowsLoads; ++i)
            load_to_lds<2>(ring + j * kRowsSlotBytes + i * 1024, rw, wo[i]);
        // (new to the compiler in every step, which else keeps xo + 64 in registers of its
        // own instead of the load's immediate)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
            asm("" : "+v"(xo[mb]));
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                fx[j][i][mb] = __builtin_bit_cast(  // (only the vector offset is bounds-checked)
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, xo[mb] + 64 * i, 0, 0));
    };
#pragma unroll
    for (int j = 0; j < kRowsSlots; ++j)
        load(j, s0 + wave + j * kRowsWaves);
    for (int st = s0 + wave; st < s1; st += kRowsSlots * kRowsWaves) {
#pragma unroll
        for (int j = 0; j < kRowsSlots; ++j) {
            const int sj = st + j * kRowsWaves;
            // this slot's loads are done: only the later slots' are in flight
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(vmcnt_only((kRowsSlots - 1) * (kRowsLoads + 2 * MB)));
            asm volatile("" ::: "memory");
            u32x4 xa[2][MB], wb[2][kRowsBlocks];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int cb = 0; cb < kRowsBlocks; ++cb)
                    wb[i][cb] = *reinterpret_cast<const u32x4 *>(
                        ring + j * kRowsSlotBytes + (fo ^ (uint32_t)(64 * i)) + cb * 16 * kInt8StepK);
                // values of x at and past H (a row's padding, or the next row)
                const int left = H - sj * kInt8StepK - 64 * i - 16 * g;
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
                    xa[i][mb] = fx[j][i][mb];
                    if (__builtin_expect(sj * kInt8StepK + kInt8StepK > H, 0)) {
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const int keep = left - 4 * d;  // valid bytes of the word
                            xa[i][mb][d] &= keep >= 4 ? 0xFFFFFFFFu : (keep <= 0 ? 0u : (1u << (8 * keep)) - 1u);
                        }
                    }
                }
            }
            // the fragments are in registers before the slot is filled again
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
            load(j, sj + kRowsSlots * kRowsWaves);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int cb = 0; cb < kRowsBlocks; ++cb)
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
                        acc[mb][cb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                            __builtin_bit_cast(i32x4, wb[i][cb]), __builtin_bit_cast(i32x4, xa[i][mb]),
                            acc[mb][cb], 0, 0, 0);
        }
    }
    // the ring's last (empty) loads are done in every wave: LDS is free
    __builtin_amdgcn_s_waitcnt(0x0070);
    i32x4 *const red = reinterpret_cast<i32x4 *>(smem);  // [wave][16 rows][kRedStride]
    // thread: row threadIdx.x / kQuads of the block, four channels
    constexpr int kQuads = kInt8SmallTile / 4;
    const int er = threadIdx.x / kQuads, ec = 4 * (threadIdx.x % kQuads);
    const int left = nvalid - ec;
    const int gcol = a.off[lane] + c0 + ec;
    float ws[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        ws[e] = e < left ? a.w_scale[lane][c0 + ec + e] : 0.f;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        if (16 * mb >= a.B)
            break;
        __syncthreads();
#pragma unroll
        for (int cb = 0; cb < kRowsBlocks; ++cb)
            red[(wave * 16 + n) * kRedStride + 4 * cb + g] = acc[mb][cb];
        __syncthreads();
        if (er >= 16)
            continue;
        i32x4 sum = red[er * kRedStride + ec / 4];
#pragma unroll
        for (int w = 1; w < kRowsWaves; ++w)
            sum += red[(w * 16 + er) * kRedStride + ec / 4];
        const int b = 16 * mb + er;
        if (a.slices > 1) {
            if (b < a.B) {
                const int64_t ld = (int64_t)a.tile0[a.k] * kInt8SmallTile;
                *reinterpret_cast<i32x4 *>(a.part + ((int64_t)slice * a.B + b) * ld +
                                           (int64_t)tile * kInt8SmallTile + ec) = sum;
            }
            continue;
        }
        float z[4];
        scaled(sum, b < a.B ? a.x_scale[b] : 0.f, ws, 4, z);
        if (!TOKENS) {
            if (b < a.B && left > 0)
                store_logits(a, b, gcol, z, left);
            continue;
        }
        float bv = -INFINITY;
        int bi = INT_MAX;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left)
                take_better(bv, bi, z[e], gcol + e);
#pragma unroll
        for (int d = 1; d < kQuads; d <<= 1)
            take_better(bv, bi, __shfl_xor(bv, d), __shfl_xor(bi, d));
        if (ec == 0 && b < a.B)
            a.pair[(int64_t)b * a.pairs + tile] = make_int2(__float_as_int(bv), bi);
    }
}

// The slices of a split product added up: one workgroup = kInt8Chunk columns
// of one row.
template <bool TOKENS>
__global__ __launch_bounds__(256) void int8_join_kernel(const Int8Args a)
{
    __shared__ float wv[4];
    __shared__ int wi[4];
    const int b = blockIdx.y;
    const int col = blockIdx.x * kInt8Chunk + 4 * threadIdx.x;  // among the tiles' columns
    const int width = int8_tile(a.few);
    const int64_t ld = (int64_t)a.tile0[a.k] * width;
    float bv = -INFINITY;
    int bi = INT_MAX;
    if (col < ld) {
        const int tile = col / width;
        const int lane = tile_lane(a, tile);
        const int c = (tile - a.tile0[lane]) * width + col % width;
        const int left = a.off[lane + 1] - a.off[lane] - c;
        if (left > 0) {
            const int32_t *p = a.part + (int64_t)b * ld + col;
            i32x4 sum = *reinterpret_cast<const i32x4 *>(p);
#pragma unroll 4
            for (int s = 1; s < a.slices; ++s)
                sum += *reinterpret_cast<const i32x4 *>(p + (int64_t)s * a.B * ld);
            float ws[4], z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                ws[e] = e < left ? a.w_scale[lane][c + e] : 0.f;
            scaled(sum, a.x_scale[b], ws, 4, z);
            const int gcol = a.off[lane] + c;
            if (!TOKENS)
                store_logits(a, b, gcol, z, left);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (TOKENS && e < left)
                    take_better(bv, bi, z[e], gcol + e);
        }
    }
    if (TOKENS) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
            take_better(bv, bi, __shfl_xor(bv, d), __shfl_xor(bi, d));
        if ((threadIdx.x & 63) == 0) {
            wv[threadIdx.x >> 6] = bv;
            wi[threadIdx.x >> 6] = bi;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < 4; ++w)
                take_better(bv, bi, wv[w], wi[w]);
            a.pair[(int64_t)b * a.pairs + blockIdx.x] = make_int2(__float_as_int(bv), bi);
        }
    }
}

// One workgroup per row folds its pairs.
constexpr int kIdsThreads = 1024;
__global__ __launch_bounds__(kIdsThreads) void int8_ids_kernel(const Int8Args a)
{
    __shared__ float wv[kIdsThreads / 64];
    __shared__ int wi[kIdsThreads / 64];
    const int64_t b = blockIdx.x;
    float bv = -INFINITY;
    int bi = INT_MAX;
    for (int t = threadIdx.x; t < a.pairs; t += kIdsThreads) {
        const int2 p = a.pair[b * a.pairs + t];
        take_better(bv, bi, __int_as_float(p.x), p.y);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        take_better(bv, bi, __shfl_xor(bv, d), __shfl_xor(bi, d));
    if ((threadIdx.x & 63) == 0) {
        wv[threadIdx.x >> 6] = bv;
        wi[threadIdx.x >> 6] = bi;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kIdsThreads / 64; ++w)
            take_better(bv, bi, wv[w], wi[w]);
        a.ids[b] = bi;
    }
}

template <int MB, bool TOKENS>
hipError_t launch_rows(const Int8Args &a, hipStream_t s)
{
    static std::atomic<uint64_t> lds_done{0};
    const hipError_t e = allow_lds((const void *)int8_rows_kernel<MB, TOKENS>, kRowsLdsBytes, lds_done);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((int8_rows_kernel<MB, TOKENS>), dim3((unsigned)((int64_t)a.tile0[a.k] * a.slices)),
                       dim3(kRowsThreads), kRowsLdsBytes, s, a);
    return hipGetLastError();
}

template <class C, bool TOKENS>
hipError_t launch_tiles_as(const Int8Args &a, hipStream_t s)
{
    const TileGrid g = tile_grid<C>(a.B, (int64_t)a.tile0[a.k] * kInt8LargeTile);
    static std::atomic<uint64_t> lds_done{0};
    const hipError_t e = allow_lds((const void *)int8_tile_kernel<C, TOKENS>, C::kLds, lds_done);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((int8_tile_kernel<C, TOKENS>), dim3((unsigned)xcd_ids(tile_count(g) * a.slices)), dim3(C::kThreads),
                       C::kLds, s, a, g);
    return hipGetLastError();
}

template <bool TOKENS>
hipError_t launch_tiles(const Int8Args &a, hipStream_t s)
{
    return int8_small(a.B, a.tile0[a.k]) ? launch_tiles_as<SmallTile, TOKENS>(a, s)
                                         : launch_tiles_as<BigTile, TOKENS>(a, s);
}

}  // namespace

int int8_slices(bool few, int32_t B, int32_t H, int32_t tiles)
{
    if (B <= 0 || tiles <= 0)
        return 1;
    // Slices of at least 8 K steps fill the card once: 512 workgroups of the
    // streaming kernel, two on a CU (the 64-row product of H 17408 and V 5120, 80
    // tiles: 47.0 us in 12 slices, two rounds, 39.0 us in 6), or a small tile for
    // every CU (V 5120, 40 tiles at B 128: 94 us whole, 38 us in 6 slices, 43 us in
    // 12, whose sums are twice as many; H 5120, V 17408, 136 tiles at B 128: 41 us
    // whole, 46 us in 3).  Splitting tiles pays from 28 steps on (V 4096 at B 128:
    // 28 us split and 24 us whole at H 2560, 29 and 32 us at H 3584).
    const int steps = (H + kInt8StepK - 1) / kInt8StepK;
    int64_t fit = 1;
    if (few)
        fit = 512 / tiles;
    else if (int8_small(B, tiles) && steps >= 28)
        fit = 256 / tile_count(tile_grid<SmallTile>(B, (int64_t)tiles * kInt8LargeTile));
    const int s = (int)std::max<int64_t>(1, std::min<int64_t>(fit, steps / 8));
    const int per = int8_slice_steps(H, s);
    return per > 0 ? std::max(1, (steps + per - 1) / per) : 1;
}

bool int8_small(int32_t B, int32_t tiles)
{
    return B <= kInt8TileSmallRows ||
           tile_count(tile_grid<BigTile>(B, (int64_t)tiles * kInt8LargeTile)) <= kInt8SmallTiles;
}

int int8_slice_steps(int32_t H, int slices)
{
    const int steps = (H + kInt8StepK - 1) / kInt8StepK;
    return ((steps + slices - 1) / slices + kRowsWaves - 1) / kRowsWaves * kRowsWaves;
}

hipError_t launch_int8_quantize_rows(const uint16_t *x, int64_t ldx, int32_t B, int32_t H, int8_t *q,
                                     int64_t ldq, float *scale, hipStream_t s)
{
    if (B <= 0)
        return hipSuccess;
    if (row_threads(H) == 256)
        hipLaunchKernelGGL(quantize_rows_kernel<256>, dim3(B), dim3(256), 0, s, x, ldx, H, q, ldq, scale);
    else
        hipLaunchKernelGGL(quantize_rows_kernel<1024>, dim3(B), dim3(1024), 0, s, x, ldx, H, q, ldq, scale);
    return hipGetLastError();
}

hipError_t launch_int8_quantize_head(const Int8QuantizeArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(quantize_head_kernel, dim3((unsigned)a.tile0[a.k]), dim3(kHeadThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_int8(const Int8Args &a, hipStream_t s)
{
    hipError_t e;
    if (!a.few)
        e = a.ids ? launch_tiles<true>(a, s) : launch_tiles<false>(a, s);
    else if (a.B <= 16)
        e = a.ids ? launch_rows<1, true>(a, s) : launch_rows<1, false>(a, s);
    else if (a.B <= 32)
        e = a.ids ? launch_rows<2, true>(a, s) : launch_rows<2, false>(a, s);
    else
        e = a.ids ? launch_rows<4, true>(a, s) : launch_rows<4, false>(a, s);
    if (e != hipSuccess)
        return e;
    if (a.slices > 1) {
        const dim3 grid((unsigned)(((int64_t)a.tile0[a.k] * int8_tile(a.few) + kInt8Chunk - 1) / kInt8Chunk), a.B);
        if (a.ids)
            hipLaunchKernelGGL(int8_join_kernel<true>, grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL(int8_join_kernel<false>, grid, dim3(256), 0, s, a);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    }
    if (a.ids) {
        hipLaunchKernelGGL(int8_ids_kernel, dim3(a.B), dim3(kIdsThreads), 0, s, a);
        e = hipGetLastError();
    }
    return e;
}

int64_t int8_launch_items(bool few, int32_t B, int64_t tiles, int32_t slices)
{
    const int64_t rows = (int64_t)B * kIdsThreads;  // one workgroup per row
    if (few)
        return std::max(rows, tiles * slices * kRowsThreads);
    // the small tiles' launch holds twice the work items of the big ones'
    return std::max(rows, (tile_count(tile_grid<SmallTile>(B, tiles * kInt8LargeTile)) * slices + 8) * SmallTile::kThreads);
}

}  // namespace sbk
