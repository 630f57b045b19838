// Device helpers shared by libsb's HIP sources: vector types, buffer
// resources and loads, the argmax order, DPP reductions over a wave, the
// workgroup order over the XCDs, and the LDS limit of large launches.
#pragma once

#include "kernels.h"

#include <atomic>

#include <float.h>
#include <limits.h>

namespace sbk {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = kWaves * 64;
constexpr uint32_t kRsrcWord3 = 0x00020000u;  // gfx9 raw buffer: 32-bit data format

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *base, int64_t bytes)
{
    uint32_t n = bytes <= 0 ? 0u : (bytes >= 0xFFFFFFFFll ? 0xFFFFFFFFu : (uint32_t)bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)n,
                                             (int)kRsrcWord3);
}

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t voff)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, 0, 0));
}

// Cache policy of the weight loads: kPolicyStream marks them non-temporal
// (each weight byte is read by one workgroup only and should not displace
// the hidden rows, which every workgroup re-reads); kPolicyShared keeps the
// default policy, for tiles that several row groups read through the L2.
constexpr int kPolicyShared = 0;
constexpr int kPolicyStream = 2;  // the nt bit of the buffer instruction

template <int POL>
__device__ __forceinline__ u32x4 load16w(__amdgpu_buffer_rsrc_t r, uint32_t voff)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, 0, POL));
}

// Raises a kernel's dynamic-LDS limit on the current device, once per device
// (the attribute is held per device; devices past 63 set it on every call).
// Concurrent first calls may both set it, which is harmless.
static hipError_t raise_lds_limit(const void *kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit))
        return hipSuccess;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess && bit)
        done.fetch_or(bit, std::memory_order_release);
    return e;
}

// The order of the argmax over (value, index): NaN above every number (the
// convention of numpy's and torch's argmax), then the order of the floats
// (+inf above every finite value, -0 equal to +0), and between equal values
// -- all NaNs count as equal -- the lower index.  It is a total order, so
// the result does not depend on the order of the fold, and every row's ID is
// one of its columns whatever its values.
__device__ __forceinline__ bool better(float v1, int i1, float v2, int i2)
{
    const bool n1 = v1 != v1, n2 = v2 != v2;
    if (n1 || n2)
        return n1 && (!n2 || i1 < i2);
    return v1 > v2 || (v1 == v2 && i1 < i2);
}

// better() for a candidate whose index is higher than the current best's.
__device__ __forceinline__ bool above(float v, float best)
{
    return v > best || (v != v && best == best);
}

// The same order on values known to hold no NaN: one compare.  The head
// epilogues use it unless a wave finds a NaN among its values (any_nan8).
__device__ __forceinline__ bool better_num(float v1, int i1, float v2, int i2)
{
    return v1 > v2 || (v1 == v2 && i1 < i2);
}

// Whether any of eight values is NaN: a NaN-propagating maximum of all of
// them (v_maximum3_f32, four instructions) compared with itself.
__device__ __forceinline__ bool any_nan8(float a, float b, float c, float d, float e, float f,
                                         float g, float h)
{
    const float m = __builtin_elementwise_maximum(
        __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c),
        __builtin_elementwise_maximum(__builtin_elementwise_maximum(d, e),
                                      __builtin_elementwise_maximum(__builtin_elementwise_maximum(f, g), h)));
    return m != m;
}

// Online logsumexp merge of (m2, s2) into (m1, s1); -inf marks "empty".
__device__ __forceinline__ void lse_merge(float &m1, float &s1, float m2, float s2)
{
    if (m2 == -INFINITY)
        return;
    if (m1 == -INFINITY) {
        m1 = m2;
        s1 = s2;
        return;
    }
    if (m2 > m1) {
        s1 = s1 * __expf(m1 - m2) + s2;
        m1 = m2;
    } else {
        s1 = s1 + s2 * __expf(m2 - m1);
    }
}

// Cross-lane reductions inside the 16-lane rows of a wave use DPP moves (a
// VALU operand modifier: no LDS traffic, no address registers).  Four steps
// pair each lane with one in the other half of a group of 2, 4, 8 and 16
// lanes: quad swaps by 1 and by 2, then the mirror of each 8-lane half and of
// the 16-lane row.  Both reductions below are symmetric in their two
// operands (floating-point addition commutes; the (max, lowest index) choice
// is a total order), so every lane of a row ends with the same bits.
constexpr int kDppQuadXor1 = 0xB1;     // quad_perm [1, 0, 3, 2]
constexpr int kDppQuadXor2 = 0x4E;     // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;  // lane i <- lane 7 - i of its 8-lane half
constexpr int kDppMirror = 0x140;      // lane i <- lane 15 - i of its row

template <int CTRL>
__device__ __forceinline__ int dpp_int(int v)
{
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, false);
}

template <int CTRL>
__device__ __forceinline__ float dpp_float(float v)
{
    return __int_as_float(dpp_int<CTRL>(__float_as_int(v)));
}

template <int CTRL, bool NAN_AWARE>
__device__ __forceinline__ void best_step(float &bv, int &bi)
{
    const float ov = dpp_float<CTRL>(bv);
    const int oi = dpp_int<CTRL>(bi);
    if (NAN_AWARE ? better(ov, oi, bv, bi) : better_num(ov, oi, bv, bi)) {
        bv = ov;
        bi = oi;
    }
}

// (max, lowest index) over each 16-lane row; every lane gets its row's.
// NAN_AWARE = false only where the wave holds no NaN.
template <bool NAN_AWARE = true>
__device__ __forceinline__ void row16_best(float &bv, int &bi)
{
    best_step<kDppQuadXor1, NAN_AWARE>(bv, bi);
    best_step<kDppQuadXor2, NAN_AWARE>(bv, bi);
    best_step<kDppHalfMirror, NAN_AWARE>(bv, bi);
    best_step<kDppMirror, NAN_AWARE>(bv, bi);
}

// The (max, lowest index) of each 16-lane row of a head epilogue, over the
// eight values y0..y7 of each thread at global columns gcol.. (the first
// nvalid of them real columns): the plain comparison, or, when any value
// of the wave is NaN, the NaN-aware order.  The branch is uniform over the
// wave, so the DPP steps see every lane of their rows.
__device__ __forceinline__ void tile_best(float y0, float y1, float y2, float y3, float y4,
                                          float y5, float y6, float y7, int nvalid, int gcol,
                                          float &bv, int &bi)
{
    const float y[8] = {y0, y1, y2, y3, y4, y5, y6, y7};
    bv = -INFINITY;
    bi = INT_MAX;
    if (nvalid > 0) {
        bv = y[0];
        bi = gcol;
    }
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(any_nan8(y0, y1, y2, y3, y4, y5, y6, y7)) == 0,
                         1)) {
#pragma unroll
        for (int j = 1; j < 8; ++j)
            if (j < nvalid && y[j] > bv) {
                bv = y[j];
                bi = gcol + j;
            }
        row16_best<false>(bv, bi);
    } else {
#pragma unroll
        for (int j = 1; j < 8; ++j)
            if (j < nvalid && above(y[j], bv)) {
                bv = y[j];
                bi = gcol + j;
            }
        row16_best<true>(bv, bi);
    }
}

// Sum over each 16-lane row; every lane gets its row's.
__device__ __forceinline__ float row16_sum(float v)
{
    v += dpp_float<kDppQuadXor1>(v);
    v += dpp_float<kDppQuadXor2>(v);
    v += dpp_float<kDppHalfMirror>(v);
    v += dpp_float<kDppMirror>(v);
    return v;
}

template <int CTRL>
__device__ __forceinline__ void lse_step(float &m, float &s)
{
    lse_merge(m, s, dpp_float<CTRL>(m), dpp_float<CTRL>(s));
}

// Over the whole wave: the rows by DPP, then the four row results (lanes 0,
// 16, 32, 48) read as wave-uniform values and merged in row order.
__device__ __forceinline__ void wave_best(float &bv, int &bi)
{
    row16_best(bv, bi);
    float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bv), 0));
    int i = __builtin_amdgcn_readlane(bi, 0);
#pragma unroll
    for (int r = 1; r < 4; ++r) {
        const float ov = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bv), 16 * r));
        const int oi = __builtin_amdgcn_readlane(bi, 16 * r);
        if (better(ov, oi, v, i)) {
            v = ov;
            i = oi;
        }
    }
    bv = v;
    bi = i;
}

// Online logsumexp (m, s) over the whole wave, as wave_best.
__device__ __forceinline__ void wave_lse(float &m, float &s)
{
    lse_step<kDppQuadXor1>(m, s);
    lse_step<kDppQuadXor2>(m, s);
    lse_step<kDppHalfMirror>(m, s);
    lse_step<kDppMirror>(m, s);
    float wm = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(m), 0));
    float ws = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s), 0));
#pragma unroll
    for (int r = 1; r < 4; ++r)
        lse_merge(wm, ws, __int_as_float(__builtin_amdgcn_readlane(__float_as_int(m), 16 * r)),
                  __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s), 16 * r)));
    m = wm;
    s = ws;
}

struct LargeGrid {
    int mblocks;  // ceil(B / block rows)
    int sm;       // m-blocks per super-tile (8, 4 or 2), or 0 for the plain order
    int nblocks;  // total 256-column blocks over all lanes
};

// Workgroups per super-tile of the XCD-aware order: as many as an XCD has CUs.
constexpr int kSuperWG = 32;

// Super-tile rows for a batch of `mblocks` 256-row blocks: 8 from 8 m-blocks
// up, 4 or 2 for exactly that many, else 0 (plain order).  Timed with
// bench.py on batches of 1 to 8 m-blocks: the super-tiles gained 2-5 % at 2
// and 4 m-blocks, lost up to 1.5 % at 3, and grouping 3, 5, 6 or 7 m-blocks
// into half-empty groups of 2 or 4 lost 15-28 %.
inline __host__ __device__ int super_rows(int mblocks)
{
    return mblocks >= 8 ? 8 : (mblocks == 4 || mblocks == 2 ? mblocks : 0);
}

// Workgroup id -> (m-block, n-block).  The blocks form super-tiles of sm
// m-blocks x kSuperWG / sm n-blocks (8 x 4 from 8 m-blocks up).  XCD x = id
// % 8 (workgroups are handed to the XCDs round-robin) takes super-tiles x,
// x+8, ..., so the 32 workgroups an XCD runs at a time read each K stage's
// hidden-row and weight slabs through its own L2: with 8 x 4, 384 KB per
// stage from beyond the L2 instead of the 1.06 MB that 32 n-blocks of one
// m-block need.  Without super-tiles the m-blocks of one n-block are
// consecutive.  A placement hint only: any bijection gives the same results.
__device__ __forceinline__ bool large_block(const LargeGrid &g, int id, int &mb, int &nb)
{
    if (g.sm > 0) {
        const int sn = kSuperWG / g.sm;
        const int mgroups = (g.mblocks + g.sm - 1) / g.sm;
        const int xcd = id & 7, local = id >> 3;
        const int st = (local / kSuperWG) * 8 + xcd, w = local % kSuperWG;
        mb = (st % mgroups) * g.sm + w % g.sm;
        nb = (st / mgroups) * sn + w / g.sm;
    } else {
        mb = id % g.mblocks;
        nb = id / g.mblocks;
    }
    return mb < g.mblocks && nb < g.nblocks;
}

// Workgroups of a large-batch launch over mblocks x nblocks blocks: in the
// super-tile order, whole super tiles, and a multiple of 8 of them.
inline int64_t large_workgroups(int mblocks, int64_t nblocks)
{
    const int sm = super_rows(mblocks);
    if (sm == 0)
        return (int64_t)mblocks * nblocks;
    const int sn = kSuperWG / sm;
    const int64_t supers = (int64_t)((mblocks + sm - 1) / sm) * ((nblocks + sn - 1) / sn);
    return (supers + 7) / 8 * 8 * kSuperWG;
}

}  // namespace
}  // namespace sbk
