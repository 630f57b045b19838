// The MFMA tile product of the loss, gradient and 8-bit kernels (gfx950).
//
// One workgroup computes a tile of C[m][n] = sum_k A[m][k] B[n][k]: 256 x 256 by
// 8 waves (BigTile), or 128 x 128 by 4 (SmallTile) where the big tiles would
// leave CUs idle or a product is so short that one tile's loads and stores have
// to run beside another's products: two small workgroups share a CU.
// Operands come in two layouts, either way without a copy in memory:
//   * kAlongK:   k contiguous, rows of the operand `ld` apart (X in X.W, both
//                operands of dZ.W^T, both int8 operands);
//   * kAcrossK:  rows of the operand contiguous, k steps `ld` apart (W in X.W,
//                both operands of X^T.dZ).
// K advances in stages of 128 bytes per row (64 bf16 or 128 int8) through LDS
// rings of three stages of A and two of B, filled by direct-to-LDS buffer
// loads of 1 KB.
//
// What bounds the big tile: a stage is 64 MFMAs per wave (2 x 8 x 4 blocks of 16 x 16 x
// 32 bf16), about 2048 cycles with two waves per SIMD, and 24 KB of fragment
// reads per wave, about 1536 cycles of the CU's LDS port.  They only overlap
// if a wave's reads run beside its own MFMAs, so each 32-deep half of a stage
// is computed while the other half's fragments arrive: the reads of half h + 1
// are issued between the MFMAs of half h.  The one barrier of a stage sits
// between its halves, where the wave already holds the second half in
// registers: behind it B's slot is free and is refilled two stages ahead, while
// A's third slot takes A's loads in the first half.  So four of a stage's eight
// loads per wave are issued in each half, spread over its MFMAs (eight in a
// row after the barrier hold the wave's MFMAs up while the CU's one address
// unit takes the 64 loads of its waves), and a load has at least most of a
// stage of time.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace sbk {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStageBytes = 128;       // K bytes of a row per stage
constexpr int kStageK = 64;            // bf16 K steps per stage

// WM x WN waves (rows x columns) of RB x CB blocks of 16 x 16.
template <int WM, int WN, int RB, int CB>
struct TileShape {
    static constexpr int kWM = WM, kWN = WN, kRB = RB, kCB = CB;
    static constexpr int kM = 16 * RB * WM, kN = 16 * CB * WN;
    static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int kABytes = kM * kStageBytes, kBBytes = kN * kStageBytes;  // a stage
    static constexpr int kALoads = kABytes / 1024 / kWaves, kBLoads = kBBytes / 1024 / kWaves;
    static constexpr int kLds = 3 * kABytes + 2 * kBBytes;
    static constexpr int kPerCu = kLds > 80 * 1024 ? 1 : 2;  // workgroups on a CU
};
typedef TileShape<2, 4, 8, 4> BigTile;    // 256 x 256, all 160 KB of LDS
typedef TileShape<2, 2, 4, 4> SmallTile;  // 128 x 128, half of it
static_assert(BigTile::kLds == 160 * 1024 && SmallTile::kLds == 80 * 1024, "LDS of a CU");

enum Layout : int { kAlongK = 0, kAcrossK = 1 };

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, int64_t bytes)
{
    const uint32_t n = bytes <= 0 ? 0u : (bytes >= 0xFFFFFFFFll ? 0xFFFFFFFFu : (uint32_t)bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)n,
                                             0x00020000);  // raw buffer, 32-bit data format
}

// Raises a kernel's dynamic-LDS limit on the current device, once per device
// (devices past 63 set it on every call; concurrent first calls may both).
inline hipError_t allow_lds(const void *kernel, int bytes, std::atomic<uint64_t> &done)
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

// ---------------------------------------------------------------------------
// Workgroup order.  Workgroup ids are handed to the 8 XCDs round-robin, so
// XCD x = id % 8 runs ids x, x + 8, ...  The tiles are numbered in bands of
// `pm` tile rows, column by column inside a band, and every XCD takes an equal
// run of consecutive numbers: the 32 tiles it runs at a time (one per CU) form
// a patch of about pm x (32 / pm) tiles, which share their operands' stages in
// the XCD's L2, and no XCD has more tiles than another.  A placement hint
// only: any bijection gives the same results.
// ---------------------------------------------------------------------------
struct TileGrid {
    int mt, nt;  // tiles in m and n
    int pm;      // tile rows of a band
};

template <class C>
inline TileGrid tile_grid(int64_t m, int64_t n)
{
    TileGrid g;
    g.mt = (int)((m + C::kM - 1) / C::kM);
    g.nt = (int)((n + C::kN - 1) / C::kN);
    g.pm = g.mt < 8 ? (g.mt > 0 ? g.mt : 1) : 8;
    return g;
}

inline int64_t tile_count(const TileGrid &g) { return (int64_t)g.mt * g.nt; }

// Workgroups of a launch over `tiles` tiles (up to 7 of them without one).
inline int64_t xcd_ids(int64_t tiles) { return (tiles + 7) / 8 * 8; }

// The tile number of workgroup `id`, or -1.
__device__ __forceinline__ int xcd_tile(int id, int tiles)
{
    const int per = (tiles + 7) / 8, t = (id & 7) * per + (id >> 3);
    return t < tiles ? t : -1;
}

__device__ __forceinline__ void tile_of(const TileGrid &g, int number, int &mt, int &nt)
{
    const int band = number / (g.pm * g.nt), r = number - band * (g.pm * g.nt);
    const int h = min(g.pm, g.mt - band * g.pm);
    mt = band * g.pm + r % h;
    nt = r / h;
}

// ---------------------------------------------------------------------------
// Stage layouts in LDS.
//   kAlongK:  row r at r * 128, its 16-byte piece p in slot p ^ ((r / 2) & 7):
//     the 16 rows of a fragment read (ds_read_b128) hit distinct banks.
//   kAcrossK: k step at k * 2 ROWS bytes, its 32-byte unit u (16 rows) in slot
//     u ^ across_swz(k): the 16 k steps of a transposing read
//     (ds_read_b64_tr_b16) hit distinct banks, in each half wave with 128 rows.
// ---------------------------------------------------------------------------
template <int ROWS>
__device__ __forceinline__ int across_swz(int k)
{
    static_assert(ROWS == 256 || ROWS == 128, "16 or 8 units of 32 bytes per k step");
    return (k & 3) | (((k >> 3) & (ROWS == 256 ? 3 : 1)) << 2);
}

// This wave's N loads of 1 KB of a stage of ROWS rows: byte offsets from the
// stage's base.
template <int LAYOUT, int ROWS, int N>
__device__ __forceinline__ void stage_offsets(uint32_t (&vo)[N], int wave, int L, int64_t ld_bytes)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int j = N * wave + i;
        if (LAYOUT == kAlongK) {
            const int r = 8 * j + (L >> 3);
            const int p = (L & 7) ^ ((r >> 1) & 7);
            vo[i] = (uint32_t)((int64_t)r * ld_bytes + 16 * p);
        } else {
            constexpr int lanes = ROWS / 8;  // of a k step
            const int k = (64 / lanes) * j + L / lanes;
            const int u = ((L % lanes) >> 1) ^ across_swz<ROWS>(k);
            vo[i] = (uint32_t)((int64_t)k * ld_bytes + 32 * u + 16 * (L & 1));
        }
    }
}

// 64 lanes' 16 bytes at offsets vo into 1 KB of LDS.
template <int POLICY = 0>
__device__ __forceinline__ void load_to_lds(uint8_t *lds, __amdgpu_buffer_rsrc_t r, uint32_t vo)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16, vo, 0, 0,
                                             POLICY);
}

template <int N>
__device__ __forceinline__ void stage_load(uint8_t *lds, __amdgpu_buffer_rsrc_t r,
                                           const uint32_t (&vo)[N], int wave)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        load_to_lds(lds + (N * wave + i) * 1024, r, vo[i]);
}

// Zero the K bytes at and past `kbytes` (< 128) of a kAlongK stage: what lies
// there in memory is a row's padding or the next row, which may be any bits.
template <int ROWS, int THREADS>
__device__ __forceinline__ void zero_stage_tail(uint8_t *lds, int kbytes)
{
    for (int idx = threadIdx.x; idx < ROWS * 8; idx += THREADS) {
        const int r = idx >> 3, p = idx & 7;
        if (16 * p + 16 <= kbytes)
            continue;
        uint8_t *piece = lds + r * kStageBytes + (p ^ ((r >> 1) & 7)) * 16;
        if (16 * p >= kbytes) {
            *reinterpret_cast<u32x4 *>(piece) = u32x4{0u, 0u, 0u, 0u};
        } else {
            for (int e = kbytes - 16 * p; e < 16; ++e)
                piece[e] = 0;
        }
    }
}

typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;

// Four 16-bit values of a column of the 4 x 16 block whose 16-byte row quarters
// the 16 lanes of a group point at.  The restrict pointer gives the read alias
// information of its own, without which the compiler makes it wait for every
// load into LDS that is in flight; run() orders the two itself.
__device__ __forceinline__ s16x4 read_across(lds_s16x4 __restrict p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}

// Fragment reader of NB 16-row blocks from operand row `row0` on (a multiple
// of 16 * NB) of ROWS rows: lane L gets row L % 16 of a block, K bytes 16 * (L
// / 16) .. of the half's 64.
template <int LAYOUT, int ROWS, int NB>
struct FragReader {
    uint32_t at;  // the lane's byte offset inside a stage, block 0, half 0

    __device__ __forceinline__ void init(int row0, int L)
    {
        const int n = L & 15, g = L >> 4;
        if (LAYOUT == kAlongK)
            at = (uint32_t)((row0 + n) * kStageBytes + ((g ^ ((n >> 1) & 7)) * 16));
        else  // k = 8 g + n / 4 (+ 4 for the second read), rows 4 (n % 4) .. + 3 of the block
            at = (uint32_t)((8 * g + (n >> 2)) * (2 * ROWS) +
                            (((row0 / 16) ^ across_swz<ROWS>(8 * g + (n >> 2))) * 32) + (n & 3) * 8);
    }
    __device__ __forceinline__ u32x4 read(const uint8_t *stage, int half, int block) const
    {
        if (LAYOUT == kAlongK)
            return *reinterpret_cast<const u32x4 *>(stage + (at ^ (uint32_t)(half * 64)) +
                                                    block * 16 * kStageBytes);
        // block < NB and row0 / 16 is a multiple of NB: the block number only
        // flips bits of the swizzled slot
        const uint8_t *p = stage + (at ^ (uint32_t)(block * 32)) + half * 32 * (2 * ROWS);
        const s16x4 lo = read_across((lds_s16x4)p);
        const s16x4 hi = read_across((lds_s16x4)(p + 4 * (2 * ROWS)));
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
        return u32x4{a[0], a[1], b[0], b[1]};
    }
};

// One 16 x 16 block step: 32 bf16 or 64 int8 K values.  The column operand
// goes first, so a lane holds four consecutive columns of one row.
__device__ __forceinline__ void block_mma(f32x4 &c, const u32x4 &row, const u32x4 &col)
{
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, col),
                                                __builtin_bit_cast(bf16x8, row), c, 0, 0, 0);
}
__device__ __forceinline__ void block_mma(i32x4 &c, const u32x4 &row, const u32x4 &col)
{
    c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, col),
                                              __builtin_bit_cast(i32x4, row), c, 0, 0, 0);
}

constexpr int kSchedMfma = 0x008, kSchedVmem = 0x010, kSchedDsRead = 0x100;

// The operand of s_waitcnt that waits for all but the wave's last n (< 64)
// vector memory operations, and for nothing else.
constexpr int vmcnt_only(int n) { return (n & 15) | ((n >> 4) << 14) | 0x0f70; }

// A workgroup barrier that no memory operation is moved across.  Unlike
// __syncthreads() it does not wait for loads into LDS that are still in flight.
__device__ __forceinline__ void block_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// This wave's LDS operations are done.
__device__ __forceinline__ void wait_lds()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
}

// The accumulators of a wave: acc[rb][cb] holds, for lane L, row 16 rb + L % 16
// and columns 16 cb + 4 (L / 16) .. + 3 of the wave's part of the tile.
template <class C, typename Acc>
struct WaveTile {
    static constexpr int kRB = C::kRB, kCB = C::kCB;
    Acc acc[kRB][kCB];
    int wave, L, row0, col0;  // the wave's first row and column inside the tile

    __device__ __forceinline__ void init()
    {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        L = threadIdx.x & 63;
        row0 = wave / C::kWN * (16 * kRB);
        col0 = wave % C::kWN * (16 * kCB);
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb)
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb)
                acc[rb][cb] = Acc{};
    }

    // Stages 0 .. nst - 1.  src.a(st) / src.b(st) give the buffers of stage st
    // (their base the stage's first K step; empty from nst on), called once
    // for each stage in ascending order; src.tail(st) the valid K bytes of
    // stage st (>= 128 where nothing has to be zeroed): the kAlongK operands
    // named by ZA / ZB are zeroed past it.  src.meanwhile() runs while the first
    // stages are on their way.
    template <int LA, int LB, bool ZA, bool ZB, typename Src>
    __device__ __forceinline__ void run(uint8_t *lds, int nst, int64_t lda_bytes, int64_t ldb_bytes,
                                        Src &src)
    {
        if (nst <= 0)
            return;
        uint32_t va[C::kALoads], vb[C::kBLoads];
        stage_offsets<LA, C::kM>(va, wave, L, lda_bytes);
        stage_offsets<LB, C::kN>(vb, wave, L, ldb_bytes);
        FragReader<LA, C::kM, kRB> ra;
        FragReader<LB, C::kN, kCB> rb_;
        ra.init(row0, L);
        rb_.init(col0, L);
        // A's ring of three slots, then B's of two
        uint8_t *const ringb = lds + 3 * C::kABytes;
        auto slot_b = [&](int st) { return ringb + (st & 1) * C::kBBytes; };
        auto mend = [&](int st, uint8_t *sa) {  // a stage whose K range ends inside it
            const int kb = src.tail(st);
            if (__builtin_expect(kb < kStageBytes, 0)) {
                if (ZA)
                    zero_stage_tail<C::kM, C::kThreads>(sa, kb);
                if (ZB)
                    zero_stage_tail<C::kN, C::kThreads>(slot_b(st), kb);
                wait_lds();
                block_barrier();
            }
        };
        stage_load(lds, src.a(0), va, wave);
        stage_load(slot_b(0), src.b(0), vb, wave);
        stage_load(lds + C::kABytes, src.a(1), va, wave);  // (empty where there is no stage 1)
        stage_load(slot_b(1), src.b(1), vb, wave);
        src.meanwhile();
        __builtin_amdgcn_s_waitcnt(vmcnt_only(C::kALoads + C::kBLoads));  // stage 0 has landed
        block_barrier();
        mend(0, lds);
        uint8_t *a0 = lds, *a1 = lds + C::kABytes, *a2 = lds + 2 * C::kABytes;  // stages st, st + 1, st + 2
        u32x4 fa[2][kRB], fb[2][kCB];
        read_half<LA, LB>(fa[0], fb[0], ra, rb_, a0, slot_b(0), 0);
        __amdgpu_buffer_rsrc_t next_a = src.a(2);
        for (int st = 0; st < nst; ++st) {
            // first half, beside A's loads of stage st + 2 and the reads of
            // the second half
            stage_load(a2, next_a, va, wave);
            read_half<LA, LB>(fa[1], fb[1], ra, rb_, a0, slot_b(st), 1);
            mma_half(fa[0], fb[0]);
            interleave<LA, LB>();
            const __amdgpu_buffer_rsrc_t next_b = src.b(st + 2);
            next_a = src.a(st + 3);
            // Stage st + 1 has landed (only A's loads of stage st + 2 are later)
            // and every wave holds the rest of this stage in registers.
            __builtin_amdgcn_s_waitcnt(vmcnt_only(C::kALoads) & ~0x0f00);  // and lgkmcnt(0)
            block_barrier();
            if (st + 1 < nst)
                mend(st + 1, a1);
            // second half, beside B's loads of stage st + 2 and the reads of
            // the next stage's first half (past the last stage: never used)
            stage_load(slot_b(st), next_b, vb, wave);
            read_half<LA, LB>(fa[0], fb[0], ra, rb_, a1, slot_b(st + 1), 0);
            mma_half(fa[1], fb[1]);
            interleave<LA, LB>();
            uint8_t *const free_slot = a0;
            a0 = a1;
            a1 = a2;
            a2 = free_slot;
        }
        __builtin_amdgcn_s_waitcnt(0x0070);
        __syncthreads();  // LDS is the caller's
    }

    // The wave's part as bf16 rows, by way of a private 128 bytes of LDS per row:
    // a lane's four columns would be stored as 32-byte pieces of 16 rows, these
    // are whole 128-byte runs of 8 rows.  put() all of it (after run()), then
    // flush(): store(row, column, 8 values) inside the tile.
    __device__ __forceinline__ void put(uint8_t *lds, int rb, int cb, uint2 bits) const
    {
        static_assert(kCB == 4, "64 columns of a wave are 128 bytes");
        const int n = L & 15, p = 2 * cb + (L >> 5);
        *reinterpret_cast<uint2 *>(lds + (wave * 16 * kRB + 16 * rb + n) * 128 + ((p ^ (n & 7)) * 16) +
                                   8 * ((L >> 4) & 1)) = bits;
    }
    template <typename Store>
    __device__ __forceinline__ void flush(const uint8_t *lds, Store store) const
    {
        wait_lds();
#pragma unroll
        for (int i = 0; i < 2 * kRB; ++i) {
            const int r = 8 * i + (L >> 3), p = L & 7;
            store(row0 + r, col0 + 8 * p,
                  *reinterpret_cast<const u32x4 *>(lds + (wave * 16 * kRB + r) * 128 + ((p ^ (r & 7)) * 16)));
        }
    }

private:
    template <int LA, int LB>
    static __device__ __forceinline__ void read_half(u32x4 (&fa)[kRB], u32x4 (&fb)[kCB],
                                                     const FragReader<LA, C::kM, kRB> &ra,
                                                     const FragReader<LB, C::kN, kCB> &rb_,
                                                     const uint8_t *sa, const uint8_t *sb, int half)
    {
#pragma unroll
        for (int cb = 0; cb < kCB; ++cb)
            fb[cb] = rb_.read(sb, half, cb);
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb)
            fa[rb] = ra.read(sa, half, rb);
    }
    __device__ __forceinline__ void mma_half(const u32x4 (&fa)[kRB],
                                             const u32x4 (&fb)[kCB])
    {
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb)
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb)
                block_mma(acc[rb][cb], fa[rb], fb[cb]);
    }
    // Asks the scheduler to spread a half's loads and its LDS reads over
    // its MFMAs.
    template <int LA, int LB>
    static __device__ __forceinline__ void interleave()
    {
        constexpr int reads = kRB * (LA == kAcrossK ? 2 : 1) + kCB * (LB == kAcrossK ? 2 : 1);
        constexpr int per = (reads + kRB - 1) / kRB;
#pragma unroll
        for (int i = 0; i < kRB; ++i) {
            if (i < C::kALoads)
                __builtin_amdgcn_sched_group_barrier(kSchedVmem, 1, 0);
            __builtin_amdgcn_sched_group_barrier(kSchedDsRead, per, 0);
            __builtin_amdgcn_sched_group_barrier(kSchedMfma, kCB, 0);
        }
    }
};

}  // namespace
}  // namespace sbk
