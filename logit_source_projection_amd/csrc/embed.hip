// Embedding lookup and its gradient (gfx950).
//
//   out_b = scale table[ids_b]                    (0 for ids_b < 0, NaN for ids_b >= V)
//   dtable_v = scale sum_{b: ids_b = v} dout_b    (IDs outside 0 .. V - 1 add nothing)
//
// The gradient's sums run over positions sorted by their IDs, in an order fixed
// by the IDs alone: no atomics on values, so repeated calls give the same bits.
#include "embed.h"

#include <algorithm>

#include "values.h"

namespace sbk {
namespace {

constexpr int kThreads = 256;
constexpr int kUnitColumns = 8 * kThreads;  // columns that a workgroup takes at a time
constexpr int64_t kMostGroups = 1 << 20;    // workgroups along x

// The row of a table that ID v (0 .. V - 1) names.
template <typename T>
__device__ __forceinline__ T *table_row(const EmbedArgs &a, int v)
{
    int lo = 0, hi = a.k;  // off[lo] <= v < off[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.off[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return static_cast<T *>(a.w[lo]) + (int64_t)(v - a.off[lo]) * a.ldw;
}

// ---------------------------------------------------------------------------
// Lookup: one workgroup per row.
// ---------------------------------------------------------------------------
template <typename TT, typename TO>
__global__ __launch_bounds__(kThreads) void embed_kernel(const EmbedArgs a)
{
    const int H = a.H;
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int id = __builtin_amdgcn_readfirstlane(a.ids[b]);
        TO *out = static_cast<TO *>(a.out) + b * a.ldo;
        const bool there = (uint32_t)id < (uint32_t)a.V;
        const TT *row = there ? table_row<TT>(a, id) : nullptr;
        const float other = id < 0 ? 0.f : NAN;
        for (int c = 8 * threadIdx.x; c < H; c += kUnitColumns) {
            float v[8];
            if (there)
                values_of(load_some(row + c, H - c), v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = there ? v[e] * a.scale : other;
            store_some(out + c, v, H - c);
        }
    }
}

// ---------------------------------------------------------------------------
// Positions sorted by their IDs, equal ones ascending, in one launch without a
// word between workgroups: each takes a range of IDs and reads all of `ids`
// twice (from the L2; 64 KB for 16384 tokens).  The first pass counts the IDs
// below its range, which is where its own positions start, and those of every ID
// in it; the second compacts the range's positions in order, a chunk at a time,
// and places them behind the earlier ones of their ID.  In a chunk wave w places
// the IDs that are w modulo 16, 64 entries at a time, all equal ones at once: a
// token that fills the batch is as quick as one that comes once.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortEach = 4;                              // IDs per thread and chunk
constexpr int kSortChunk = kSortThreads * kSortEach;
constexpr int kSortRange = 4096;                          // IDs per workgroup at most
constexpr int kSortGroups = 256;                          // workgroups where ranges allow

inline int sort_range(int V)
{
    return std::min(kSortRange, (V + kSortGroups - 1) / kSortGroups);
}

__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(const EmbedArgs a, int range)
{
    __shared__ int32_t next[kSortRange];        // counts, then where an ID's next position goes
    __shared__ int2 list[kSortChunk];           // {ID - lo, position} of the chunk
    __shared__ int32_t sums[kSortWaves];
    const int lo = blockIdx.x * range, n = min(range, a.V - lo);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int i = threadIdx.x; i < n; i += kSortThreads)
        next[i] = 0;
    __syncthreads();
    int below = 0;
    for (int b = threadIdx.x; b < a.B; b += kSortThreads) {
        const int id = a.ids[b];
        below += (uint32_t)id < (uint32_t)lo;
        const uint32_t at = (uint32_t)id - (uint32_t)lo;
        if (at < (uint32_t)n)
            atomicAdd(&next[at], 1);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        below += __shfl_xor(below, d);
    if (lane == 0)
        sums[wave] = below;
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w)
        base += sums[w];
    // counts to starting places, 64 IDs at a time by the first wave
    if (wave == 0) {
        for (int i0 = 0; i0 < n; i0 += 64) {
            const int i = i0 + lane, count = i < n ? next[i] : 0;
            int upto = count;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int v = __shfl_up(upto, d);
                upto += lane >= d ? v : 0;
            }
            if (i < n) {
                next[i] = base + upto - count;
                if (!a.add)
                    a.start[lo + i] = base + upto - count;
            }
            base += __shfl(upto, 63);
        }
        if (lane == 0 && lo + n == a.V)
            a.start[a.add ? 0 : a.V] = base;
    }
    for (int b0 = 0; b0 < a.B; b0 += kSortChunk) {
        // wave w compacts the chunk's IDs [256 w, 256 w + 256)
        int id[kSortEach], mine = 0;
        uint64_t hit[kSortEach];
#pragma unroll
        for (int i = 0; i < kSortEach; ++i) {
            const int b = b0 + (wave * kSortEach + i) * 64 + lane;
            id[i] = b < a.B ? (int)((uint32_t)a.ids[b] - (uint32_t)lo) : -1;
            hit[i] = __ballot((uint32_t)id[i] < (uint32_t)n);
            mine += __popcll(hit[i]);
        }
        __syncthreads();  // `sums` and the list are free, `next` is whole
        if (lane == 0)
            sums[wave] = mine;
        __syncthreads();
        int at = 0, entries = 0;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            at += w < wave ? sums[w] : 0;
            entries += sums[w];
        }
#pragma unroll
        for (int i = 0; i < kSortEach; ++i) {
            if (hit[i] >> lane & 1)
                list[at + __popcll(hit[i] & (((uint64_t)1 << lane) - 1))] =
                    make_int2(id[i], b0 + (wave * kSortEach + i) * 64 + lane);
            at += __popcll(hit[i]);
        }
        __syncthreads();
        for (int e0 = 0; e0 < entries; e0 += 64) {
            const int2 entry = e0 + lane < entries ? list[e0 + lane] : make_int2(-1, 0);
            uint64_t todo = __ballot(entry.x >= 0 && entry.x % kSortWaves == wave);
            while (todo) {
                const int one = __builtin_amdgcn_readlane(entry.x, __builtin_ctzll(todo));
                const uint64_t same = __ballot(entry.x == one);
                const int place = next[one];
                if (entry.x == one) {
                    const int p = place + __popcll(same & (((uint64_t)1 << lane) - 1));
                    a.order[p] = entry.y;
                    a.sorted[p] = lo + one;
                }
                next[one] = place + __popcll(same);  // (by every lane: the next read is its own)
                todo &= ~same;
            }
        }
    }
}

// Rows without a position are zeros.
template <typename T>
__global__ __launch_bounds__(kThreads) void embed_zero_kernel(const EmbedArgs a)
{
    const float zeros[8] = {};
    for (int v = blockIdx.x; v < a.V; v += gridDim.x) {
        if (a.start[v] != a.start[v + 1])
            continue;
        T *row = table_row<T>(a, v);
        for (int c = 8 * threadIdx.x; c < a.H; c += kUnitColumns)
            store_some(row + c, zeros, a.H - c);
    }
}

template <typename T>
__device__ __forceinline__ void store_row(const EmbedArgs &a, int id, int c, const float (&sum)[8])
{
    T *to = table_row<T>(a, id) + c;
    const int n = a.H - c;
    float v[8];
    if (a.add) {
        values_of(load_some(to, n), v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] += a.scale * sum[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = a.scale * sum[e];
    }
    store_some(to, v, n);
}

// ---------------------------------------------------------------------------
// Sums of runs of kEmbedRun sorted positions, a unit of columns per thread.  An
// ID whose positions all lie in the run is done here; the sums of one that came
// from the run before go to the run's first partial row, of one that starts here
// and goes on to its second.
// ---------------------------------------------------------------------------
template <typename TT, typename TO>
__global__ __launch_bounds__(kThreads) void embed_runs_kernel(const EmbedArgs a)
{
    const int c = blockIdx.y * kUnitColumns + 8 * threadIdx.x;
    const int total = a.start[a.add ? 0 : a.V];
    const int run = blockIdx.x, p0 = run * kEmbedRun, p1 = min(p0 + kEmbedRun, total);
    if (c >= a.H || p0 >= p1)
        return;
    float sum[8] = {};
    bool begins = p0 == 0 || a.sorted[p0 - 1] != a.sorted[p0];
    for (int p = p0; p < p1; ++p) {
        const int id = a.sorted[p];
        float v[8];
        values_of(load_some(static_cast<const TO *>(a.dout) + (int64_t)a.order[p] * a.lddo + c, a.H - c), v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum[e] += v[e];
        const bool ends = p + 1 == total || a.sorted[p + 1] != id;
        if (!ends && p + 1 < p1)
            continue;
        if (begins && ends)
            store_row<TT>(a, id, c, sum);
        else
            store_some(a.part + (2 * (int64_t)run + begins) * a.ldpart + c, sum, 8);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum[e] = 0.f;
        begins = true;
    }
}

// IDs whose positions span runs: the workgroup of the run that they start in adds
// the partial rows in order.
template <typename TT>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(const EmbedArgs a)
{
    const int c = blockIdx.y * kUnitColumns + 8 * threadIdx.x;
    const int total = a.start[a.add ? 0 : a.V];
    const int run = blockIdx.x;
    int p1 = (run + 1) * kEmbedRun;
    if (c >= a.H || p1 >= total)
        return;
    const int id = a.sorted[p1];
    // it goes on behind this run, and did not come from the one before
    if (a.sorted[p1 - 1] != id || (run > 0 && a.sorted[p1 - kEmbedRun - 1] == id))
        return;
    float sum[8], v[8];
    values_of(load_unit(a.part + (2 * (int64_t)run + 1) * a.ldpart + c), sum);
    for (int r = run + 1; p1 < total && a.sorted[p1] == id; ++r, p1 += kEmbedRun) {
        values_of(load_unit(a.part + 2 * (int64_t)r * a.ldpart + c), v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum[e] += v[e];
    }
    store_row<TT>(a, id, c, sum);
}

template <typename TT, typename TO>
hipError_t lookup(const EmbedArgs &a, hipStream_t s)
{
    const unsigned rows = (unsigned)std::min<int64_t>(a.B, kMostGroups);
    hipLaunchKernelGGL((embed_kernel<TT, TO>), dim3(rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

template <typename TT, typename TO>
hipError_t sums(const EmbedArgs &a, hipStream_t s)
{
    hipError_t e;
    if (!a.add) {
        const unsigned rows = (unsigned)std::min<int64_t>(a.V, kMostGroups);
        hipLaunchKernelGGL((embed_zero_kernel<TT>), dim3(rows), dim3(kThreads), 0, s, a);
        if ((e = hipGetLastError()) != hipSuccess || a.B == 0)
            return e;
    }
    const dim3 grid((unsigned)a.runs, (unsigned)((a.H + kUnitColumns - 1) / kUnitColumns));
    hipLaunchKernelGGL((embed_runs_kernel<TT, TO>), grid, dim3(kThreads), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess || a.runs < 2)
        return e;
    hipLaunchKernelGGL((embed_join_kernel<TT>), dim3(grid.x - 1, grid.y), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_embed(const EmbedArgs &a, hipStream_t s)
{
    if (a.table_bf16)
        return a.rows_bf16 ? lookup<bf16_t, bf16_t>(a, s) : lookup<bf16_t, float>(a, s);
    return a.rows_bf16 ? lookup<float, bf16_t>(a, s) : lookup<float, float>(a, s);
}

hipError_t launch_embed_sort(const EmbedArgs &a, hipStream_t s)
{
    const int range = sort_range(a.V);
    hipLaunchKernelGGL(embed_sort_kernel, dim3((unsigned)((a.V + range - 1) / range)), dim3(kSortThreads), 0, s, a, range);
    return hipGetLastError();
}

hipError_t launch_embed_sums(const EmbedArgs &a, hipStream_t s)
{
    if (a.table_bf16)
        return a.rows_bf16 ? sums<bf16_t, bf16_t>(a, s) : sums<bf16_t, float>(a, s);
    return a.rows_bf16 ? sums<float, bf16_t>(a, s) : sums<float, float>(a, s);
}

}  // namespace sbk
