// Embedding lookup and its gradient (gfx950).
//
//   out_b = scale table[ids_b]                    (0 for ids_b < 0, NaN for ids_b >= V)
//   dtable_v = scale sum_{b: ids_b = v} dout_b    (IDs outside 0 .. V - 1 add nothing)
//
// The gradient's sums run over positions sorted by their IDs, in an order fixed
// by the IDs alone: no atomics on values, so repeated calls give the same bits.
#include "embed.h"

#include <algorithm>

#include "tile_gemm.h"
#include "values.h"

namespace sbk {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMostGroups = 1 << 20; // workgroups along x

// Threads for rows of H columns, 8 to each: a row in equal parts of up to kThreads
// threads, so that few are idle.
inline int row_threads(int H)
{
    const int units = std::max(1, (H + 7) / 8), parts = (units + kThreads - 1) / kThreads;
    return std::max(64, ((units + parts - 1) / parts + 63) / 64 * 64);
}

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
    return in_memory(static_cast<T *>(a.w[lo])) + (int64_t)(v - a.off[lo]) * a.ldw;
}

// ---------------------------------------------------------------------------
// Lookup: `team` threads per row (a power of two up to 32, or the workgroup).
// ---------------------------------------------------------------------------
constexpr int kLookupUnits = 4;  // loads of a thread under way

template <typename TT, typename TO>
__global__ __launch_bounds__(kThreads) void embed_kernel(const EmbedArgs a, int team)
{
    const int H = a.H, at = threadIdx.x % team, teams = blockDim.x / team;
    for (int64_t b = (int64_t)blockIdx.x * teams + threadIdx.x / team; b < a.B; b += (int64_t)gridDim.x * teams) {
        int id = a.ids[b];
        if (teams == 1)
            id = __builtin_amdgcn_readfirstlane(id);
        TO *out = static_cast<TO *>(a.out) + b * a.ldo;
        const bool there = (uint32_t)id < (uint32_t)a.V;
        const TT *row = table_row<const TT>(a, there ? id : 0);
        const float other = id < 0 ? 0.f : NAN;
        for (int c0 = 8 * at; c0 < H; c0 += 8 * kLookupUnits * team) {
            Unit<TT> raw[kLookupUnits];
#pragma unroll
            for (int k = 0; k < kLookupUnits; ++k)
                raw[k] = load_at(row, c0 + 8 * k * team, H);
#pragma unroll
            for (int k = 0; k < kLookupUnits; ++k) {
                const int c = c0 + 8 * k * team;
                float v[8];
                values_of(raw[k], v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = there ? v[e] * a.scale : other;
                if (c < H)
                    store_some(out + c, v, H - c);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Positions sorted by ID, equal ones ascending, in one launch without a word
// between workgroups.  Workgroup g takes the IDs that are g modulo the number of groups (so that
// neighbouring IDs, which often come together, are spread) and reads all of `ids`
// (from the L2; 64 KB for 16384 tokens).  A first pass counts the IDs of the groups
// before, which is where its own positions start, and those of every ID of its own; a
// second compacts its positions in order, a chunk at a time, and places them behind
// the earlier ones of their ID.  Up to a chunk of IDs stay in registers between the
// passes.  In a chunk wave w places the IDs whose number in the group is w modulo 16,
// 64 entries at a time, all equal ones at once.  An ID of a 32nd of all tokens or
// more (padding that is not negative, say) is placed by the whole workgroup instead,
// straight from the registers: 16384 equal tokens took 70 us in one wave's hands.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortEach = 16;                             // IDs per thread and chunk at most
constexpr int kSortChunk = kSortThreads * kSortEach;      // 2^14
constexpr int kSortRange = 4096;                          // IDs per workgroup at most
constexpr int kSortNeighbours = kSortRange / kSortThreads;
constexpr int kSortHot = 32;                              // IDs that may be this share of all

// The place of an ID in `start`.
__device__ __forceinline__ int embed_slot(const EmbedArgs &a, uint32_t v)
{
    return (int)(v & ((1u << a.shift) - 1)) * a.range + (int)(v >> a.shift);
}

// The IDs of a chunk, 64 neighbours to a wave's load: their number in the group, or
// kSortOther of another group's; `before` counts those of groups before this one.
constexpr uint32_t kSortOther = 0xFFFFFFFFu;

template <int EACH>
__device__ __forceinline__ int sort_place(int b0, int k)
{
    return b0 + ((threadIdx.x >> 6) * EACH + k) * 64 + (threadIdx.x & 63);
}

template <int EACH>
__device__ __forceinline__ void sort_load(const EmbedArgs &a, int b0, uint32_t (&id)[EACH], int &before)
{
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int b = sort_place<EACH>(b0, k);
        id[k] = b < a.B ? (uint32_t)a.ids[b] : kSortOther;
    }
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const uint32_t group = id[k] & ((1u << a.shift) - 1);
        const bool there = id[k] < (uint32_t)a.V;
        before += there && group < blockIdx.x;
        id[k] = there && group == blockIdx.x ? id[k] >> a.shift : kSortOther;
    }
}

// EACH: IDs per thread and chunk.  One, for up to 1024 tokens, has no ID that is hot.
template <int EACH>
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(const EmbedArgs a)
{
    constexpr int kChunk = kSortThreads * EACH;
    extern __shared__ int32_t smem[];
    int32_t *next = smem;                     // counts, then where an ID's next position goes
    uint32_t *list = reinterpret_cast<uint32_t *>(smem + kSortRange);  // number << 14 | place in the chunk
    __shared__ int32_t sums[kSortWaves], hot[kSortHot], hots;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, range = a.range;
    int before = 0, none = 0;
    uint32_t id[EACH];
    sort_load(a, 0, id, before);
    for (int i = threadIdx.x; i < range; i += kSortThreads)
        next[i] = 0;
    if (threadIdx.x == 0)
        hots = 0;
    __syncthreads();
    for (int b0 = 0; b0 < a.B; b0 += kChunk) {
        if (b0 > 0)
            sort_load(a, b0, id, before);
#pragma unroll
        for (int k = 0; k < EACH; ++k)
            if (id[k] != kSortOther)
                atomicAdd(&next[id[k]], 1);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        before += __shfl_xor(before, d);
    if (lane == 0)
        sums[wave] = before;
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w)
        base += sums[w];
    // counts to starting places, kSortNeighbours neighbours per thread
    const int most = max(kSortThreads, a.B / kSortHot);
    int count[kSortNeighbours], upto = 0;
#pragma unroll
    for (int e = 0; e < kSortNeighbours; ++e) {
        const int i = kSortNeighbours * threadIdx.x + e;
        count[e] = i < range ? next[i] : 0;
        upto += count[e];
        if (count[e] > most)  // (fewer than kSortHot IDs have so many)
            hot[atomicAdd(&hots, 1)] = i;
    }
    const int own = upto;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        upto += lane >= d ? v : 0;
    }
    __syncthreads();  // `sums` has been read
    if (lane == 63)
        sums[wave] = upto;
    __syncthreads();
    base += upto - own;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w)
        base += w < wave ? sums[w] : 0;
#pragma unroll
    for (int e = 0; e < kSortNeighbours; ++e) {
        const int i = kSortNeighbours * threadIdx.x + e;
        if (i < range) {
            next[i] = a.start[blockIdx.x * range + i] = base;
            base += count[e];
            if (i == range - 1 && blockIdx.x + 1 == gridDim.x)
                a.start[range << a.shift] = base;
        }
    }
    // Where this wave's hits of a chunk start among the workgroup's, and all of them.
    // (The first barrier also makes `next` whole, and the second the list free.)
    auto places = [&](int mine, int &all) {
        __syncthreads();
        if (lane == 0)
            sums[wave] = mine;
        __syncthreads();
        int at = 0;
        all = 0;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            at += w < wave ? sums[w] : 0;
            all += sums[w];
        }
        return at;
    };
    const uint64_t earlier = ((uint64_t)1 << lane) - 1;
    for (int b0 = 0; b0 < a.B; b0 += kChunk) {
        if (a.B > kChunk)
            sort_load(a, b0, id, none);
        for (int h = 0; EACH > 1 && h < hots; ++h) {
            const int one = hot[h];
            int mine = 0, all;
#pragma unroll
            for (int k = 0; k < EACH; ++k)
                mine += __popcll(__ballot(id[k] == (uint32_t)one));
            int p = places(mine, all);
            p += next[one];  // (behind the barriers that make it whole)
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                const uint64_t hit = __ballot(id[k] == (uint32_t)one);
                if (hit >> lane & 1) {
                    const int to = p + __popcll(hit & earlier);
                    a.order[to] = sort_place<EACH>(b0, k);
                    a.sorted[to] = (one << a.shift) + blockIdx.x;
                    id[k] = kSortOther;
                }
                p += __popcll(hit);
            }
            __syncthreads();  // `next` has been read
            if (threadIdx.x == 0)
                next[one] += all;
        }
        int mine = 0, entries;
#pragma unroll
        for (int k = 0; k < EACH; ++k)
            mine += __popcll(__ballot(id[k] != kSortOther));
        int at = places(mine, entries);
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const uint64_t hit = __ballot(id[k] != kSortOther);
            if (hit >> lane & 1)
                list[at + __popcll(hit & earlier)] = id[k] << 14 | (uint32_t)sort_place<EACH>(0, k);
            at += __popcll(hit);
        }
        __syncthreads();
        for (int e0 = 0; e0 < entries; e0 += 64) {
            const bool there = e0 + lane < entries;
            const uint32_t entry = there ? list[e0 + lane] : 0u;
            const int which = there ? (int)(entry >> 14) : -1;
            uint64_t todo = __ballot(there && which % kSortWaves == wave);
            while (todo) {
                const int one = __builtin_amdgcn_readlane(which, __builtin_ctzll(todo));
                const uint64_t same = __ballot(which == one);
                const int place = next[one];
                if (which == one) {
                    const int p = place + __popcll(same & earlier);
                    a.order[p] = b0 + (int)(entry & (kChunk - 1));
                    a.sorted[p] = (one << a.shift) + blockIdx.x;
                }
                next[one] = place + __popcll(same);  // (by every lane: the next read is its own)
                todo &= ~same;
            }
        }
    }
}
static_assert(kSortChunk == 1 << 14 && kSortRange <= 1 << 18, "an entry of the list is 32 bits");

// n values of a row of the gradient from their sums.
template <bool ADD, typename T>
__device__ __forceinline__ void store_row(const EmbedArgs &a, T *to, int n, const float (&sum)[8])
{
    float v[8];
    if (ADD) {
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
// Sums of runs of kEmbedRun sorted positions, a unit of columns per thread: of the IDs
// of up to kEmbedLong positions that start in the run, all of them.  The workgroup of
// a piece's first run also has those of the longer IDs in the piece: the sum of one
// that goes on behind it goes to the piece's second partial row, of one that came from
// before to its first.  Rows are loaded kRunLoads at a time.
// ---------------------------------------------------------------------------
constexpr int kRunLoads = 8;
static_assert(kEmbedRun + kEmbedLong <= 64 && kEmbedPiece <= 64 && kEmbedPiece % kEmbedRun == 0,
              "the positions of a run and of a piece are a wave's lanes");
static_assert(kEmbedPiece <= kEmbedLong, "an ID that is summed in pieces spans two or more of them");

template <typename TT, typename TO, bool ADD>
__device__ __forceinline__ void sum_run(const EmbedArgs &a, int run, int c)
{
    const int total = a.start[a.range << a.shift], lane = threadIdx.x & 63;
    const int p0 = run * kEmbedRun, p = p0 + lane;
    if (p0 >= total)
        return;
    // lane l: position p0 + l, its ID, and the ID's first position and the one behind
    const int id = a.sorted[min(p, total - 1)];
    const int row = a.order[min(p, total - 1)];
    const int32_t *start = a.start + embed_slot(a, (uint32_t)id);
    const int first = start[0], behind = start[1];
    const bool many = behind - first > kEmbedLong;
    const bool mine = p < total && (many ? p0 % kEmbedPiece == 0 && lane < kEmbedPiece : first >= p0 && first < p0 + kEmbedRun);
    const uint64_t stores = __ballot(mine && (p + 1 == behind || (many && lane == kEmbedPiece - 1)));
    const uint64_t wholes = __ballot(!many);
    char *to = many ? reinterpret_cast<char *>(a.part + (2 * (int64_t)(p0 / kEmbedPiece) + (first >= p0)) * a.ldpart)
                    : reinterpret_cast<char *>(table_row<TT>(a, id));
    const int to_low = (int)reinterpret_cast<uint64_t>(to), to_high = (int)(reinterpret_cast<uint64_t>(to) >> 32);
    float sum[8] = {};
    uint64_t todo = __ballot(mine);
    while (todo) {
        // the next kRunLoads of them; the last one again where there are no more, which
        // is added behind its own store and lost
        int at[kRunLoads];
        uint64_t now = 0;
        Unit<TO> raw[kRunLoads];
#pragma unroll
        for (int q = 0; q < kRunLoads; ++q) {
            at[q] = todo ? __builtin_ctzll(todo) : at[q > 0 ? q - 1 : 0];
            now |= todo & -todo;
            todo &= todo - 1;
            raw[q] = load_at(static_cast<const TO *>(a.dout) + (int64_t)__builtin_amdgcn_readlane(row, at[q]) * a.lddo,
                             c, a.H);
        }
#pragma unroll
        for (int q = 0; q < kRunLoads; ++q) {
            float v[8];
            values_of(raw[q], v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum[e] += v[e];
            if (stores & now & (uint64_t)1 << at[q]) {
                now ^= (uint64_t)1 << at[q];
                const uint64_t row_at = (uint32_t)__builtin_amdgcn_readlane(to_low, at[q]) |
                                        (uint64_t)(uint32_t)__builtin_amdgcn_readlane(to_high, at[q]) << 32;
                if (c < a.H) {
                    if (wholes >> at[q] & 1)
                        store_row<ADD>(a, in_memory(reinterpret_cast<TT *>(row_at)) + c, a.H - c, sum);
                    else
                        store_some(in_memory(reinterpret_cast<float *>(row_at)) + c, sum, 8);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[e] = 0.f;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Zeros for the rows that no ID names, nearly all of the call's bytes.  A thread has one
// 16-byte chunk and workgroups follow each other through the table: in that order
// 151936 rows of 10 KB take 235 us with the sort (227 us as a plain fill); workgroups
// with a row or two each took 297.  What there is to save is the time up to the store:
// chunks are numbered within 31 bits and divided by multiplication (245 us and more
// otherwise), and the row's lane is looked for, by the scalar unit where a wave is in
// one row, while the flags are under way.  They share a launch with the sums, whose
// loads run beside them (3333 rows, V 50257, H 1111: 61 us, 75 in two launches).
// ---------------------------------------------------------------------------
struct ZeroRows {
    int32_t first, rows;   // of the table, rows * chunks < 2^31
    int32_t chunks;        // of a row, the last one possibly short
    uint32_t factor;       // chunk k is in row (k * factor) >> shift
    int32_t shift;
};

ZeroRows zero_rows(int first, int V, int64_t row_bytes)
{
    ZeroRows z;
    z.chunks = (int32_t)((row_bytes + 15) / 16);
    z.first = first;
    z.rows = (int32_t)std::min<int64_t>(V - first, (((int64_t)1 << 31) - 1) / z.chunks);
    // 2^(shift - 31) >= chunks, factor = 2^shift / chunks rounded up: off by less than
    // chunks / 2^shift of it, so that k < 2^31 chunks never reach the next row
    z.shift = 31;
    while ((int64_t)1 << (z.shift - 31) < z.chunks)
        ++z.shift;
    z.factor = (uint32_t)((((uint64_t)1 << z.shift) + z.chunks - 1) / z.chunks);
    return z;
}

template <typename T>
__device__ __forceinline__ void write_zero(const EmbedArgs &a, const ZeroRows &z, uint32_t k)
{
    if (k >= (uint32_t)z.rows * (uint32_t)z.chunks)
        return;
    const int row = (int)((uint64_t)k * z.factor >> z.shift), v = z.first + row;
    const int32_t *start = a.start + embed_slot(a, (uint32_t)v);
    const int first = start[0], behind = start[1];
    const int one = __builtin_amdgcn_readfirstlane(v);
    constexpr int kEach = 16 / sizeof(T);
    const int c = kEach * (int)(k - (uint32_t)row * (uint32_t)z.chunks);
    T *to = (__all(v == one) ? table_row<T>(a, one) : table_row<T>(a, v)) + c;
    __builtin_amdgcn_sched_barrier(0);
    if (first != behind)
        return;
    const int n = a.H - c;
    if (n >= kEach) {
        *reinterpret_cast<raw4 *>(to) = raw4{0u, 0u, 0u, 0u};
        return;
    }
    for (int e = 0; e < n; ++e)
        to[e] = 0;
}

// Sums, and behind their `groups` workgroups zeros, which run beside them.  A
// workgroup has a run's columns, or where few threads do, several runs'.
template <typename TT, typename TO, bool ADD>
__global__ __launch_bounds__(kThreads) void embed_sums_kernel(const EmbedArgs a, const ZeroRows z, int threads,
                                                              int parts, uint32_t groups)
{
    if (blockIdx.x >= groups) {
        write_zero<TT>(a, z, (blockIdx.x - groups) * kThreads + threadIdx.x);
        return;
    }
    const int per = kThreads / threads, team = threadIdx.x / threads, part = blockIdx.x % parts;
    const int run = __builtin_amdgcn_readfirstlane((int)(blockIdx.x / parts) * per + team);
    if (team < per)
        sum_run<TT, TO, ADD>(a, run, 8 * (part * threads + (int)threadIdx.x % threads));
}

// ---------------------------------------------------------------------------
// IDs whose positions span pieces: their partial rows added, by the workgroup of the
// piece that they start in.  It looks at a piece per wave and has kJoinColumns columns
// of them.  A wave adds up to kJoinAlone rows by itself, in order; of more each of the
// waves adds an equal share, and the shares are added in order.
// ---------------------------------------------------------------------------
constexpr int kJoinColumns = 256, kJoinWaves = kThreads / 64, kJoinAlone = 16, kJoinLoads = 8;

// The partial rows [i0, i1) of the ID that starts in `piece`: the piece's second row, then
// the first of each piece behind.
__device__ __forceinline__ float4 add_parts(const EmbedArgs &a, int piece, int i0, int i1, int c)
{
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    const float *part = a.part + min((int64_t)c, a.ldpart - 4);
    for (; i0 < i1; i0 += kJoinLoads) {
        float4 v[kJoinLoads];
#pragma unroll
        for (int k = 0; k < kJoinLoads; ++k) {
            const int i = min(i0 + k, i1 - 1);
            v[k] = *reinterpret_cast<const float4 *>(part + (2 * (int64_t)(piece + i) + (i == 0)) * a.ldpart);
        }
#pragma unroll
        for (int k = 0; k < kJoinLoads; ++k) {
            const bool there = i0 + k < i1;
            sum.x += there ? v[k].x : 0.f;
            sum.y += there ? v[k].y : 0.f;
            sum.z += there ? v[k].z : 0.f;
            sum.w += there ? v[k].w : 0.f;
        }
    }
    return sum;
}

// Four columns per lane to the eight that a store takes: even lanes store.
template <typename T>
__device__ __forceinline__ void store_joined(const EmbedArgs &a, int id, int c, const float4 &sum)
{
    const float v[8] = {sum.x, sum.y, sum.z, sum.w, __shfl_down(sum.x, 1), __shfl_down(sum.y, 1),
                        __shfl_down(sum.z, 1), __shfl_down(sum.w, 1)};
    if ((threadIdx.x & 1) == 0 && c < a.H) {
        T *row = table_row<T>(a, id) + c;
        a.add ? store_row<true>(a, row, a.H - c, v) : store_row<false>(a, row, a.H - c, v);
    }
}

template <typename TT>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(const EmbedArgs a)
{
    __shared__ float4 shares[kJoinWaves][64];
    const int total = a.start[a.range << a.shift];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    // lane l: the ID that starts in piece kJoinWaves * x + l and goes on behind it
    const int piece0 = blockIdx.x * kJoinWaves, p0 = (piece0 + lane) * kEmbedPiece, last = p0 + kEmbedPiece - 1;
    int id = 0, rows = 0;
    if (lane < kJoinWaves && last < total) {
        id = a.sorted[last];
        const int32_t *start = a.start + embed_slot(a, (uint32_t)id);
        const int first = start[0], behind = start[1];
        if (first >= p0 && behind > last + 1 && behind - first > kEmbedLong)
            rows = (behind - 1) / kEmbedPiece - (piece0 + lane) + 1;
    }
    const int c = blockIdx.y * kJoinColumns + 4 * lane;
    const int mine = __builtin_amdgcn_readlane(rows, wave);
    if (mine > 0 && mine <= kJoinAlone)
        store_joined<TT>(a, __builtin_amdgcn_readlane(id, wave), c, add_parts(a, piece0 + wave, 0, mine, c));
    for (uint64_t todo = __ballot(rows > kJoinAlone); todo; todo &= todo - 1) {
        const int l = __builtin_ctzll(todo), n = __builtin_amdgcn_readlane(rows, l);
        const int each = (n + kJoinWaves - 1) / kJoinWaves;
        const float4 share = add_parts(a, piece0 + l, wave * each, min(n, (wave + 1) * each), c);
        __syncthreads();  // the shares are free
        shares[wave][lane] = share;
        __syncthreads();
        if (wave == 0) {
            float4 sum = shares[0][lane];
#pragma unroll
            for (int w = 1; w < kJoinWaves; ++w) {
                const float4 v = shares[w][lane];
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
            }
            store_joined<TT>(a, __builtin_amdgcn_readlane(id, l), c, sum);
        }
    }
}

template <typename TT, typename TO>
hipError_t lookup(const EmbedArgs &a, hipStream_t s)
{
    const int units = (a.H + 7) / 8;
    int threads = kThreads, team = 8;
    while (team < units && team < 64)
        team <<= 1;
    if (team == 64)
        team = threads = row_threads(a.H);
    const int64_t groups = ((int64_t)a.B + threads / team - 1) / (threads / team);
    hipLaunchKernelGGL((embed_kernel<TT, TO>), dim3((unsigned)std::min(groups, kMostGroups)), dim3(threads), 0, s, a, team);
    return hipGetLastError();
}

template <typename TT, typename TO>
hipError_t sums(const EmbedArgs &a, hipStream_t s)
{
    const int threads = row_threads(a.H), parts = (a.H + 8 * threads - 1) / (8 * threads), per = kThreads / threads;
    unsigned groups = (unsigned)((a.runs + per - 1) / per * parts);
    hipError_t e = hipSuccess;
    if (a.add)
        hipLaunchKernelGGL((embed_sums_kernel<TT, TO, true>), dim3(groups), dim3(kThreads), 0, s, a, ZeroRows{}, threads, parts, groups);
    for (int first = 0; !a.add && first < a.V;) {
        const ZeroRows z = zero_rows(first, a.V, a.H * (int64_t)sizeof(TT));
        const unsigned zeros = ((unsigned)z.rows * (unsigned)z.chunks + kThreads - 1) / kThreads;
        hipLaunchKernelGGL((embed_sums_kernel<TT, TO, false>), dim3(groups + zeros), dim3(kThreads), 0, s, a, z, threads, parts, groups);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        first += z.rows;
        groups = 0;
    }
    if ((e = hipGetLastError()) != hipSuccess || a.B <= std::max(kEmbedPiece, kEmbedLong))
        return e;
    const dim3 grid((unsigned)((a.B + kEmbedPiece * kJoinWaves - 1) / (kEmbedPiece * kJoinWaves)), (unsigned)((a.H + kJoinColumns - 1) / kJoinColumns));
    hipLaunchKernelGGL((embed_join_kernel<TT>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

template <int EACH>
hipError_t sort(const EmbedArgs &a, hipStream_t s)
{
    constexpr int kLds = kSortRange * 4 + kSortThreads * EACH * 4;
    static std::atomic<uint64_t> allowed{0};
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(embed_sort_kernel<EACH>), kLds, allowed);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((embed_sort_kernel<EACH>), dim3(1u << a.shift), dim3(kSortThreads), kLds, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_embed(const EmbedArgs &a, hipStream_t s)
{
    if (a.table_bf16)
        return a.rows_bf16 ? lookup<bf16_t, bf16_t>(a, s) : lookup<bf16_t, float>(a, s);
    return a.rows_bf16 ? lookup<float, bf16_t>(a, s) : lookup<float, float>(a, s);
}

// 256 groups, one for every CU, or as many as leave no more IDs in one than it counts.
int embed_shift(int32_t V)
{
    int shift = 8;
    while ((int64_t)kSortRange << shift < V)
        ++shift;
    return shift;
}

bool embed_grad_fits(int32_t B, int32_t H)
{
    const int64_t threads = row_threads(H), parts = ((int64_t)H + 8 * threads - 1) / (8 * threads);
    const int64_t runs = ((int64_t)B + kEmbedRun - 1) / kEmbedRun;
    // (the zeros behind the sums are below 2^31 threads, and a grid below 2^32)
    return runs * parts * kThreads < (int64_t)1 << 31 &&
           ((int64_t)H + kJoinColumns - 1) / kJoinColumns <= 65535;
}

// As few IDs per thread as one chunk needs: 300 tokens' gradient (V 1500, H 300, bf16) takes
// 14.4 us, 2000 tokens' 17.2; with 16 throughout 17.6 and 19.5.
hipError_t launch_embed_sort(const EmbedArgs &a, hipStream_t s)
{
    return a.B <= kSortThreads ? sort<1>(a, s) : a.B <= 4 * kSortThreads ? sort<4>(a, s) : sort<kSortEach>(a, s);
}

hipError_t launch_embed_sums(const EmbedArgs &a, hipStream_t s)
{
    if (a.table_bf16)
        return a.rows_bf16 ? sums<bf16_t, bf16_t>(a, s) : sums<bf16_t, float>(a, s);
    return a.rows_bf16 ? sums<float, bf16_t>(a, s) : sums<float, float>(a, s);
}

}  // namespace sbk
