// Verification of drafted tokens (gfx950).
//
// Sequence i has drafts x_0 .. x_(n-1), target logits z_0 .. z_n and draft logits
// y_0 .. y_(n-1).  With p_j = softmax(z_j / t), q_j = softmax(y_j / t), draft j is
// accepted while u_j q_j(x_j) < p_j(x_j).  Behind the accepted ones follows a token
// drawn from max(p_j - q_j, 0) of the first rejected draft j (p_j itself where
// that is 0 everywhere), or from p_n: the first column v whose cumulative sum
// passes u' times the whole.
//
// Everything behind the logits is in 64 bits.  A drawn token is where a random
// number meets the borders of a cumulative sum: a shift of 1e-8, as fp32
// exponentials give, moves one draw in a thousand over a flat row of 150000
// columns, and no two splits of a sum would agree.  On this chip fp64
// multiply-adds run at the rate of (unpacked) fp32 ones.
#include "verify.h"

#include <limits.h>
#include <math.h>

#include "values.h"
#include "verify_place.h"

namespace sbk {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kUnits = kVerifyChunk / (8 * kThreads);  // units of 8 columns per thread

// How the token behind the accepted ones is found.
enum How : int {
    kDone = 0,      // written already (greedy, or no distribution)
    kRow = 1,       // drawn from p
    kLess = 2,      // drawn from max(p - q, 0)
    kWithout = 3    // drawn from p without the rejected token (no draft logits)
};

// exp of x <= 0 (0 of -inf and NaN): x = k ln 2 + r, exp(r) by its Taylor series to
// r^11 / 11!, whose rest is below 0.3466^12 / 12! = 6e-15 of the value.
__device__ __forceinline__ double exp_of(double x)
{
    x = fmax(x, -800.0);
    const double k = rint(x * 1.4426950408889634074);
    double r = fma(k, -0.693147180559945286227, x);
    r = fma(k, -2.319046813846299558e-17, r);
    double e = 1.0 / 39916800;
    e = fma(e, r, 1.0 / 3628800);
    e = fma(e, r, 1.0 / 362880);
    e = fma(e, r, 1.0 / 40320);
    e = fma(e, r, 1.0 / 5040);
    e = fma(e, r, 1.0 / 720);
    e = fma(e, r, 1.0 / 120);
    e = fma(e, r, 1.0 / 24);
    e = fma(e, r, 1.0 / 6);
    e = fma(e, r, 0.5);
    e = fma(e, r, 1.0);
    e = fma(e, r, 1.0);
    return ldexp(e, (int)k);
}

// The order of the argmax: NaN above every number, then larger values, then lower
// columns (the projection calls' order).
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

// The larger, NaN where one is.
__device__ __forceinline__ float most_of(float a, float b)
{
    return a != a ? a : b != b ? b : fmaxf(a, b);
}

__device__ __forceinline__ float wave_most(float v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v = most_of(v, __shfl_xor(v, d));
    return v;
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ void wave_best(float &v, int &i)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        take_better(v, i, __shfl_xor(v, d), __shfl_xor(i, d));
}

// A sequence's place and temperature.
struct Sequence {
    int first, count;
    bool greedy;
    double scale;  // 1 / temperature
    __device__ __forceinline__ Sequence(const VerifyArgs &a, int i)
    {
        const Place place = place_of(a.offsets[i], a.offsets[i + 1], a.drafts, a.K);
        first = place.first;
        count = place.count;
        const float t = a.temperature ? a.temperature[i] : 1.f;
        greedy = !(t > 0.f);
        scale = greedy ? 1.0 : 1.0 / (double)t;
    }
    // rows of the matrices
    __device__ __forceinline__ int64_t target(int i, int j) const { return (int64_t)first + i + j; }
    __device__ __forceinline__ int64_t draft(int j) const { return (int64_t)first + j; }
};

__device__ __forceinline__ RowPart *parts_of(const VerifyArgs &a, int i, int slot)
{
    return a.parts + ((int64_t)i * (2 * a.K + 1) + slot) * a.chunks;
}

template <typename T>
__device__ __forceinline__ void load_chunk(const void *rows, int64_t ld, int64_t row, int c0, int V,
                                           Unit<T> (&v)[kUnits])
{
    const T *p = static_cast<const T *>(rows) + row * ld;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int c = c0 + 8 * (i * kThreads + (int)threadIdx.x);
        if (c < V)
            v[i] = load_some(p + c, V - c);
        else
            clear(v[i]);
    }
}

// ---------------------------------------------------------------------------
// Every chunk of every row that a sequence may need.
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(kThreads) void verify_rows_kernel(const VerifyArgs a)
{
    __shared__ float mosts[kWaves];
    __shared__ double sums[kWaves];
    __shared__ int ats[kWaves];
    const int chunk = blockIdx.x % a.chunks;
    const int slots = 2 * a.K + 1;
    const int i = blockIdx.x / a.chunks / slots, slot = blockIdx.x / a.chunks % slots;
    const Sequence s(a, i);
    const bool is_draft = slot > a.K;
    // rows that are not there, and draft rows that nothing asks for
    if (is_draft ? slot - a.K - 1 >= s.count || !a.draft || s.greedy : slot > s.count)
        return;
    const int c0 = chunk * kVerifyChunk, V = a.V;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    Unit<T> raw[kUnits];
    if (is_draft)
        load_chunk<T>(a.draft, a.ldd, s.draft(slot - a.K - 1), c0, V, raw);
    else
        load_chunk<T>(a.target, a.ldt, s.target(i, slot), c0, V, raw);
    RowPart &to = parts_of(a, i, slot)[chunk];
    if (s.greedy) {
        float best = -INFINITY;
        int at = INT_MAX;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            float v[8];
            values_of(raw[k], v);
            const int c = c0 + 8 * (k * kThreads + (int)threadIdx.x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < V)
                    take_better(best, at, v[e], c + e);
        }
        wave_best(best, at);
        if (lane == 0) {
            mosts[wave] = best;
            ats[wave] = at;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kWaves; ++w)
                take_better(best, at, mosts[w], ats[w]);
            to.most = best;
            to.at = at;
        }
        return;
    }
    float most = -INFINITY;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        float v[8];
        values_of(raw[k], v);
        const int c = c0 + 8 * (k * kThreads + (int)threadIdx.x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < V)
                most = v[e] < INFINITY ? most_of(most, v[e]) : NAN;
    }
    most = wave_most(most);
    if (lane == 0)
        mosts[wave] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        most = most_of(most, mosts[w]);
    double sum = 0.0;
    if (most > -INFINITY) {
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            float v[8];
            values_of(raw[k], v);
            const int c = c0 + 8 * (k * kThreads + (int)threadIdx.x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double x = exp_of(((double)v[e] - (double)most) * s.scale);
                sum += c + e < V ? x : 0.0;
            }
        }
    }
    sum = wave_sum(sum);
    if (lane == 0)
        sums[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWaves; ++w)
            sum += sums[w];
        to.sum = sum;
        to.most = most;
    }
}

// A row's softmax: p(v) = exp((z - most) scale) / sum.  `there` is false where the row
// has no distribution.
struct Softmax {
    float most;
    double over;  // 1 / sum
    bool there;
    __device__ __forceinline__ double of(float z, double scale) const
    {
        return exp_of(((double)z - (double)most) * scale) * over;
    }
    // the part of a chunk
    __device__ __forceinline__ double part(const RowPart &r, double scale) const
    {
        return r.most > -INFINITY ? r.sum * exp_of(((double)r.most - (double)most) * scale) * over : 0.0;
    }
};

// From the row's chunks, by one wave.
__device__ __forceinline__ Softmax softmax_of(const RowPart *parts, int chunks, double scale)
{
    const int lane = threadIdx.x & 63;
    float most = -INFINITY;
    for (int c = lane; c < chunks; c += 64)
        most = most_of(most, parts[c].most);
    most = wave_most(most);
    Softmax s{most, 0.0, most > -INFINITY};
    if (!s.there)
        return s;
    double sum = 0.0;
    for (int c = lane; c < chunks; c += 64)
        if (parts[c].most > -INFINITY)
            sum += parts[c].sum * exp_of(((double)parts[c].most - (double)most) * scale);
    s.over = 1.0 / wave_sum(sum);
    return s;
}

// A row's best column, by one wave.
__device__ __forceinline__ int best_of(const RowPart *parts, int chunks)
{
    float v = -INFINITY;
    int at = INT_MAX;
    for (int c = threadIdx.x & 63; c < chunks; c += 64)
        take_better(v, at, parts[c].most, parts[c].at);
    wave_best(v, at);
    return at;
}

template <typename T>
__device__ __forceinline__ float logit(const void *rows, int64_t ld, int64_t row, int v)
{
    return value_of(static_cast<const T *>(rows)[row * ld + v]);
}

// Whether draft j of a sequence is accepted, by one wave.
template <typename T>
__device__ __forceinline__ bool accepts(const VerifyArgs &a, const Sequence &s, int i, int j)
{
    const int x = a.tokens[s.first + j];
    if ((uint32_t)x >= (uint32_t)a.V)
        return false;
    if (s.greedy)
        return best_of(parts_of(a, i, j), a.chunks) == x;
    const Softmax p = softmax_of(parts_of(a, i, j), a.chunks, s.scale);
    if (!p.there)
        return false;
    const double px = p.of(logit<T>(a.target, a.ldt, s.target(i, j), x), s.scale);
    double qx = 1.0;
    if (a.draft) {
        const Softmax q = softmax_of(parts_of(a, i, a.K + 1 + j), a.chunks, s.scale);
        if (!q.there)
            return false;
        qx = q.of(logit<T>(a.draft, a.ldd, s.draft(j), x), s.scale);
    }
    return (double)a.u[s.first + j] * qx < px;
}

// What is left of the columns of a unit of row j, to draw from.
template <typename T>
struct Rest {
    Softmax p, q;
    double scale;
    int how, without;
    __device__ __forceinline__ void of(const Unit<T> &zs, const Unit<T> &ys, int c, int V, double (&r)[8]) const
    {
        // p and q are rounded before their difference: fused, equal ones would leave
        // what the rounding of one took
#pragma clang fp contract(off)
        float z[8], y[8];
        values_of(zs, z);
        values_of(ys, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            r[e] = p.of(z[e], scale);
            if (how == kLess)
                r[e] = fmax(r[e] - q.of(y[e], scale), 0.0);
            if (c + e >= V || (how == kWithout && c + e == without))
                r[e] = 0.0;
        }
    }
};

// ---------------------------------------------------------------------------
// One workgroup per sequence and chunk: what is accepted (each workgroup finds
// that for itself, from the parts, four drafts at a time), and the sum of what is
// left in the chunk.  Where the next token is drawn from a whole row, the rows'
// parts hold that sum already.
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(kThreads) void verify_rest_kernel(const VerifyArgs a)
{
    __shared__ int firsts[kWaves];
    __shared__ double sums[kWaves];
    const int i = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
    const Sequence s(a, i);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    int rejected = s.count;
    for (int j = wave; j < s.count; j += kWaves)
        if (!accepts<T>(a, s, i, j)) {
            rejected = j;
            break;
        }
    if (lane == 0)
        firsts[wave] = rejected;
    __syncthreads();
    int j = s.count;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        j = min(j, firsts[w]);
    const RowPart *row = parts_of(a, i, j);
    const int x = j < s.count ? a.tokens[s.first + j] : -1;
    Rest<T> rest;
    rest.how = kRow;
    rest.scale = s.scale;
    rest.without = x;
    if (s.greedy) {
        rest.how = kDone;
    } else {
        rest.p = softmax_of(row, a.chunks, s.scale);
        if (!rest.p.there) {
            rest.how = kDone;
        } else if (j < s.count) {
            if (a.draft) {
                rest.q = softmax_of(parts_of(a, i, a.K + 1 + j), a.chunks, s.scale);
                if (rest.q.there)
                    rest.how = kLess;
            } else if ((uint32_t)x < (uint32_t)a.V) {
                rest.how = kWithout;
            }
        }
    }
    if (chunk == 0) {
        const int next = s.greedy ? best_of(row, a.chunks) : -1;
        for (int k = threadIdx.x; k <= a.K; k += kThreads)
            a.out[i * a.ldo + k] = k < j ? a.tokens[s.first + k] : k == j && rest.how == kDone ? next : -1;
        if (threadIdx.x == 0) {
            a.accepted[i] = j;
            a.made[i] = Decision{j, rest.how};
        }
    }
    if (rest.how == kDone)
        return;
    const int c0 = chunk * kVerifyChunk;
    double *to = a.rest + (int64_t)i * a.chunks + chunk;
    if (rest.how == kRow || (rest.how == kWithout && (uint32_t)(x - c0) >= (uint32_t)kVerifyChunk)) {
        if (threadIdx.x == 0)
            *to = rest.p.part(row[chunk], s.scale);
        return;
    }
    Unit<T> z[kUnits], y[kUnits];
    load_chunk<T>(a.target, a.ldt, s.target(i, j), c0, a.V, z);
    if (rest.how == kLess) {
        load_chunk<T>(a.draft, a.ldd, s.draft(j), c0, a.V, y);
    } else {
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
            clear(y[k]);
    }
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        double r[8];
        rest.of(z[k], y[k], c0 + 8 * (k * kThreads + (int)threadIdx.x), a.V, r);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum += r[e];
    }
    sum = wave_sum(sum);
    if (lane == 0)
        sums[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWaves; ++w)
            sum += sums[w];
        *to = sum;
    }
}

// Prefix sums over a wave, in lane order.
__device__ __forceinline__ double wave_upto(double v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(v, d);
        v += lane >= d ? o : 0.0;
    }
    return v;
}

// ---------------------------------------------------------------------------
// One workgroup per sequence: the chunk whose cumulative sum passes the random
// number's share of the whole, then the column in it.
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(const VerifyArgs a)
{
    __shared__ double unit_sums[kUnits][kWaves];
    __shared__ int found, last;
    const int i = blockIdx.x;
    const Decision d = a.made[i];
    if (d.how == kDone)
        return;
    const Sequence s(a, i);
    const int j = d.accepted;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const RowPart *row = parts_of(a, i, j);
    Rest<T> rest;
    rest.how = d.how;
    rest.scale = s.scale;
    rest.without = d.how == kWithout ? a.tokens[s.first + j] : -1;
    rest.p = softmax_of(row, a.chunks, s.scale);
    if (d.how == kLess)
        rest.q = softmax_of(parts_of(a, i, a.K + 1 + j), a.chunks, s.scale);
    const double *sums = a.rest + (int64_t)i * a.chunks;
    const float u = a.u_next[i];
    // Every wave looks for the chunk by itself.  Where nothing is left, the row itself
    // is drawn from.
    int chunk = 0;
    double before = 0.0, goal = 0.0;
    for (int pass = 0; pass < 2; ++pass) {
        const bool whole = pass == 1;
        if (whole)
            rest.how = kRow;
        double total = 0.0;
        for (int c0 = 0; c0 < a.chunks; c0 += 64) {
            const int c = c0 + lane;
            total += wave_sum(c < a.chunks ? whole ? rest.p.part(row[c], s.scale) : sums[c] : 0.0);
        }
        if (!(total > 0.0))
            continue;
        // (a number outside [0, 1) draws the first or the last column)
        goal = (u > 0.f ? (double)u : 0.0) * total;
        double upto = 0.0;
        chunk = -1;
        for (int c0 = 0; c0 < a.chunks; c0 += 64) {
            const int c = c0 + lane;
            const double v = c < a.chunks ? whole ? rest.p.part(row[c], s.scale) : sums[c] : 0.0;
            const double mine = upto + wave_upto(v);
            const uint64_t past = __ballot(v > 0.0 && mine > goal), some = __ballot(v > 0.0);
            // the first chunk past the goal, else the last one with anything left
            const int at = past ? __builtin_ctzll(past) : some ? 63 - __builtin_clzll(some) : -1;
            if (at >= 0) {
                chunk = c0 + at;
                before = __shfl(mine, at) - __shfl(v, at);
            }
            if (past)
                break;
            upto = __shfl(mine, 63);
        }
        break;
    }
    if (threadIdx.x == 0) {
        found = INT_MAX;
        last = -1;
    }
    const int c0 = chunk * kVerifyChunk;
    Unit<T> z[kUnits], y[kUnits];
    load_chunk<T>(a.target, a.ldt, s.target(i, j), c0, a.V, z);
    if (rest.how == kLess) {
        load_chunk<T>(a.draft, a.ldd, s.draft(j), c0, a.V, y);
    } else {
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
            clear(y[k]);
    }
    double r[kUnits][8], upto[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        rest.of(z[k], y[k], c0 + 8 * (k * kThreads + (int)threadIdx.x), a.V, r[k]);
        double sum = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum += r[k][e];
        upto[k] = wave_upto(sum);
        if (lane == 63)
            unit_sums[k][wave] = upto[k];
        upto[k] -= sum;
    }
    __syncthreads();
    int mine = INT_MAX, behind = -1;
    double base = before;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w == wave) {
                double sum = base + upto[k];
                const int c = c0 + 8 * (k * kThreads + (int)threadIdx.x);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sum += r[k][e];
                    if (r[k][e] > 0.0) {
                        behind = c + e;
                        if (sum > goal && mine == INT_MAX)
                            mine = c + e;
                    }
                }
            }
            base += unit_sums[k][w];
        }
    }
    if (mine != INT_MAX)
        atomicMin(&found, mine);
    if (behind >= 0)
        atomicMax(&last, behind);
    __syncthreads();
    if (threadIdx.x == 0)
        a.out[i * a.ldo + j] = found != INT_MAX ? found : last;
}

template <typename T>
hipError_t verify(const VerifyArgs &a, hipStream_t s)
{
    const unsigned per = (unsigned)a.N * (unsigned)a.chunks;
    hipLaunchKernelGGL((verify_rows_kernel<T>), dim3(per * (2 * a.K + 1)), dim3(kThreads), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((verify_rest_kernel<T>), dim3(per), dim3(kThreads), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    hipLaunchKernelGGL((verify_pick_kernel<T>), dim3((unsigned)a.N), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(const VerifyArgs &a, hipStream_t s)
{
    return a.bf16 ? verify<bf16_t>(a, s) : verify<float>(a, s);
}

}  // namespace sbk
