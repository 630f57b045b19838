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

#include <algorithm>

#include "values.h"
#include "verify_place.h"

namespace sbk {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kMostJudges = 16;  // waves of a sequence's verdict

// How the token behind the accepted ones is found.
enum How : int {
    kDone = 0,      // greedy, or no distribution
    kRow = 1,       // drawn from p
    kLess = 2,      // drawn from max(p - q, 0)
    kWithout = 3    // drawn from p without the rejected token (no draft logits)
};

// 2^f of -1/2 <= f <= 1/2, exactly 1 of 0: 1 + f g(f), g through (2^f - 1) / f at the 9
// Chebyshev nodes; off by up to 3.7e-14 of it.  A logit is off by its own rounding, 2^-24
// of itself in fp32, and a random number falls between a share and the one found once in
// 10^7.  With 10 nodes (5.7e-16) 64 sequences of 7 drafts, V 151936 in fp32, take 148 us, 144
// with 9.
__device__ __forceinline__ double power_within(double f)
{
    double e = 1.02031210633917290e-07;
    e = fma(e, f, 1.32552248786688168e-06);
    e = fma(e, f, 1.52526868462677196e-05);
    e = fma(e, f, 1.54034558524538382e-04);
    e = fma(e, f, 1.33335581790431116e-03);
    e = fma(e, f, 9.61812915940255843e-03);
    e = fma(e, f, 5.55041086647604237e-02);
    e = fma(e, f, 2.40226506958129887e-01);
    e = fma(e, f, 6.93147180559945286e-01);
    return fma(e, f, 1.0);
}

// 2^t of t <= 1, 0 of -inf and NaN.
__device__ __forceinline__ double power_of(double t)
{
    t = fmax(t, -1100.0);
    const double k = rint(t);
    return ldexp(power_within(t - k), (int)k);
}

// 2^((z - most) rate) of a row's or a chunk's logits, whose largest is `most`: exactly 1 of
// the largest, so that rows of 2^n equal logits have shares of 2^-n exactly.  (Powers
// against the whole number next to most rate save the difference, 2 of 145 us for 64
// sequences of 7 drafts, V 151936, and put such shares 4e-14 off to either side.)  A logit
// takes 17 64-bit instructions: the difference's product with the rate, rounded to a whole
// number k by the size of 3 2^51, and the rest after k are one fused multiply-add each, and
// k is the low word.  Logits whose power is 0 anyway are raised to one that still is (so is
// -inf).
struct Shares {
    double rate, most, low;
    __device__ __forceinline__ Shares(float largest, double r)
    {
        rate = fmax(r, 1e-290);  // (a temperature of +inf; -inf logits stay at 0)
        most = largest;
        low = -1100.0 / rate;
    }
    __device__ __forceinline__ double of(float z) const
    {
        constexpr double kRound = 6755399441055744.0;  // 3 2^51
        const double d = fmax((double)z - most, low), k = fma(d, rate, kRound);
        return ldexp(power_within(fma(d, rate, kRound - k)), __double2loint(k));
    }
    // the factor from these powers to those of a row whose largest logit is row_most
    __device__ __forceinline__ double to(float row_most) const
    {
        return power_of((most - (double)row_most) * rate);
    }
};

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

__device__ __forceinline__ void wave_best(float &v, int &i)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        take_better(v, i, __shfl_xor(v, d), __shfl_xor(i, d));
}

// A sequence's place and temperature: exp(z / t) is 2^(z rate).
struct Sequence {
    int first, count;
    bool greedy;
    double rate;
    __device__ __forceinline__ Sequence(const VerifyArgs &a, int i)
    {
        const Place place = place_of(a.offsets[i], a.offsets[i + 1], a.drafts, a.K);
        first = place.first;
        count = place.count;
        const float t = a.temperature ? a.temperature[i] : 1.f;
        greedy = !(t > 0.f);
        rate = 1.4426950408889634074 / (greedy ? 1.0 : (double)t);
    }
    // rows of the matrices
    __device__ __forceinline__ int64_t target(int i, int j) const { return (int64_t)first + i + j; }
    __device__ __forceinline__ int64_t draft(int j) const { return (int64_t)first + j; }
};

__device__ __forceinline__ RowPart *parts_of(const VerifyArgs &a, int i, int slot)
{
    return a.parts + ((int64_t)i * a.slots + slot) * a.chunks;
}

// COLUMNS of a row, 8 to a thread at a time and neighbours in neighbouring threads.
// Those behind the last are -inf, which no sum and no draw sees.
template <typename T, int COLUMNS>
struct Chunk {
    static constexpr int kUnits = COLUMNS / (8 * kThreads);
    Unit<T> raw[kUnits];
    __device__ __forceinline__ static int column(int k) { return 8 * (k * kThreads + (int)threadIdx.x); }
    // from p, which `left` columns are there of
    __device__ __forceinline__ void load(const T *p, int left)
    {
        if (left >= COLUMNS) {
#pragma unroll
            for (int k = 0; k < kUnits; ++k)
                raw[k] = load_unit(p + column(k));
            return;
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
            raw[k] = load_at(p, column(k), left);
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
            fill(raw[k], left - column(k));
    }
    __device__ __forceinline__ static void fill(Unit<float> &u, int n)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            (e < 4 ? u.a : u.b)[e & 3] = e < n ? (e < 4 ? u.a : u.b)[e & 3] : 0xFF800000u;
    }
    __device__ __forceinline__ static void fill(Unit<bf16_t> &u, int n)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            u.a[e] = 2 * e + 1 < n ? u.a[e] : 2 * e < n ? (u.a[e] & 0xFFFFu) | 0xFF800000u : 0xFF80FF80u;
    }
};

template <typename T>
__device__ __forceinline__ const T *row_at(const void *rows, int64_t ld, int64_t row, int c0)
{
    return static_cast<const T *>(rows) + row * ld + c0;
}

// ---------------------------------------------------------------------------
// Every chunk of every row that a sequence may need: the largest logit, and the sum of
// the powers or, of a greedy sequence, the largest logit's column.  Workgroups take one
// chunk after the other, the next one's loads under way while the powers of one are
// summed.  64 sequences of 7 drafts with draft logits, 16 of them greedy, V 151936 in fp32:
// 110 to 123 us.  The 515 MB that they read take 79 at 6.5 TB/s; 41.2 million wave
// instructions, 23 for each logit whose power is summed (17 are the power and its sum),
// take 90 at the 5.2 cycles each that a loop of powers alone takes, and a third of the
// waves' cycles are waits.
// Twice as many workgroups as are resident: those whose rows are not there leave room for
// others (17 ragged sequences, V 50257: the call takes 22.1 us, with as many as are resident
// 24.5; the 64 sequences 144.3 and 145.8).
// ---------------------------------------------------------------------------
constexpr uint32_t kRowGroups = 2048;

// A chunk to take: workgroup's items number, ... (none: to is NULL)
template <typename T>
struct Item {
    RowPart *to;
    const T *from;
    int left, c0;
    bool greedy;
    double rate;
};

// The first item from `at` on, in steps, that a sequence may need; `at` moves to it.
template <typename T>
__device__ __forceinline__ Item<T> next_item(const VerifyArgs &a, uint32_t &at, uint32_t items)
{
    const uint32_t each = (uint32_t)a.slots * (uint32_t)a.chunks;
    Item<T> item = {};
    for (; at < items; at += gridDim.x) {
        const int i = (int)(at / each), rest = (int)(at % each);
        const int slot = rest / a.chunks, chunk = rest % a.chunks;
        const Sequence s(a, i);
        const bool is_draft = slot > a.K;
        // rows that are not there, and draft rows that nothing asks for
        if (is_draft ? slot - a.K - 1 >= s.count || s.greedy : slot > s.count)
            continue;
        item.to = parts_of(a, i, slot) + chunk;
        item.c0 = chunk * kVerifyChunk;
        item.left = a.V - item.c0;
        item.from = is_draft ? row_at<T>(a.draft, a.ldd, s.draft(slot - a.K - 1), item.c0)
                             : row_at<T>(a.target, a.ldt, s.target(i, slot), item.c0);
        item.greedy = s.greedy;
        item.rate = s.rate;
        break;
    }
    return item;
}

template <typename PART>
__device__ __forceinline__ double sum_of_powers(const PART &part, const Shares &shares)
{
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < PART::kUnits; ++k) {
        float v[8];
        values_of(part.raw[k], v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum += shares.of(v[e]);
    }
    return sum;
}

template <typename T>
__global__ __launch_bounds__(kThreads, 4) void verify_rows_kernel(const VerifyArgs a, uint32_t items)
{
    __shared__ float mosts[kWaves];
    __shared__ double sums[kWaves];
    __shared__ int ats[kWaves];
    typedef Chunk<T, kVerifyChunk> Part;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    uint32_t at = blockIdx.x;
    Item<T> item = next_item<T>(a, at, items);
    Part next;
    if (item.to)
        next.load(item.from, item.left);
    while (item.to) {
        const Item<T> now = item;
        const Part part = next;
        at += gridDim.x;
        item = next_item<T>(a, at, items);
        float most = -INFINITY;
#pragma unroll
        for (int k = 0; k < Part::kUnits; ++k) {
            float v[8];
            values_of(part.raw[k], v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                most = most_of(most, v[e]);
        }
        if (item.to)
            next.load(item.from, item.left);
        most = wave_most(most);
        if (lane == 0)
            mosts[wave] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            most = most_of(most, mosts[w]);
        if (now.greedy) {
            // the lowest column that is a NaN, or else equals the largest (columns behind
            // the last come after those that are there)
            int low = INT_MAX;
#pragma unroll
            for (int k = Part::kUnits - 1; k >= 0; --k) {
                float v[8];
                values_of(part.raw[k], v);
#pragma unroll
                for (int e = 7; e >= 0; --e)
                    if (most != most ? v[e] != v[e] : v[e] == most)
                        low = Part::column(k) + e;
            }
#pragma unroll
            for (int d = 1; d < 64; d <<= 1)
                low = min(low, __shfl_xor(low, d));
            if (lane == 0)
                ats[wave] = low;
            __syncthreads();
            if (threadIdx.x == 0) {
#pragma unroll
                for (int w = 0; w < kWaves; ++w)
                    low = min(low, ats[w]);
                now.to->most = most;
                now.to->at = now.c0 + low;
            }
            continue;
        }
        if (most == INFINITY)
            most = NAN;
        double sum = 0.0;
        if (most > -INFINITY)
            sum = sum_of_powers(part, Shares(most, now.rate));
        sum = wave_sum(sum);
        if (lane == 0)
            sums[wave] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kWaves; ++w)
                sum += sums[w];
            now.to->sum = sum;
            now.to->most = most;
        }
    }
}

__device__ __forceinline__ bool there(const Softmax &s) { return s.most > -INFINITY; }
// From the row's chunks, by one wave.
__device__ __forceinline__ Softmax softmax_of(const RowPart *parts, int chunks, double rate)
{
    const int lane = threadIdx.x & 63;
    // (the first 64 chunks are read once)
    const RowPart none = {0.0, -INFINITY, 0}, first = lane < chunks ? parts[lane] : none;
    float most = first.most;
    for (int c = lane + 64; c < chunks; c += 64)
        most = most_of(most, parts[c].most);
    Softmax s{0.0, wave_most(most)};
    if (!there(s))
        return s;
    double sum = first.most > -INFINITY ? first.sum * Shares(first.most, rate).to(s.most) : 0.0;
    for (int c = lane + 64; c < chunks; c += 64)
        if (parts[c].most > -INFINITY)
            sum += parts[c].sum * Shares(parts[c].most, rate).to(s.most);
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

// ---------------------------------------------------------------------------
// What becomes of a sequence, a workgroup each: the first row that rejects its draft (the
// row behind the last draft always does), a row per wave at a time.
// ---------------------------------------------------------------------------
// What a wave finds about row j: `accepted` is whether its draft is, `how` and `next` tell
// how the token is found where it is not.
template <typename T>
__device__ __forceinline__ Verdict judge(const VerifyArgs &a, const Sequence &s, int i, int j, int &next)
{
    Verdict d = {{0.0, NAN}, {0.0, NAN}, 0, kDone};
    next = -1;
    const bool drafted = j < s.count;
    const int x = drafted ? a.tokens[s.first + j] : -1;
    const bool inside = (uint32_t)x < (uint32_t)a.V;
    if (s.greedy) {
        next = best_of(parts_of(a, i, j), a.chunks);
        d.accepted = drafted && next == x;
        return d;
    }
    const bool both = drafted && a.draft;
    const float z = inside ? value_of(*row_at<T>(a.target, a.ldt, s.target(i, j), x)) : -INFINITY;
    const float y = inside && both ? value_of(*row_at<T>(a.draft, a.ldd, s.draft(j), x)) : -INFINITY;
    const float u = drafted ? a.u[s.first + j] : 0.f;
    d.p = softmax_of(parts_of(a, i, j), a.chunks, s.rate);
    if (both)
        d.q = softmax_of(parts_of(a, i, a.K + 1 + j), a.chunks, s.rate);
    if (!there(d.p))
        return d;
    d.how = kRow;
    if (!drafted)
        return d;
    const bool comparable = inside && (!both || there(d.q));
    const double qx = both && comparable ? Shares(d.q.most, s.rate).of(y) * d.q.over : 1.0;
    d.accepted = comparable && (double)u * qx < Shares(d.p.most, s.rate).of(z) * d.p.over;
    if (both && there(d.q))
        d.how = kLess;
    else if (!both && inside)
        d.how = kWithout;
    return d;
}

template <typename T>
__global__ __launch_bounds__(64 * kMostJudges) void verify_judge_kernel(const VerifyArgs a)
{
    __shared__ int firsts[kMostJudges];
    const int i = blockIdx.x, waves = blockDim.x >> 6;
    const Sequence s(a, i);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    int mine = INT_MAX, next = -1;
    Verdict verdict;
    for (int j = wave; j <= s.count; j += waves) {
        verdict = judge<T>(a, s, i, j, next);
        if (!verdict.accepted) {
            mine = j;
            break;
        }
    }
    if (lane == 0)
        firsts[wave] = mine;
    __syncthreads();
    int j = INT_MAX;
    for (int w = 0; w < waves; ++w)
        j = min(j, firsts[w]);
    if (mine != j)
        return;
    // the wave of that row writes the sequence's results
    for (int k = lane; k <= a.K; k += 64)
        a.out[i * a.ldo + k] = k < j ? a.tokens[s.first + k] : k == j ? next : -1;
    if (lane == 0) {
        verdict.accepted = j;
        a.accepted[i] = j;
        a.made[i] = verdict;
        a.done[(int64_t)i * kVerifyDone] = 0;
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
// The draw: a workgroup per sequence and kVerifyDraw columns sums up what is left of
// them.  The last of a sequence's workgroups to be done (none waits for another) finds
// the one whose cumulative sum passes the random number's share of the whole, then the
// column.
// 2048 columns, one unit to a thread: a call on one sequence (V 151936, fp32) takes 16.8
// us, on 64 of them 144.3; with 4096 18.0 and 146.0.
// ---------------------------------------------------------------------------
template <typename T>
struct Rest {
    typedef Chunk<T, kVerifyDraw> Part;
    Part z, y;
    __device__ __forceinline__ void load(const VerifyArgs &a, const Sequence &s, const Verdict &d, int i, int c0)
    {
        z.load(row_at<T>(a.target, a.ldt, s.target(i, d.accepted), c0), a.V - c0);
        if (d.how == kLess)
            y.load(row_at<T>(a.draft, a.ldd, s.draft(d.accepted), c0), a.V - c0);
    }
    // A unit's shares of p and what is left of them; x: the rejected token's column, from
    // these columns' first on.
    __device__ __forceinline__ void find(const Verdict &d, const Shares &ps, const Shares &qs, int x, int k,
                                         double (&p)[8], double (&r)[8]) const
    {
        // p and q are rounded before their difference: fused, equal ones would leave
        // what the rounding of one took
#pragma clang fp contract(off)
        float v[8];
        values_of(z.raw[k], v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            p[e] = ps.of(v[e]) * d.p.over;
        if (d.how == kLess) {
            values_of(y.raw[k], v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[e] = fmax(p[e] - qs.of(v[e]) * d.q.over, 0.0);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[e] = d.how == kWithout && Part::column(k) + e == x ? 0.0 : p[e];
        }
    }
};

__device__ __forceinline__ double sum_of(const double (&v)[8])
{
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

template <typename T>
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(const VerifyArgs a)
{
    typedef typename Rest<T>::Part Part;
    constexpr int kUnits = Part::kUnits;
    __shared__ double sums[2][kUnits][kWaves];
    __shared__ int token, last;
    __shared__ bool draws;
    const int i = blockIdx.x / a.draws, mine = blockIdx.x % a.draws;
    const Verdict d = a.made[i];
    const Sequence s(a, i);
    if (d.how == kDone)
        return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, j = d.accepted;
    const int x = d.how == kWithout ? a.tokens[s.first + j] : -1;
    const float u = a.u_next[i];
    double *rests = a.rest + (int64_t)i * a.draws * 2;
    const Shares ps(d.p.most, s.rate), qs(d.q.most, s.rate);
    // First these columns' sums, then in the last workgroup the columns of the one that was
    // found, by the same code: as code of its own, run by one workgroup and fetched
    // from memory, that took it 3 us more.
    Rest<T> rest;
    int from = 0, at = mine;
    double before = 0.0, goal = 0.0, r[kUnits][8], upto[kUnits];
    for (bool found = false;; found = true) {
        rest.load(a, s, d, i, at * kVerifyDraw);
        double whole = 0.0;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            double p[8];
            rest.find(d, ps, qs, x - at * kVerifyDraw, k, p, r[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[k][e] = from > 0 ? p[e] : r[k][e];
            const double sum = sum_of(r[k]);
            whole += sum_of(p);
            upto[k] = wave_upto(sum);
            if (lane == 63)
                sums[0][k][wave] = upto[k];
            upto[k] -= sum;
        }
        whole = wave_sum(whole);
        if (lane == 0)
            sums[1][0][wave] = whole;
        __syncthreads();
        if (found)
            break;
        if (threadIdx.x == 0) {
            double left = 0.0;
            whole = 0.0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
#pragma unroll
                for (int k = 0; k < kUnits; ++k)
                    left += sums[0][k][w];
                whole += sums[1][0][w];
            }
            // Written through to memory, complete before they are counted, and read from memory
            // (device-scope atomics): no workgroup needs a fence, which writes back and
            // empties its XCD's L2 (4800 of them took 80 us).
            __hip_atomic_store(&rests[2 * mine], left, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(&rests[2 * mine + 1], whole, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            __builtin_amdgcn_s_waitcnt(0);
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            draws = __hip_atomic_fetch_add(&a.done[(int64_t)i * kVerifyDone], 1u, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT) + 1 == (uint32_t)a.draws;
            token = INT_MAX;
            last = -1;
        }
        __syncthreads();
        if (!draws)
            return;
        // Every wave looks for the columns' workgroup by itself.  Where nothing is left, p is
        // drawn from.
        for (; from < 2; ++from) {
            auto weight = [&](int c) {
                return c < a.draws ? __hip_atomic_load(&rests[2 * c + from], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                                   : 0.0;
            };
            const double first = weight(lane);  // (read once)
            double total = wave_sum(first);
            for (int c0 = 64; c0 < a.draws; c0 += 64)
                total += wave_sum(weight(c0 + lane));
            if (!(total > 0.0))
                continue;
            // (a number outside [0, 1) draws the first or the last column: no sum passes
            // infinity, but those below may pass the total, which is added in another order)
            goal = u >= 1.f ? (double)INFINITY : (u > 0.f ? (double)u : 0.0) * total;
            double behind = 0.0;
            for (int c0 = 0; c0 < a.draws; c0 += 64) {
                const double v = c0 == 0 ? first : weight(c0 + lane), to = behind + wave_upto(v);
                const uint64_t past = __ballot(v > 0.0 && to > goal), some = __ballot(v > 0.0);
                // the first past the goal, else the last with anything left
                const int one = past ? __builtin_ctzll(past) : some ? 63 - __builtin_clzll(some) : -1;
                if (one >= 0) {
                    at = c0 + one;
                    before = __shfl(to, one) - __shfl(v, one);
                }
                if (past)
                    break;
                behind = __shfl(to, 63);
            }
            break;
        }
    }
    int past = INT_MAX, behind = -1;
    double base = before;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        double mass = base + upto[k];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            mass += w < wave ? sums[0][k][w] : 0.0;
            base += sums[0][k][w];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            mass += r[k][e];
            if (r[k][e] > 0.0) {
                behind = Part::column(k) + e;
                if (mass > goal && past == INT_MAX)
                    past = behind;
            }
        }
    }
    // (by one lane of each wave: of 64 an atomic takes one at a time)
#pragma unroll 1
    for (int lanes = 1; lanes < 64; lanes <<= 1) {
        past = min(past, __shfl_xor(past, lanes));
        behind = max(behind, __shfl_xor(behind, lanes));
    }
    if (lane == 0) {
        atomicMin(&token, past);
        atomicMax(&last, behind);
    }
    __syncthreads();
    if (threadIdx.x == 0)
        a.out[i * a.ldo + j] = at * kVerifyDraw + (token != INT_MAX ? token : last);
}

template <typename T>
hipError_t verify(const VerifyArgs &a, hipStream_t s)
{
    // as many items for each workgroup
    const uint32_t items = (uint32_t)a.N * (uint32_t)a.chunks * (uint32_t)a.slots;
    const uint32_t rounds = (items + kRowGroups - 1) / kRowGroups;
    hipLaunchKernelGGL((verify_rows_kernel<T>), dim3((items + rounds - 1) / rounds), dim3(kThreads), 0, s, a, items);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int judges = std::min(a.K + 1, kMostJudges);
    hipLaunchKernelGGL((verify_judge_kernel<T>), dim3((unsigned)a.N), dim3(64 * judges), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    hipLaunchKernelGGL((verify_draw_kernel<T>), dim3((unsigned)a.N * (unsigned)a.draws), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(const VerifyArgs &a, hipStream_t s)
{
    return a.bf16 ? verify<bf16_t>(a, s) : verify<float>(a, s);
}

}  // namespace sbk
