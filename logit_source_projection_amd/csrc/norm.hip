// Layer norm of rows and its gradient (gfx950).
//
//   mean = sum_h x / H,  rstd = 1 / sqrt(sum_h (x - mean)^2 / H + eps)
//   xh = (x - mean) rstd,  y = xh w + b
//   g = dy w,  dx = rstd (g - sum_h g / H - xh sum_h g xh / H)
//   dw = sum_b dy xh,  db = sum_b dy
//
// Sums are fp32; the variance is that of the differences from the mean, not a
// difference of two large sums.  y, dx, dw and db are rounded once.
//
// Both are bound by the bytes of their rows, so a row is read once: the team of
// lanes that has it keeps it in registers (UNITS units of 8 values per lane)
// across its sums, with the next row's loads already under way.  A team is 8 to 64
// lanes of a wave for rows that fit (no barrier), else a workgroup of as many
// waves as the row needs.  Longer rows (kMostUnits) are read again for every sum.
#include "norm.h"

#include <algorithm>

#include "values.h"

namespace sbk {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMostWaves = 16;              // of a team
constexpr int64_t kMostRows = 1 << 20;      // workgroups that rows are dealt to
constexpr int kCus = 256;

// The values of a unit that n values are there of (more in whole ones), 0 behind them.
template <bool WHOLE, typename T>
__device__ __forceinline__ void values_in(const Unit<T> &u, int n, float (&v)[8])
{
    values_of(u, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = WHOLE || e < n ? v[e] : 0.f;
}

// Values c .. of a parameter, 0 behind its n last ones, `other` where there is none.
template <bool WHOLE, typename T>
__device__ __forceinline__ void load_param(const T *p, int c, int n, float (&v)[8])
{
    if (WHOLE)
        values_of(load_some(p + c, n), v);
    else
        values_in<false>(load_at(p, c, c + n), n, v);
}
template <bool WHOLE>
__device__ __forceinline__ void load_param(const void *p, bool bf16, int c, int n, float other, float (&v)[8])
{
    if (!p) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = other;
    } else if (bf16) {
        load_param<WHOLE>(static_cast<const bf16_t *>(p), c, n, v);
    } else {
        load_param<WHOLE>(static_cast<const float *>(p), c, n, v);
    }
}

// ---------------------------------------------------------------------------
// Teams.  TEAM lanes of a wave, or with TEAM 0 the whole workgroup.  WHOLE: H is a
// multiple of 8, and no unit is there in part (code for such units between the loads and
// their use cost 8192 fp32 rows of H 5120 10 us of 52).  Others load whole 16 bytes and
// clear what is behind the row where it is used: 8192 rows of H 5001 in bf16 take 35 us
// and their gradient 72; with loads of 8, 4 and 2 bytes, each waited for, 39 and 100.
// ---------------------------------------------------------------------------
template <int TEAM, int UNITS, bool WHOLE>
struct Team {
    int at, lanes;   // this lane in its team, and the team's lanes
    int64_t row;     // the team's first row and the distance to its next
    int64_t step;
    __device__ __forceinline__ Team()
    {
        if (TEAM == 0) {
            at = threadIdx.x;
            lanes = blockDim.x;
            row = blockIdx.x;
            step = gridDim.x;
        } else {
            constexpr int kTeams = kThreads / (TEAM ? TEAM : 1);
            at = threadIdx.x & (TEAM - 1);
            lanes = TEAM;
            row = (int64_t)blockIdx.x * kTeams + threadIdx.x / (TEAM ? TEAM : 1);
            step = (int64_t)gridDim.x * kTeams;
        }
    }
    __device__ __forceinline__ int column(int k) const { return 8 * (k * lanes + at); }
    // The sum over the team.  With TEAM 0 `scratch` holds a float per wave, and is free
    // again behind the team's next barrier.
    __device__ __forceinline__ float sum(float v, float *scratch) const
    {
        v = lanes_sum<TEAM ? TEAM : 64>(v);
        if (TEAM == 0) {
            if ((threadIdx.x & 63) == 0)
                scratch[threadIdx.x >> 6] = v;
            __syncthreads();
            v = scratch[0];
            for (int w = 1; w < (int)blockDim.x / 64; ++w)
                v += scratch[w];
        }
        return v;
    }
    template <typename T>
    __device__ __forceinline__ void load(const T *row, int H, Unit<T> (&v)[UNITS]) const
    {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const int c = column(k);
            if (c < H)
                v[k] = WHOLE ? load_unit(row + c) : load_at(row, c, H);
            else
                clear(v[k]);
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T *row, int H, int k, const float (&v)[8]) const
    {
        const int c = column(k);
        if (c >= H)
            return;
        if (WHOLE)
            store_unit(row + c, v);
        else
            store_some(row + c, v, H - c);
    }
};

template <typename TX, typename TY, int TEAM, int UNITS, int THREADS, bool WHOLE>
__global__ __launch_bounds__(THREADS) void norm_kernel(const NormArgs a)
{
    __shared__ float scratch[2][kMostWaves];
    const Team<TEAM, UNITS, WHOLE> team;
    const int H = a.H;
    float w[UNITS][8], s[UNITS][8];
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
        const int c = team.column(k);
        load_param<WHOLE>(a.weight, a.params_bf16, c, H - c, 1.f, w[k]);
        load_param<WHOLE>(a.bias, a.params_bf16, c, H - c, 0.f, s[k]);
    }
    Unit<TX> next[UNITS];
    if (team.row < a.B)
        team.load(static_cast<const TX *>(a.x) + team.row * a.ldx, H, next);
    for (int64_t b = team.row; b < a.B; b += team.step) {
        float v[UNITS][8], sum = 0.f;
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            values_in<WHOLE>(next[k], H - team.column(k), v[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum += v[k][e];
        }
        if (b + team.step < a.B)
            team.load(static_cast<const TX *>(a.x) + (b + team.step) * a.ldx, H, next);
        const float mean = team.sum(sum, scratch[0]) / H;
        float squares = 0.f;
#pragma unroll
        for (int k = 0; k < UNITS; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[k][e] -= mean;
                squares += team.column(k) + (WHOLE ? 0 : e) < H ? v[k][e] * v[k][e] : 0.f;
            }
        const float rstd = 1.f / sqrtf(team.sum(squares, scratch[1]) / H + a.eps);
        if (team.at == 0) {
            if (a.mean)
                a.mean[b] = mean;
            if (a.rstd)
                a.rstd[b] = rstd;
        }
        TY *y = static_cast<TY *>(a.y) + b * a.ldy;
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[k][e] = v[k][e] * rstd * w[k][e] + s[k][e];
            team.store(y, H, k, v[k]);
        }
    }
}

// dx, and the parameters' sums over the rows of the workgroup.
template <typename TX, typename TY, int TEAM, int UNITS, int THREADS, bool WHOLE>
__global__ __launch_bounds__(THREADS) void norm_grad_kernel(const NormArgs a)
{
    __shared__ float scratch[2][2][kMostWaves];
    const Team<TEAM, UNITS, WHOLE> team;
    const int H = a.H;
    float w[UNITS][8], dw[UNITS][8], db[UNITS][8];
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
        const int c = team.column(k);
        load_param<WHOLE>(a.weight, a.params_bf16, c, H - c, 1.f, w[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            dw[k][e] = db[k][e] = 0.f;
    }
    // (teams of more than 8 waves have no registers left for the next row)
    constexpr bool kAhead = THREADS <= 512;
    Unit<TX> nx[UNITS];
    Unit<TY> ng[UNITS];
    float nmean = 0.f, nrstd = 0.f;
    if (kAhead && team.row < a.B) {
        team.load(static_cast<const TX *>(a.x) + team.row * a.ldx, H, nx);
        team.load(static_cast<const TY *>(a.dy) + team.row * a.lddy, H, ng);
        nmean = a.mean_in[team.row];
        nrstd = a.rstd_in[team.row];
    }
    int parity = 0;
    for (int64_t b = team.row; b < a.B; b += team.step, parity ^= 1) {
        Unit<TX> x[UNITS];
        Unit<TY> g[UNITS];
        if (!kAhead) {
            team.load(static_cast<const TX *>(a.x) + b * a.ldx, H, x);
            team.load(static_cast<const TY *>(a.dy) + b * a.lddy, H, g);
            nmean = a.mean_in[b];
            nrstd = a.rstd_in[b];
        } else {
#pragma unroll
            for (int k = 0; k < UNITS; ++k) {
                x[k] = nx[k];
                g[k] = ng[k];
            }
        }
        const float mean = nmean, rstd = nrstd;
        if (kAhead && b + team.step < a.B) {
            team.load(static_cast<const TX *>(a.x) + (b + team.step) * a.ldx, H, nx);
            team.load(static_cast<const TY *>(a.dy) + (b + team.step) * a.lddy, H, ng);
            nmean = a.mean_in[b + team.step];
            nrstd = a.rstd_in[b + team.step];
        }
        float sum = 0.f, cross = 0.f;
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            float xv[8], gv[8];
            values_in<WHOLE>(x[k], H - team.column(k), xv);
            values_in<WHOLE>(g[k], H - team.column(k), gv);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (xv[e] - mean) * rstd;
                dw[k][e] += gv[e] * xh;
                db[k][e] += gv[e];
                sum += gv[e] * w[k][e];
                cross += gv[e] * w[k][e] * xh;
            }
        }
        if (!a.dx)
            continue;
        float m, c2;
        if (TEAM == 0) {
            // one barrier a row: the rows' scratch alternates
            sum = wave_sum(sum);
            cross = wave_sum(cross);
            if ((threadIdx.x & 63) == 0) {
                scratch[parity][0][threadIdx.x >> 6] = sum;
                scratch[parity][1][threadIdx.x >> 6] = cross;
            }
            __syncthreads();
            m = scratch[parity][0][0];
            c2 = scratch[parity][1][0];
            for (int i = 1; i < (int)blockDim.x / 64; ++i) {
                m += scratch[parity][0][i];
                c2 += scratch[parity][1][i];
            }
        } else {
            m = lanes_sum<TEAM ? TEAM : 64>(sum);
            c2 = lanes_sum<TEAM ? TEAM : 64>(cross);
        }
        m /= H;
        c2 /= H;
        TX *dx = static_cast<TX *>(a.dx) + b * a.lddx;
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            float xv[8], gv[8];
            values_in<WHOLE>(x[k], H - team.column(k), xv);
            values_in<WHOLE>(g[k], H - team.column(k), gv);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                xv[e] = rstd * (gv[e] * w[k][e] - m - (xv[e] - mean) * rstd * c2);
            team.store(dx, H, k, xv);
        }
    }
    if (!a.part)
        return;
    if (TEAM != 0) {
        // the workgroup's teams: those of a wave, then the waves in order
        __shared__ alignas(16) float joined[kWaves][2][TEAM ? 8 * TEAM * UNITS : 1];
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int k = 0; k < UNITS; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int d = TEAM; d < 64; d <<= 1) {
                    dw[k][e] += __shfl_xor(dw[k][e], d);
                    db[k][e] += __shfl_xor(db[k][e], d);
                }
        if ((threadIdx.x & 63) < TEAM)
#pragma unroll
            for (int k = 0; k < UNITS; ++k) {
                store_some(&joined[wave][0][team.column(k)], dw[k], 8);
                store_some(&joined[wave][1][team.column(k)], db[k], 8);
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * 8 * TEAM * UNITS; i += kThreads) {
            const int which = i / (8 * TEAM * UNITS), c = i % (8 * TEAM * UNITS);
            float v = joined[0][which][c];
#pragma unroll
            for (int u = 1; u < kWaves; ++u)
                v += joined[u][which][c];
            if (c < a.ldpart)
                a.part[((int64_t)blockIdx.x * 2 + which) * a.ldpart + c] = v;
        }
        return;
    }
    float *part = a.part + (int64_t)blockIdx.x * 2 * a.ldpart;
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
        const int c = team.column(k);
        if (c < H) {
            store_some(part + c, dw[k], 8);
            store_some(part + a.ldpart + c, db[k], 8);
        }
    }
}

// ---------------------------------------------------------------------------
// Few rows, in one launch: the parameters' gradients need no sum over a row, so their
// workgroups (kFewColumns units of columns, a row per kFewColumns threads) run beside the
// ones of dx, a row each.  What such a call costs is launches: 16 rows of H 5120 in bf16
// take 3.8 us, 6.9 with teams and a second launch for the sums, and the host a launch
// less.  The columns' threads walk the rows, so it is for few: 256 rows of H 5120 in
// bf16 8.7 us against 11.4, of H 8192 in fp32 11.5 against 15.5; 512 rows 16.9 against
// 12.8, and 9.0 against 6.4 at H 512.
// ---------------------------------------------------------------------------
constexpr int kFewMost = 256, kFewColumns = 16, kFewRows = kThreads / kFewColumns, kFewUnits = 4;

template <typename TX, typename TY, bool WHOLE>
__device__ __forceinline__ void few_dx(const NormArgs &a, int row, float (&scratch)[2][kMostWaves])
{
    const TX *x = static_cast<const TX *>(a.x) + row * a.ldx;
    const TY *dy = static_cast<const TY *>(a.dy) + row * a.lddy;
    TX *dx = static_cast<TX *>(a.dx) + row * a.lddx;
    const float mean = a.mean_in[row], rstd = a.rstd_in[row];
    Unit<TX> xs[kFewUnits];
    Unit<TY> gs[kFewUnits];
    float g[kFewUnits][8], xh[kFewUnits][8], sum = 0.f, cross = 0.f;
#pragma unroll
    for (int k = 0; k < kFewUnits; ++k) {
        const int c = 8 * (threadIdx.x + k * kThreads);
        xs[k] = load_at(x, c, a.H);
        gs[k] = load_at(dy, c, a.H);
        load_param<WHOLE>(a.weight, a.params_bf16, c, a.H - c, 1.f, g[k]);
    }
#pragma unroll
    for (int k = 0; k < kFewUnits; ++k) {
        const int left = a.H - 8 * (int)(threadIdx.x + k * kThreads);
        float gv[8];
        values_of(xs[k], xh[k]);
        values_of(gs[k], gv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool in = (WHOLE ? 0 : e) < left;
            g[k][e] = in ? g[k][e] * gv[e] : 0.f;
            xh[k][e] = in ? (xh[k][e] - mean) * rstd : 0.f;
            sum += g[k][e];
            cross += g[k][e] * xh[k][e];
        }
    }
    const int wave = threadIdx.x >> 6;
    sum = wave_sum(sum);
    cross = wave_sum(cross);
    if ((threadIdx.x & 63) == 0) {
        scratch[0][wave] = sum;
        scratch[1][wave] = cross;
    }
    __syncthreads();
    sum = cross = 0.f;
    for (int w = 0; w < kThreads / 64; ++w) {
        sum += scratch[0][w];
        cross += scratch[1][w];
    }
    sum /= a.H;
    cross /= a.H;
#pragma unroll
    for (int k = 0; k < kFewUnits; ++k) {
        const int c = 8 * (threadIdx.x + k * kThreads);
        float out[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            out[e] = rstd * (g[k][e] - sum - xh[k][e] * cross);
        if (c < a.H)
            store_some(dx + c, out, a.H - c);
    }
}

template <typename TX, typename TY, bool WHOLE>
__global__ __launch_bounds__(kThreads) void norm_grad_few_kernel(const NormArgs a)
{
    __shared__ float scratch[2][kMostWaves];
    __shared__ float joined[kFewRows][2][8 * kFewColumns];
    const int rows = a.dx ? a.B : 0;
    if ((int)blockIdx.x < rows) {
        few_dx<TX, TY, WHOLE>(a, blockIdx.x, scratch);
        return;
    }
    const int first = 8 * kFewColumns * ((int)blockIdx.x - rows);
    const int unit = threadIdx.x % kFewColumns, at = threadIdx.x / kFewColumns, c = first + 8 * unit;
    float weight[8] = {}, bias[8] = {};
    if (c < a.H) {
        for (int row = at; row < a.B; row += kFewRows) {
            float x[8], g[8];
            values_of(load_at(static_cast<const TX *>(a.x) + row * a.ldx, c, a.H), x);
            values_of(load_at(static_cast<const TY *>(a.dy) + row * a.lddy, c, a.H), g);
            const float mean = a.mean_in[row], rstd = a.rstd_in[row];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                weight[e] += g[e] * ((x[e] - mean) * rstd);
                bias[e] += g[e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        joined[at][0][8 * unit + e] = weight[e];
        joined[at][1][8 * unit + e] = bias[e];
    }
    __syncthreads();
    const int which = threadIdx.x / (8 * kFewColumns), column = threadIdx.x % (8 * kFewColumns);
    void *param = which ? a.dbias : a.dweight;
    if (!param || first + column >= a.H)
        return;
    float v = joined[0][which][column];
#pragma unroll
    for (int r = 1; r < kFewRows; ++r)
        v += joined[r][which][column];
    if (a.params_bf16)
        put(static_cast<bf16_t *>(param) + first + column, v);
    else
        put(static_cast<float *>(param) + first + column, v);
}
static_assert(kThreads == 2 * 8 * kFewColumns, "a thread per value of the parameters' gradients");

// ---------------------------------------------------------------------------
// Rows that no team holds: one workgroup per row, reading it once per sum.
// ---------------------------------------------------------------------------
// The sum over the workgroup; every thread has it.  `scratch` holds a float per
// wave and is free again after the next barrier.
__device__ __forceinline__ float group_sum(float v, float *scratch)
{
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0)
        scratch[threadIdx.x >> 6] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
        v += scratch[w];
    return v;
}

template <typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void norm_long_kernel(const NormArgs a)
{
    __shared__ float scratch[2][kWaves];
    const int H = a.H, units = (H + 7) / 8;
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        const TX *x = static_cast<const TX *>(a.x) + b * a.ldx;
        TY *y = static_cast<TY *>(a.y) + b * a.ldy;
        float sum = 0.f, v[8];
        for (int u = threadIdx.x; u < units; u += kThreads) {
            values_of(load_some(x + 8 * u, H - 8 * u), v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum += v[e];
        }
        const float mean = group_sum(sum, scratch[0]) / H;
        float squares = 0.f;
        for (int u = threadIdx.x; u < units; u += kThreads) {
            values_of(load_some(x + 8 * u, H - 8 * u), v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = 8 * u + e < H ? v[e] - mean : 0.f;
                squares += d * d;
            }
        }
        const float rstd = 1.f / sqrtf(group_sum(squares, scratch[1]) / H + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[b] = mean;
            if (a.rstd)
                a.rstd[b] = rstd;
        }
        for (int u = threadIdx.x; u < units; u += kThreads) {
            float w[8], s[8];
            values_of(load_some(x + 8 * u, H - 8 * u), v);
            load_param<false>(a.weight, a.params_bf16, 8 * u, H - 8 * u, 1.f, w);
            load_param<false>(a.bias, a.params_bf16, 8 * u, H - 8 * u, 0.f, s);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = (v[e] - mean) * rstd * w[e] + s[e];
            store_some(y + 8 * u, v, H - 8 * u);
        }
    }
}

// dx, a workgroup per row.
template <typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void norm_grad_rows_kernel(const NormArgs a)
{
    __shared__ float scratch[2][kWaves];
    const int H = a.H, units = (H + 7) / 8;
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        const TX *x = static_cast<const TX *>(a.x) + b * a.ldx;
        const TY *dy = static_cast<const TY *>(a.dy) + b * a.lddy;
        TX *dx = static_cast<TX *>(a.dx) + b * a.lddx;
        const float mean = a.mean_in[b], rstd = a.rstd_in[b];
        float sum = 0.f, cross = 0.f;
        float xv[8], gv[8], w[8];
        for (int u = threadIdx.x; u < units; u += kThreads) {
            const int n = H - 8 * u;
            values_of(load_some(x + 8 * u, n), xv);
            values_of(load_some(dy + 8 * u, n), gv);
            load_param<false>(a.weight, a.params_bf16, 8 * u, n, 1.f, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = e < n ? gv[e] * w[e] : 0.f;
                sum += g;
                cross += e < n ? g * ((xv[e] - mean) * rstd) : 0.f;
            }
        }
        // (both scratch arrays are free: the last read of each is a barrier away)
        const float m = group_sum(sum, scratch[0]) / H, k = group_sum(cross, scratch[1]) / H;
        for (int u = threadIdx.x; u < units; u += kThreads) {
            const int n = H - 8 * u;
            values_of(load_some(x + 8 * u, n), xv);
            values_of(load_some(dy + 8 * u, n), gv);
            load_param<false>(a.weight, a.params_bf16, 8 * u, n, 1.f, w);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                xv[e] = rstd * (gv[e] * w[e] - m - (xv[e] - mean) * rstd * k);
            store_some(dx + 8 * u, xv, n);
        }
    }
}

// The parameters' sums over one run of rows, a unit of columns per thread.
template <typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void norm_grad_columns_kernel(const NormArgs a)
{
    const int u = blockIdx.x * kThreads + threadIdx.x, n = a.H - 8 * u;
    if (n <= 0)
        return;
    float dw[8] = {}, db[8] = {};
    for (int64_t b = blockIdx.y; b < a.B; b += gridDim.y) {
        float xv[8], gv[8];
        values_of(load_some(static_cast<const TX *>(a.x) + b * a.ldx + 8 * u, n), xv);
        values_of(load_some(static_cast<const TY *>(a.dy) + b * a.lddy + 8 * u, n), gv);
        const float mean = a.mean_in[b], rstd = a.rstd_in[b];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw[e] += gv[e] * ((xv[e] - mean) * rstd);
            db[e] += gv[e];
        }
    }
    float *part = a.part + (int64_t)blockIdx.y * 2 * a.ldpart + 8 * u;
    store_some(part, dw, 8);
    store_some(part + a.ldpart, db, 8);
}

// ---------------------------------------------------------------------------
// dw and db: the runs' sums added in order.  A workgroup has kJoinColumns columns of
// one of them; each of its kJoinRuns groups of threads adds an equal share of the
// runs in order, and the shares are added in order.  32 columns: 1333 rows of H 1111 in
// fp32 15.0 us with the launch before, 8192 rows of H 2048 in bf16 26.3; 64: 16.1 and 27.9.
// ---------------------------------------------------------------------------
constexpr int kJoinColumns = 32, kJoinQuads = kJoinColumns / 4, kJoinRuns = kThreads / kJoinQuads;

__global__ __launch_bounds__(kThreads) void norm_params_kernel(const NormArgs a)
{
    __shared__ alignas(16) float shares[kJoinRuns][kJoinColumns];
    const bool bias = blockIdx.y != 0;
    void *to = bias ? a.dbias : a.dweight;
    if (!to)
        return;
    const int quad = threadIdx.x % kJoinQuads, share = threadIdx.x / kJoinQuads;
    const int c = blockIdx.x * kJoinColumns + 4 * quad;
    const int each = (a.parts + kJoinRuns - 1) / kJoinRuns, last = min(a.parts, (share + 1) * each);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < a.H) {
        const float *part = a.part + bias * a.ldpart + c;
#pragma unroll 8
        for (int p = share * each; p < last; ++p) {
            const float4 o = *reinterpret_cast<const float4 *>(part + (int64_t)2 * p * a.ldpart);
            v.x += o.x;
            v.y += o.y;
            v.z += o.z;
            v.w += o.w;
        }
    }
    *reinterpret_cast<float4 *>(&shares[share][4 * quad]) = v;
    __syncthreads();
    const int at = blockIdx.x * kJoinColumns + threadIdx.x;
    if (threadIdx.x >= kJoinColumns || at >= a.H)
        return;
    float sum = shares[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kJoinRuns; ++i)
        sum += shares[i][threadIdx.x];
    if (a.params_bf16)
        put(static_cast<bf16_t *>(to) + at, sum);
    else
        put(static_cast<float *>(to) + at, sum);
}

// ---------------------------------------------------------------------------
// Launches.
// ---------------------------------------------------------------------------
struct Shape {
    int team, units, threads, teams;  // teams per workgroup
};

constexpr int kMostUnits = 64 * kMostWaves * 2;  // of a row that a team holds

Shape shape_of(int H)
{
    const int units = (H + 7) / 8;
    for (int team = 8; team <= 64; team <<= 1)
        if (units <= team)
            return {team, 1, kThreads, kThreads / team};
    if (units <= 128)
        return {64, 2, kThreads, kWaves};
    return {0, 2, (units + 127) / 128 * 64, 1};
}

// Workgroups that rows are dealt to: as many as put `waves` waves on every CU (one
// workgroup on each at least).  The loads of the next row are under way while one is
// summed, so few waves suffice and more only add ends: forward of 8192 rows of H 5120
// in bf16 30 us with 16 waves per CU, 36 with 32, 53 with 8; gradient 52 us with 8,
// 58 with 10, 63 with 16 (each workgroup leaves a row of partial sums).
constexpr int kForwardWaves = 16, kGradWaves = 8;

int groups_of(const Shape &t, int64_t B, int waves)
{
    const int64_t all = (B + t.teams - 1) / t.teams;
    const int64_t resident = kCus * (int64_t)std::max(1, waves * 64 / t.threads);
    return (int)std::min(all, resident);
}

// RUN(team, units, most threads) of the shape t.
#define SHAPES \
    if (t.team == 8) \
        RUN(8, 1, kThreads); \
    else if (t.team == 16) \
        RUN(16, 1, kThreads); \
    else if (t.team == 32) \
        RUN(32, 1, kThreads); \
    else if (t.team == 64 && t.units == 1) \
        RUN(64, 1, kThreads); \
    else if (t.team == 64) \
        RUN(64, 2, kThreads); \
    else if (t.threads <= 512) \
        RUN(0, 2, 512); \
    else \
        RUN(0, 2, 64 * kMostWaves);

template <typename TX, typename TY, bool WHOLE>
hipError_t forward(const NormArgs &a, hipStream_t s)
{
    if ((a.H + 7) / 8 > kMostUnits) {
        hipLaunchKernelGGL((norm_long_kernel<TX, TY>), dim3((unsigned)std::min<int64_t>(a.B, kMostRows)), dim3(kThreads), 0, s, a);
        return hipGetLastError();
    }
    const Shape t = shape_of(a.H);
    const dim3 grid((unsigned)groups_of(t, a.B, kForwardWaves)), threads(t.threads);
#define RUN(TEAM, UNITS, MOST) \
    hipLaunchKernelGGL((norm_kernel<TX, TY, TEAM, UNITS, MOST, WHOLE>), grid, threads, 0, s, a)
    SHAPES
#undef RUN
    return hipGetLastError();
}

template <typename TX, typename TY, bool WHOLE>
hipError_t gradient(const NormArgs &a, hipStream_t s)
{
    if (norm_grad_few(a.B, a.H)) {
        const int chunks = a.dweight || a.dbias ? (a.H + 8 * kFewColumns - 1) / (8 * kFewColumns) : 0;
        hipLaunchKernelGGL((norm_grad_few_kernel<TX, TY, WHOLE>), dim3((unsigned)((a.dx ? a.B : 0) + chunks)),
                           dim3(kThreads), 0, s, a);
        return hipGetLastError();
    }
    if ((a.H + 7) / 8 <= kMostUnits) {
        const Shape t = shape_of(a.H);
        const dim3 grid((unsigned)norm_parts(a.B, a.H)), threads(t.threads);
#define RUN(TEAM, UNITS, MOST) \
    hipLaunchKernelGGL((norm_grad_kernel<TX, TY, TEAM, UNITS, MOST, WHOLE>), grid, threads, 0, s, a)
        SHAPES
#undef RUN
        return hipGetLastError();
    }
    if (a.dx) {
        hipLaunchKernelGGL((norm_grad_rows_kernel<TX, TY>), dim3((unsigned)std::min<int64_t>(a.B, kMostRows)), dim3(kThreads), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || !a.part)
            return e;
    }
    const unsigned chunks = (unsigned)(((a.H + 7) / 8 + kThreads - 1) / kThreads);
    hipLaunchKernelGGL((norm_grad_columns_kernel<TX, TY>), dim3(chunks, (unsigned)norm_parts(a.B, a.H)),
                       dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

bool norm_grad_few(int32_t B, int32_t H) { return B <= kFewMost && H <= 8 * kFewUnits * kThreads; }

int norm_parts(int32_t B, int32_t H)
{
    if (norm_grad_few(B, H))
        return 0;
    if ((H + 7) / 8 > kMostUnits)
        return std::min(B, 256);
    return groups_of(shape_of(H), B, kGradWaves);
}

// call<TX, TY, WHOLE>(a, s) of the call's types.
#define OF_TYPES(call) \
    const bool whole = a.H % 8 == 0; \
    if (a.x_bf16 && a.y_bf16) \
        return whole ? call<bf16_t, bf16_t, true>(a, s) : call<bf16_t, bf16_t, false>(a, s); \
    if (a.x_bf16) \
        return whole ? call<bf16_t, float, true>(a, s) : call<bf16_t, float, false>(a, s); \
    if (a.y_bf16) \
        return whole ? call<float, bf16_t, true>(a, s) : call<float, bf16_t, false>(a, s); \
    return whole ? call<float, float, true>(a, s) : call<float, float, false>(a, s);

hipError_t launch_norm(const NormArgs &a, hipStream_t s) { OF_TYPES(forward) }
hipError_t launch_norm_grad(const NormArgs &a, hipStream_t s) { OF_TYPES(gradient) }

hipError_t launch_norm_params(const NormArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(norm_params_kernel, dim3((unsigned)((a.H + kJoinColumns - 1) / kJoinColumns), 2),
                       dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace sbk
