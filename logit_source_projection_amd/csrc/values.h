// Rows of fp32 or bf16 values as units of eight floats, and sums over a
// workgroup (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sbk {

// Whether `rows` rows, `ld` elements of `bytes` bytes apart, pass what 47-bit
// addresses reach.  A quotient: the product of a wild stride passes 64 bits.
inline bool spans_addresses(int64_t rows, int64_t ld, int64_t bytes)
{
    return ld > ((int64_t)1 << 47) / ((rows > 0 ? rows : 1) * bytes);
}

namespace {

typedef uint32_t raw4 __attribute__((ext_vector_type(4)));
typedef __bf16 half8 __attribute__((ext_vector_type(8)));

// Element types: float, and uint16_t for the bits of a bf16 number.
typedef uint16_t bf16_t;

__device__ __forceinline__ float value_of(float v) { return v; }
__device__ __forceinline__ float value_of(bf16_t bits) { return __uint_as_float((uint32_t)bits << 16); }
// Rounded to the type (nearest, ties to even).
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16_t *p, float v) { *p = __builtin_bit_cast(bf16_t, (__bf16)v); }

// A pointer that the compiler would not know to be to device memory (one taken out of
// a table, say): flat accesses count as LDS ones too, and loads would wait for stores.
template <typename T>
__device__ __forceinline__ T *in_memory(T *p)
{
    return (T *)(__attribute__((address_space(1))) T *)p;
}

// Eight values as they lie in memory.
template <typename T>
struct Unit;
template <>
struct Unit<float> {
    raw4 a, b;
};
template <>
struct Unit<bf16_t> {
    raw4 a;
};

__device__ __forceinline__ Unit<float> load_unit(const float *p)
{
    return {reinterpret_cast<const raw4 *>(p)[0], reinterpret_cast<const raw4 *>(p)[1]};
}
__device__ __forceinline__ Unit<bf16_t> load_unit(const bf16_t *p)
{
    return {*reinterpret_cast<const raw4 *>(p)};
}
__device__ __forceinline__ void clear(Unit<float> &u) { u.a = u.b = raw4{0u, 0u, 0u, 0u}; }
__device__ __forceinline__ void clear(Unit<bf16_t> &u) { u.a = raw4{0u, 0u, 0u, 0u}; }

__device__ __forceinline__ void values_of(const Unit<float> &u, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = __uint_as_float(u.a[e]);
        v[4 + e] = __uint_as_float(u.b[e]);
    }
}
__device__ __forceinline__ void values_of(const Unit<bf16_t> &u, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(u.a[e] << 16);
        v[2 * e + 1] = __uint_as_float(u.a[e] & 0xFFFF0000u);
    }
}

// A unit whose first n values are there; the others are 0 and not read.  (By 16, 8,
// 4 and 2 bytes, whose places are as aligned as they are long.)
__device__ __forceinline__ raw4 load_words(const uint32_t *p, int n)
{
    raw4 w = {0u, 0u, 0u, 0u};
    if (n >= 4)
        return *reinterpret_cast<const raw4 *>(p);
    if (n >= 2) {
        const uint2 two = *reinterpret_cast<const uint2 *>(p);
        w[0] = two.x;
        w[1] = two.y;
    }
    if (n & 1) {
        const uint32_t one = p[n - 1];
        w[0] = n == 1 ? one : w[0];
        w[2] = n == 3 ? one : 0u;
    }
    return w;
}
__device__ __forceinline__ Unit<float> load_some(const float *p, int n)
{
    if (n >= 8)
        return load_unit(p);
    Unit<float> u;
    const uint32_t *words = reinterpret_cast<const uint32_t *>(p);
    u.a = load_words(words, max(n, 0));
    u.b = load_words(words + 4, max(n - 4, 0));
    return u;
}
__device__ __forceinline__ Unit<bf16_t> load_some(const bf16_t *p, int n)
{
    if (n >= 8)
        return load_unit(p);
    Unit<bf16_t> u;
    u.a = load_words(reinterpret_cast<const uint32_t *>(p), max(n, 0) >> 1);
    if (n > 0 && n & 1) {
        const uint32_t one = p[n - 1];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            u.a[e] = n >> 1 == e ? one : u.a[e];
    }
    return u;
}

// The unit at column c of a row of H (>= 1) columns, in whole 16-byte loads without a
// branch: what lies behind the row's last 16 bytes is not read (the row's first ones are
// instead), and columns behind H hold anything.
__device__ __forceinline__ Unit<float> load_at(const float *row, int c, int H)
{
    return {*reinterpret_cast<const raw4 *>(row + (c < H ? c : 0)),
            *reinterpret_cast<const raw4 *>(row + (c + 4 < H ? c + 4 : 0))};
}
__device__ __forceinline__ Unit<bf16_t> load_at(const bf16_t *row, int c, int H)
{
    return {*reinterpret_cast<const raw4 *>(row + (c < H ? c : 0))};
}
// Eight values, rounded to the type.
__device__ __forceinline__ void store_unit(float *p, const float (&v)[8])
{
    raw4 a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        a[e] = __float_as_uint(v[e]);
        b[e] = __float_as_uint(v[4 + e]);
    }
    reinterpret_cast<raw4 *>(p)[0] = a;
    reinterpret_cast<raw4 *>(p)[1] = b;
}
__device__ __forceinline__ void store_unit(bf16_t *p, const float (&v)[8])
{
    half8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[e] = (__bf16)v[e];
    *reinterpret_cast<half8 *>(p) = h;
}

// The first n of eight values, rounded to the type.
__device__ __forceinline__ void store_words(uint32_t *p, const raw4 &w, int n)
{
    if (n >= 4) {
        *reinterpret_cast<raw4 *>(p) = w;
        return;
    }
    if (n >= 2)
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    if (n > 0 && n & 1)
        p[n - 1] = n == 1 ? w[0] : w[2];
}
__device__ __forceinline__ void store_some(float *p, const float (&v)[8], int n)
{
    raw4 a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        a[e] = __float_as_uint(v[e]);
        b[e] = __float_as_uint(v[4 + e]);
    }
    uint32_t *words = reinterpret_cast<uint32_t *>(p);
    store_words(words, a, n);
    if (n > 4)
        store_words(words + 4, b, n - 4);
}
__device__ __forceinline__ void store_some(bf16_t *p, const float (&v)[8], int n)
{
    half8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[e] = (__bf16)v[e];
    const raw4 w = __builtin_bit_cast(raw4, h);
    store_words(reinterpret_cast<uint32_t *>(p), w, n >> 1);
    if (n < 8 && n & 1) {
        uint32_t one = w[0];
#pragma unroll
        for (int e = 1; e < 4; ++e)
            one = n >> 1 == e ? w[e] : one;
        p[n - 1] = (bf16_t)one;
    }
}

// The value of another lane of the 16 that a DPP control reaches.
template <int CONTROL>
__device__ __forceinline__ float dpp(float v)
{
    return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), CONTROL, 0xF, 0xF, true));
}

// The sum over LANES neighbouring lanes (8, 16, 32 or 64), in each of them.  Lanes add
// what lies across the middle of ever larger groups, so that all find the same bits.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v)
{
    v += dpp<0xB1>(v);   // quad_perm [1, 0, 3, 2]
    v += dpp<0x4E>(v);   // quad_perm [2, 3, 0, 1]
    v += dpp<0x141>(v);  // row_half_mirror
    if (LANES >= 16)
        v += dpp<0x140>(v);  // row_mirror
    if (LANES >= 32)
        v += __shfl_xor(v, 16);
    if (LANES >= 64)
        v += __shfl_xor(v, 32);
    return v;
}

__device__ __forceinline__ float wave_sum(float v) { return lanes_sum<64>(v); }

template <int CONTROL>
__device__ __forceinline__ double dpp(double v)
{
    return __hiloint2double(__builtin_amdgcn_mov_dpp(__double2hiint(v), CONTROL, 0xF, 0xF, true),
                            __builtin_amdgcn_mov_dpp(__double2loint(v), CONTROL, 0xF, 0xF, true));
}

__device__ __forceinline__ double wave_sum(double v)
{
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

// The larger, NaN where one is.
__device__ __forceinline__ float most_of(float a, float b) { return __builtin_elementwise_maximum(a, b); }

__device__ __forceinline__ float wave_most(float v)
{
    v = most_of(v, dpp<0xB1>(v));
    v = most_of(v, dpp<0x4E>(v));
    v = most_of(v, dpp<0x141>(v));
    v = most_of(v, dpp<0x140>(v));
    v = most_of(v, __shfl_xor(v, 16));
    return most_of(v, __shfl_xor(v, 32));
}

}  // namespace
}  // namespace sbk
