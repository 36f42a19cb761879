// Symmetric 8-bit quantisation of rows (not part of the ABI).
//
//   s = max|x| / 127 (1 if that is zero), q = clamp(rint(x / s), -127, 127),
// each operation rounded to fp32; a row with a NaN or an infinity: s = NaN,
// q = 0. The quotient's rounding to an integer decides the code, so it has to
// be the exact division's. x times the rounded reciprocal of s is off from
// the rounded quotient by at most 3 steps of fp32, |x / s| <= 127 (1 + 2^-22)
// making that less than 5e-5: the nearest integer is the same wherever the
// product lies further than that from a half. Only the vectors (8 values of a
// lane) with a value nearer to one divide.
#pragma once

#include "int8_columns.hpp"
#include "int8_common.hpp"

namespace dgw4 {
namespace {

constexpr float kNearHalf = 0.5f - 6e-5f;

template <class Tx>
struct Vec8 {
    typedef Tx type __attribute__((ext_vector_type(8)));
};

// v moved down by d elements (0 < d < 8), zeros above.
template <class V>
__device__ inline V moved_down(V v, int d)
{
    constexpr int kDwords = sizeof(V) / 4;
    typedef uint32_t dwords __attribute__((ext_vector_type(kDwords)));
    dwords u = __builtin_bit_cast(dwords, v);
    auto by = [&](int n) {
#pragma unroll
        for (int i = 0; i < kDwords; ++i)
            u[i] = i + n < kDwords ? u[(i + n) % kDwords] : 0u;
    };
    if (d & 4)
        by(kDwords / 2);
    if (d & 2)
        by(kDwords / 4);
    if (d & 1) {
        if constexpr (kDwords == 8) {
            by(1);
        } else {
#pragma unroll
            for (int i = 0; i < kDwords; ++i)
                u[i] = u[i] >> 16 | (i + 1 < kDwords ? u[(i + 1) % kDwords] << 16 : 0u);
        }
    }
    return __builtin_bit_cast(V, u);
}

// Eight values of a row from k on (0 past K), at any alignment of the element.
// Past K - 8 the row's last eight are loaded and moved, so that no load waits
// for a branch.
template <class Tx>
__device__ inline typename Vec8<Tx>::type load8(const Tx *row, int k, int K)
{
    typename Vec8<Tx>::type v{};
    if (K >= 8) {
        const int at = min(k, K - 8);
        __builtin_memcpy(&v, row + at, sizeof v);
        if (at < k)
            v = k >= K ? typename Vec8<Tx>::type{} : moved_down(v, k - at);
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (k + i < K)
                v[i] = row[k + i];
    }
    return v;
}

// The largest magnitude among eight values as fp32 bits; above those of
// infinity if there is a NaN. The 16-bit types are ranked as they are, two at
// a time: without the sign, a float's bits are in the floats' order.
__device__ inline uint32_t top8(Vec8<float>::type v)
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = max(top, __builtin_bit_cast(uint32_t, (float)v[i]) & 0x7FFFFFFFu);
    return top;
}

template <class V>
__device__ inline uint32_t top8_16(V v)
{
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    const uint4 u = __builtin_bit_cast(uint4, v);
    const uint32_t m = 0x7FFF7FFFu;
    auto mx = [](uint32_t x, uint32_t y) {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, x),
                                                                      __builtin_bit_cast(u16x2, y)));
    };
    const uint32_t t = mx(mx(u.x & m, u.y & m), mx(u.z & m, u.w & m));
    return max(t & 0xFFFFu, t >> 16);
}

__device__ inline uint32_t top8(Vec8<_Float16>::type v)
{
    const uint32_t t = top8_16(v);
    return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)t)) & 0x7FFFFFFFu;
}

__device__ inline uint32_t top8(Vec8<__bf16>::type v) { return top8_16(v) << 16; }

__device__ inline float row_scale(uint32_t top)
{
    if (top >= 0x7F800000u)
        return __builtin_nanf("");
    const float s = __fdiv_rn(__builtin_bit_cast(float, top), 127.0f);
    return s == 0.0f ? 1.0f : s;
}

// What a row's codes are made with: its scale, the scale's reciprocal (0 where
// every vector divides: 1 / s or x / s could leave fp32's normal range) and
// whether the row is finite.
struct RowScale {
    float s, inv;
    bool finite;
};

__device__ inline RowScale row_scales(uint32_t top)
{
    RowScale r;
    r.s = row_scale(top);
    r.finite = top < 0x7F800000u;
    r.inv = r.s >= 1e-30f && r.s <= 1e30f ? __fdiv_rn(1.0f, r.s) : 0.0f;
    return r;
}

template <class Tx>
__device__ inline uint2 codes8(typename Vec8<Tx>::type v, const RowScale &rs)
{
    float q[8], off = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = __fmul_rn(to_f32((Tx)v[i]), rs.inv);
        q[i] = rintf(t);
        off = fmaxf(off, fabsf(__fsub_rn(t, q[i])));
    }
    if (rs.inv == 0.0f || off > kNearHalf) {
        // here alone a quotient can pass 127: where the scale is subnormal
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[i] = fminf(fmaxf(rintf(__fdiv_rn(to_f32((Tx)v[i]), rs.s)), -127.0f), 127.0f);
    }
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        b[i] = (uint32_t)(int)q[i];
    // the low bytes of two, then of four words
    auto pair = [](uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x0C0C0400u); };
    uint2 o;
    o.x = pair(b[0], b[1]) | pair(b[2], b[3]) << 16;
    o.y = pair(b[4], b[5]) | pair(b[6], b[7]) << 16;
    return rs.finite ? o : make_uint2(0, 0);
}

// The maximum over N neighbouring lanes.
template <int N>
__device__ inline uint32_t lanes_top(uint32_t v)
{
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1)
        v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return v;
}

// A row by threads tid of N (neighbouring lanes of a wave, or a workgroup with
// room for its waves' maxima in s_part), eight values at a time: the row's codes into q[0 .. end)
// (8-byte aligned, end a multiple of 16, zero from K on); returns the scale in
// every thread. The first kKept vectors of a thread stay in registers between
// the maximum and the codes.
template <class Tx, int N, int kKept>
__device__ inline float quantize_row(const Tx *__restrict__ row, int K, int end, char *q, int tid, uint32_t *s_part)
{
    typename Vec8<Tx>::type v[kKept];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kKept; ++j)
        v[j] = load8<Tx>(row, (j * N + tid) * 8, K);
#pragma unroll
    for (int j = 0; j < kKept; ++j)
        top = max(top, top8(v[j]));
    const int rest = (kKept * N + tid) * 8;
    each_column<N * 8>(rest, K, [&](int k) { top = max(top, top8(load8<Tx>(row, k, K))); });
    top = lanes_top<(N < 64 ? N : 64)>(top);
    if constexpr (N > 64) {
        if ((tid & 63) == 0)
            s_part[tid >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N / 64; ++i)
            top = max(top, s_part[i]);
    }
    const RowScale rs = row_scales(top);
#pragma unroll
    for (int j = 0; j < kKept; ++j) {
        const int k = (j * N + tid) * 8;
        if (k < end)
            *reinterpret_cast<uint2 *>(q + k) = codes8<Tx>(v[j], rs);
    }
    each_column<N * 8>(rest, end, [&](int k) {
        *reinterpret_cast<uint2 *>(q + k) = codes8<Tx>(load8<Tx>(row, k, K), rs);
    });
    return rs.s;
}

}  // namespace
}  // namespace dgw4
