// One row's symmetric 8-bit quantisation by one wave (not part of the ABI).
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

#include "int8_common.hpp"

namespace dgw4 {
namespace {

constexpr float kNearHalf = 0.5f - 6e-5f;

template <class Tx>
struct Vec8 {
    typedef Tx type __attribute__((ext_vector_type(8)));
};

// Eight values of a row from k on (0 past K), whole vectors at any alignment
// of the element.
template <class Tx>
__device__ inline typename Vec8<Tx>::type load8(const Tx *row, int k, int K)
{
    typename Vec8<Tx>::type v;
    if (k + 8 <= K) {
        __builtin_memcpy(&v, row + k, sizeof v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = k + i < K ? row[k + i] : (Tx)0.0f;
    }
    return v;
}

// The bits of the largest magnitude; above those of infinity if there is a NaN.
template <class Tx>
__device__ inline uint32_t top8(typename Vec8<Tx>::type v, uint32_t top)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = max(top, __builtin_bit_cast(uint32_t, to_f32((Tx)v[i])) & 0x7FFFFFFFu);
    return top;
}

__device__ inline float row_scale(uint32_t top)
{
    if (top >= 0x7F800000u)
        return __builtin_nanf("");
    const float s = __fdiv_rn(__builtin_bit_cast(float, top), 127.0f);
    return s == 0.0f ? 1.0f : s;
}

// Whether a row of this scale may take the reciprocal: 1 / s and x / s within
// fp32's normal range.
__device__ inline bool reciprocal_ok(float s) { return s >= 1e-30f && s <= 1e30f; }

template <class Tx>
__device__ inline uint2 codes8(typename Vec8<Tx>::type v, float s, float inv, bool fast, bool finite)
{
    float q[8], off = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = __fmul_rn(to_f32((Tx)v[i]), inv);
        q[i] = rintf(t);
        off = fmaxf(off, fabsf(__fsub_rn(t, q[i])));
    }
    if (!fast || off > kNearHalf) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[i] = rintf(__fdiv_rn(to_f32((Tx)v[i]), s));
    }
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        b[i] = (uint32_t)(int)fminf(fmaxf(q[i], -127.0f), 127.0f) & 0xFFu;
    uint2 o;
    o.x = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
    o.y = b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24;
    return finite ? o : make_uint2(0, 0);
}

__device__ inline uint32_t wave_top(uint32_t v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return v;
}

// A row by one wave into q[0 .. end) (8-byte aligned, end a multiple of 16,
// zero from K on); returns the scale, in every lane. Rows of up to 64 * 8 *
// kKept values are read once.
template <class Tx>
__device__ inline float quantize_row(const Tx *__restrict__ row, int K, int end, char *q, int lane)
{
    constexpr int kKept = 6;
    typename Vec8<Tx>::type v[kKept];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kKept; ++j)
        v[j] = load8<Tx>(row, (j * 64 + lane) * 8, K);
#pragma unroll
    for (int j = 0; j < kKept; ++j)
        top = top8<Tx>(v[j], top);
    for (int k = (kKept * 64 + lane) * 8; k < K; k += 512)
        top = top8<Tx>(load8<Tx>(row, k, K), top);
    top = wave_top(top);
    const float s = row_scale(top);
    const bool finite = top < 0x7F800000u, fast = reciprocal_ok(s);
    const float inv = __fdiv_rn(1.0f, s);
#pragma unroll
    for (int j = 0; j < kKept; ++j) {
        const int k = (j * 64 + lane) * 8;
        if (k < end)
            *reinterpret_cast<uint2 *>(q + k) = codes8<Tx>(v[j], s, inv, fast, finite);
    }
    for (int k = (kKept * 64 + lane) * 8; k < end; k += 512)
        *reinterpret_cast<uint2 *>(q + k) = codes8<Tx>(load8<Tx>(row, k, K), s, inv, fast, finite);
    return s;
}

}  // namespace
}  // namespace dgw4
