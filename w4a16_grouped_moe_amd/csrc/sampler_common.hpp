// What the samplers share (not part of the ABI): the noise and the partial of a
// part of a row.
#pragma once

#include "dgw4_internal.hpp"

namespace dgw4 {
namespace {

struct Partial {
    float m, z, s;                                 // max, sum exp(l - m), sum exp(l - m) * (l - m)
    float av;                                      // argmax value and index
    int ai;
    float sv;                                      // best Gumbel score and index
    int si;
    int pad;
};
static_assert(sizeof(Partial) == 32, "partial layout");

__device__ inline void philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                     uint32_t k1, uint32_t (&out)[4])
{
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        if (r > 0) {
            k0 += 0x9E3779B9u;
            k1 += 0xBB67AE85u;
        }
        // each full 64-bit product in one v_mad_u64_u32 (instead of a
        // separate high and low multiply, both quarter rate)
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
        const uint32_t h0 = (uint32_t)(p0 >> 32), l0 = (uint32_t)p0;
        const uint32_t h1 = (uint32_t)(p1 >> 32), l1 = (uint32_t)p1;
        const uint32_t n0 = h1 ^ c1 ^ k0, n2 = h0 ^ c3 ^ k1;
        c0 = n0;
        c1 = l1;
        c2 = n2;
        c3 = l0;
    }
    out[0] = c0;
    out[1] = c1;
    out[2] = c2;
    out[3] = c3;
}

// G = -log(-log U) through the hardware base-2 logarithm (v_log_f32).
// U = (floor(w / 2^9) + 1/2) 2^-23 takes 23 bits so that every value is an
// exact fp32 number: it lies in [2^-24, 1 - 2^-24], never 0 or 1 (24 bits
// would round the top value, 2^24 - 1/2, up to 2^24 and give U = 1, an
// infinite score). -log U is then in [6.0e-8, 16.7], both ends normal, so no
// range handling is needed; the log's error is below one ulp of the score.
__device__ inline float gumbel(uint32_t w)
{
    constexpr float kLn2 = 0.693147180559945309f;
    const float u = ((float)(w >> 9) + 0.5f) * (1.0f / 8388608.0f);
    const float e = -kLn2 * __builtin_amdgcn_logf(u);
    return -kLn2 * __builtin_amdgcn_logf(e);
}

}  // namespace
}  // namespace dgw4
