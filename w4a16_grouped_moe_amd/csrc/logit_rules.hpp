// The rules' arithmetic on one logit and the word that a column of a tile
// carries (not part of the ABI).
#pragma once

#include "step_end.hpp"

namespace dgw4 {
namespace {

// A column's word: how often its token was generated in bits 0 .. 20, whether
// the prompt holds it in bit 21, the place of its bias plus one above.
constexpr uint32_t kCount = (1u << 21) - 1, kPrompt = 1u << 21;
constexpr int kPlaceBit = 22;

// A sequence's rules.
struct Sequence {
    float repetition, frequency, presence, scale;
    const float *bias;
};

__device__ inline int sequence_of(const dgw4_logit_rules &u, int r)
{
    const int s = u.row_seq ? u.row_seq[r] : r;
    return (uint32_t)s < (uint32_t)u.sequences ? s : -1;
}

__device__ inline const uint32_t *mask_of(const dgw4_logit_rules &u, int r)
{
    if (!u.mask)
        return nullptr;
    const int m = u.mask_row ? u.mask_row[r] : r;
    return (uint32_t)m < (uint32_t)u.mask_rows ? u.mask + (long long)m * u.ld_mask : nullptr;
}

__device__ inline Sequence sequence(const dgw4_logit_rules &u, int s)
{
    Sequence q = {1.0f, 0.0f, 0.0f, 1.0f, nullptr};
    if (s >= 0) {
        q.repetition = u.repetition ? u.repetition[s] : 1.0f;
        q.frequency = u.frequency ? u.frequency[s] : 0.0f;
        q.presence = u.presence ? u.presence[s] : 0.0f;
        q.scale = u.scale ? u.scale[s] : 1.0f;
        q.bias = u.n_bias > 0 ? u.bias + (long long)s * u.ld_bias : nullptr;
    }
    return q;
}

// a * b, rounded to fp32. The empty asm keeps that rounding: the compiler would
// otherwise form the product and the sum or difference after it in one fma.
__device__ inline float rounded_product(float a, float b)
{
    float v = a * b;
    asm("" : "+v"(v));
    return v;
}

// A logit after its sequence's rules but the scale. An absent rule's constant
// changes no bits: l / 1, l - 0 * c, l - 0 and, later, l * 1 are l (-0 - 0 is -0).
__device__ inline float adjusted(float l, uint32_t word, const Sequence &q)
{
    const uint32_t c = word & kCount;
    const float penalised = l > 0.0f ? l / q.repetition : rounded_product(l, q.repetition);
    const float less = penalised - rounded_product(q.frequency, (float)c);
    l = c ? less - q.presence : word & kPrompt ? penalised : l;
    if (word >> kPlaceBit)
        l = l + q.bias[(word >> kPlaceBit) - 1];
    return l;
}

}  // namespace
}  // namespace dgw4
