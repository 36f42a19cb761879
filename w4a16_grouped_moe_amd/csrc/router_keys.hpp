// The order in which router logits are ranked, shared by the router and the
// few-token layer (not part of the ABI).
#pragma once

#include "dgw4_internal.hpp"

namespace dgw4 {
namespace {

// A logit's bits as an unsigned integer in the floats' order: negative values
// complemented, non-negative ones with the top bit set; -0 as +0.
__device__ inline uint32_t order_key(float v)
{
    uint32_t b = __builtin_bit_cast(uint32_t, v);
    if (b == 0x80000000u)
        b = 0u;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

}  // namespace
}  // namespace dgw4
