// Conversions between fp32 and the element types of activations, logits and
// outputs (not part of the ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dgw4 {
namespace {

__device__ inline float to_f32(float v) { return v; }
__device__ inline float to_f32(_Float16 v) { return (float)v; }
__device__ inline float to_f32(__bf16 v)
{
    return __builtin_bit_cast(float, (uint32_t)__builtin_bit_cast(uint16_t, v) << 16);
}

// v rounded to Ty. The empty asm keeps the fp32 rounding of the product before
// it: the compiler would otherwise form the product and its fp16 rounding in
// one v_fma_mixlo_f16.
template <class Ty>
__device__ inline Ty from_f32(float v)
{
    asm("" : "+v"(v));
    return (Ty)v;
}

}  // namespace
}  // namespace dgw4
