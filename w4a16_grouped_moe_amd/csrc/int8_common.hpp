// Device helpers of the 8-bit sources (not part of the ABI).
#pragma once

#include "gemm_common.hpp"

#include "dgw4.h"

namespace dgw4 {
namespace {

// every rounding of the 8-bit entry points is stated in the header: no product
// is folded into a sum or a conversion
#pragma clang fp contract(off)

typedef int i32x4 __attribute__((ext_vector_type(4)));

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

// One output: the integer sum, rounded to fp32, times the token's scale, times
// the channel's, each product rounded, then rounded to Ty.
template <class Ty>
__device__ inline Ty scaled(int acc, float xs, float ws)
{
    return from_f32<Ty>(__fmul_rn(__fmul_rn((float)acc, xs), ws));
}

// Four neighbouring outputs of a row, channels c .. c + 3 of N, at any alignment
// of the element: one store (rows of odd length stay near the rate of aligned
// ones), element stores where the row ends.
template <class Ty>
__device__ inline void store4(Ty *row, int c, int N, i32x4 acc, float xs, f32x4 ws)
{
    typedef Ty ty4 __attribute__((ext_vector_type(4)));
    ty4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = scaled<Ty>(acc[i], xs, ws[i]);
    if (c + 3 < N) {
        __builtin_memcpy(row + c, &v, sizeof v);
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (c + i < N)
                row[c + i] = v[i];
    }
}

// The scales of channels c .. c + 3 (0 past N).
__device__ inline f32x4 channel_scales(const I8Args &a, int c)
{
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = c + i < a.N ? a.ws[c + i] : 0.0f;
    return v;
}

constexpr uint32_t kPast = 0x80000000u;          // an offset past every buffer here

// 64 lanes x 16 bytes from the buffer into LDS at lds (wave-uniform), lane
// after lane. No register receives the data; the caller waits on vmcnt.
__device__ inline void copy_to_lds(rsrc_t r, uint32_t voff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(r)
                 : "memory", "m0");
}

// All of this wave's LDS reads have returned and at most N of its copies are
// still in flight; then the workgroup's barrier.
template <int N>
__device__ inline void stage_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// A pointer into LDS as the byte offset that copies take.
__device__ inline uint32_t lds_offset(const void *p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

}  // namespace
}  // namespace dgw4
