// 8-bit rows with one scale each, and their products.
#include "gemm_common.hpp"

#include "dgw4.h"

namespace dgw4 {
namespace {

// every rounding below is stated in the header: no product is folded into a
// sum or a conversion
#pragma clang fp contract(off)

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ inline float to_f32(float v) { return v; }
__device__ inline float to_f32(_Float16 v) { return (float)v; }
__device__ inline float to_f32(__bf16 v)
{
    return __builtin_bit_cast(float, (uint32_t)__builtin_bit_cast(uint16_t, v) << 16);
}

// One workgroup per row; the row is read twice, the second time from the
// caches.
template <class Tp>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const Tp *__restrict__ x, int K, long long ldx,
                                                            int8_t *__restrict__ q, long long ldq,
                                                            float *__restrict__ s)
{
    __shared__ uint32_t s_top[4];
    const size_t row = blockIdx.x;
    const Tp *xr = x + row * ldx;
    uint32_t top = 0;
    for (int k = threadIdx.x; k < K; k += 256)
        top = max(top, __builtin_bit_cast(uint32_t, to_f32(xr[k])) & 0x7FFFFFFFu);
    for (int o = 32; o > 0; o >>= 1)
        top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if ((threadIdx.x & 63) == 0)
        s_top[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
    const bool finite = top < 0x7F800000u;
    float sc = __fdiv_rn(__builtin_bit_cast(float, top), 127.0f);
    if (sc == 0.0f)
        sc = 1.0f;
    const int Kp = (K + 15) / 16 * 16;
    for (int k = threadIdx.x; k < Kp; k += 256) {
        float v = 0.0f;
        if (k < K && finite)
            v = fminf(fmaxf(rintf(__fdiv_rn(to_f32(xr[k]), sc)), -127.0f), 127.0f);
        q[row * ldq + k] = (int8_t)(int)v;
    }
    if (threadIdx.x == 0)
        s[row] = finite ? sc : __builtin_nanf("");
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

// A wave per 16 rows x 16 channels, K in steps of 64 from global memory.
template <class Ty>
__global__ void __launch_bounds__(64) w8a8_simple_kernel(I8Args a)
{
    const int lane = threadIdx.x;
    const int r = lane & 15, p = lane >> 4;
    const int n0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
    const int n = n0 + r, t = t0 + r;
    const int8_t *xp = a.xq + (size_t)min(t, a.T - 1) * a.ldx;
    const int8_t *wp = a.wq + (size_t)min(n, a.N - 1) * a.ldw;
    i32x4 acc = {0, 0, 0, 0};
    for (int k = 0; k < a.K; k += 64) {
        i32x4 xv = {0, 0, 0, 0}, wv = {0, 0, 0, 0};
        const int at = k + p * 16;
        if (at < a.K) {
            xv = *(const i32x4 *)(xp + at);
            wv = *(const i32x4 *)(wp + at);
        }
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, xv, acc, 0, 0, 0);
    }
    if (t >= a.T)
        return;
    const float xs = a.xs[t];
    Ty *y = (Ty *)a.y + (size_t)t * a.ldy;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = n0 + 4 * p + i;
        if (c < a.N)
            y[c] = from_f32<Ty>(__fmul_rn(__fmul_rn((float)acc[i], xs), a.ws[c]));
    }
}

}  // namespace

hipError_t launch_quantize_rows(const void *x, int type, int rows, int K, long long ldx, int8_t *q,
                                long long ldq, float *s, hipStream_t stream)
{
    const dim3 grid(rows), block(256);
    if (type == DGW4_F32)
        quantize_rows_kernel<float><<<grid, block, 0, stream>>>((const float *)x, K, ldx, q, ldq, s);
    else if (type == DGW4_F16)
        quantize_rows_kernel<_Float16><<<grid, block, 0, stream>>>((const _Float16 *)x, K, ldx, q, ldq, s);
    else
        quantize_rows_kernel<__bf16><<<grid, block, 0, stream>>>((const __bf16 *)x, K, ldx, q, ldq, s);
    return hipGetLastError();
}

hipError_t launch_w8a8_linear(const I8Args &a, hipStream_t stream)
{
    const dim3 grid((a.N + 15) / 16, (a.T + 15) / 16), block(64);
    if (a.type == DGW4_F32)
        w8a8_simple_kernel<float><<<grid, block, 0, stream>>>(a);
    else if (a.type == DGW4_F16)
        w8a8_simple_kernel<_Float16><<<grid, block, 0, stream>>>(a);
    else
        w8a8_simple_kernel<__bf16><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace dgw4
