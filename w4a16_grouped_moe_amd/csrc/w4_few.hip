// The dense W4A16 product for few tokens, y = x deq(W)^T.
//
// With W = (q - z) s per group of g weights along K,
//   y[t, n] = sum_j s[n, j] (sum_k (16 + q[n, k]) x[t, k] - (16 + z[n, j]) sum_k x[t, k]).
// 16 + q is one mask and one or away from the packed nibble (the nibble in the
// top mantissa bits of 16.0, in fp16 and in bf16 alike) and exact, so the MFMA
// sums exact products in fp32; the offset 16 triples the size of the terms
// against q - z, where the usual 1024 + q would cost seven bits.
//
// v_mfma_f32_16x16x32 takes 16 tokens as rows and 16 channels as columns: a lane
// holds one channel, so one scale and one zero point serve its four outputs. Of
// a group, lane (p, r) holds channel r's quarter p: its 16 (or 8) bytes are
// two nibbles a byte in K order, eight nibbles a dword.
#include "gemm_common.hpp"
#include "step_end.hpp"

namespace dgw4 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <class Tx>
struct Codes;
template <>
struct Codes<_Float16> {
    typedef f16x8 vec;
    static constexpr uint32_t kMask = 0x03C003C0u, kBase = 0x4C004C00u;
    static constexpr int kTop = 6;               // bit of the mantissa that is worth one
};
template <>
struct Codes<__bf16> {
    typedef bf16x8 vec;
    static constexpr uint32_t kMask = 0x00780078u, kBase = 0x41804180u;
    static constexpr int kTop = 3;
};

// Eight nibbles as 16 + q, in K order [0,4,1,5,2,6,3,7].
template <class Tx>
__device__ inline typename Codes<Tx>::vec codes8(uint32_t w, uint32_t base)
{
    constexpr uint32_t m = Codes<Tx>::kMask;
    constexpr int t = Codes<Tx>::kTop;
    auto to = [&](int bit) { return ((bit < t ? w << (t - bit) : w >> (bit - t)) & m) | base; };
    return __builtin_bit_cast(typename Codes<Tx>::vec, u32x4{to(0), to(4), to(8), to(12)});
}

__device__ inline f32x4 mfma(f16x8 a, f16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ inline f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ inline float half_bits(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }

// One wave: 16 channels, 16 tokens, all of K.
template <class Tx, class Ty, int G>
__global__ void __launch_bounds__(256) w4_few_kernel(W4FewArgs a)
{
    typedef typename Codes<Tx>::vec vec;
    const int lane = threadIdx.x & 63, r = lane & 15, p = lane >> 4;
    const int item = blockIdx.x * 4 + ((int)threadIdx.x >> 6), t0 = blockIdx.y * 16;
    if (item * 16 >= a.N)
        return;
    const int n = min(item * 16 + r, a.N - 1), groups = a.K / G;
    const size_t row = (size_t)a.K / 2;
    const uint8_t *q = a.tiled ? a.q + (size_t)item * 16 * row + lane * (G / 8) : a.q + (size_t)n * row + p * (G / 8);
    const size_t step = a.tiled ? 8 * G : G / 2;
    const Tx *x = (const Tx *)a.x + (size_t)min(t0 + r, a.T - 1) * a.ldx + p * (G / 4);
    uint32_t base = Codes<Tx>::kBase;
    asm("" : "+v"(base));
    vec ones;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        ones[i] = (Tx)1.0f;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < groups; ++j) {
        Frag<G> w = *reinterpret_cast<const Frag<G> *>(q + j * step);
        const float s = half_bits(a.s[(size_t)n * groups + j]), z = half_bits(a.z[(size_t)n * groups + j]);
        f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f}, xs = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < G / 32; ++i) {
            uint4 v;
            __builtin_memcpy(&v, x + j * G + i * 8, 16);
            const vec xv = __builtin_bit_cast(vec, permute8(v));
            sum = mfma(xv, codes8<Tx>(frag_word<G>(w, i), base), sum);
            xs = mfma(xv, ones, xs);
        }
        acc += s * sum - s * (16.0f + z) * xs;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + p * 4 + i;
        if (t < a.T && item * 16 + r < a.N)
            ((Ty *)a.y)[(size_t)t * a.ldy + n] = (Ty)acc[i];
    }
}

template <class Tx, class Ty>
hipError_t run(const W4FewArgs &a, int g, hipStream_t st)
{
    const dim3 grid((a.N + 63) / 64, (a.T + 15) / 16);
    if (g == 128)
        w4_few_kernel<Tx, Ty, 128><<<grid, dim3(256), 0, st>>>(a);
    else
        w4_few_kernel<Tx, Ty, 64><<<grid, dim3(256), 0, st>>>(a);
    return hipGetLastError();
}

template <class Tx>
hipError_t run_y(const W4FewArgs &a, int g, hipStream_t st)
{
    return a.y_type == DGW4_F32   ? run<Tx, float>(a, g, st)
           : a.y_type == DGW4_F16 ? run<Tx, _Float16>(a, g, st)
                                  : run<Tx, __bf16>(a, g, st);
}

}  // namespace

hipError_t launch_w4_few(const W4FewArgs &a, int g, hipStream_t stream)
{
    return a.x_type == DGW4_F16 ? run_y<_Float16>(a, g, stream) : run_y<__bf16>(a, g, stream);
}

}  // namespace dgw4
