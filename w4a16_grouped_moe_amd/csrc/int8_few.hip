// Products of 8-bit rows for few tokens (up to 32), y[t, n] = xs[t] ws[n]
// sum_k xq wq, from codes or straight from activations.
//
// The weights, read once, are all the work. The tokens' codes lie in LDS
// (quantised there from the activations, or copied), rows 16 bytes off the
// bank period so that the 16 rows of an MFMA fragment fall on all banks, zero
// past K. A wave holds six fragments of weights (16 channels x 64 bytes) and
// refills each as soon as it has been used; v_mfma_i32_16x16x64_i8 takes the
// channels as its row operand.
//
//   KS = 8: the eight waves of a workgroup share 16 channels, each taking every
//           eighth 128 bytes of K, and add their sums in LDS: short products,
//           where the time is one round trip to memory.
//   KS = 1: a wave takes 16 channels over all of K, with no barrier: many
//           channels (the LM head).
#include "int8_common.hpp"
#include "int8_quant.hpp"

namespace dgw4 {
namespace {

constexpr int kI8Threads = 512, kI8Waves = kI8Threads / 64;
constexpr int kUnit = 128;               // bytes of K a wave takes at a time (whole cache lines)
constexpr int kHeld = 3;                 // units in flight per wave

__host__ __device__ constexpr int code_stride(int K) { return (K + kUnit - 1) / kUnit * kUnit + 16; }

// The tokens' codes into LDS, zero from K to the end of its last unit, and the
// scales: quantised from activations of type Tx, a wave per row.
template <class Tx>
__device__ inline void codes_from(const I8FewArgs &a, char *codes, float *s_xs)
{
    const int lane = threadIdx.x & 63;
    const int stride = code_stride(a.g.K);
    for (int t = threadIdx.x >> 6; t < a.g.T; t += kI8Waves) {
        const Tx *row = reinterpret_cast<const Tx *>(a.x) + (size_t)t * a.ld;
        const float sc = quantize_row<Tx>(row, a.k_x, stride - 16, codes + t * stride, lane);
        if (lane == 0)
            s_xs[t] = sc;
    }
}

__device__ inline void codes_copied(const I8FewArgs &a, char *codes, float *s_xs)
{
    const int stride = code_stride(a.g.K), pieces = stride / 16 - 1;
    for (int i = threadIdx.x; i < a.g.T * pieces; i += kI8Threads) {
        const int t = i / pieces, c = i - t * pieces;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c * 16 < a.g.K)
            v = *reinterpret_cast<const uint4 *>(a.g.xq + (size_t)t * a.g.ldx + c * 16);
        *reinterpret_cast<uint4 *>(codes + t * stride + c * 16) = v;
    }
    if ((int)threadIdx.x < a.g.T)
        s_xs[threadIdx.x] = a.g.xs[threadIdx.x];
}

template <int TB, int KS, class Ty>
__global__ void __launch_bounds__(kI8Threads, 4) i8_few_kernel(I8FewArgs a)
{
    __shared__ float s_xs[16 * TB];
    __shared__ i32x4 s_red[KS == 1 ? 1 : 2][KS == 1 ? 1 : kI8Waves][TB][64];
    extern __shared__ char s_codes[];    // [T][code_stride(K)]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r = lane & 15, p = lane >> 4;
    const int stride = code_stride(a.g.K);
    const int units = (a.g.K + kUnit - 1) / kUnit;
    // this wave's items (16 channels each): a contiguous run
    const int items = (a.g.N + 15) / 16;
    const int takers = KS == 1 ? (int)gridDim.x * kI8Waves : (int)gridDim.x;
    const int me = KS == 1 ? (int)blockIdx.x * kI8Waves + wave : (int)blockIdx.x;
    const int per = items / takers, rest = items % takers;
    int it = me * per + min(me, rest);
    const int end = it + per + (me < rest ? 1 : 0);
    const int first = KS == 1 ? 0 : wave;                  // the wave's units: first, first + KS, ...
    const int mine = (units - first + KS - 1) / KS;        // (it may have none)
    const int batches = max(1, (units + KS * kHeld - 1) / (KS * kHeld));

    struct Source {
        rsrc_t rsrc;
        uint32_t lane;
        int u;
    };
    auto source = [&](int item, int b) {
        const int i = min(item, items - 1);
        const int rows = min(16, a.g.N - i * 16);
        Source q;
        q.rsrc = make_rsrc(a.g.wq + (size_t)i * 16 * a.g.ldw,
                           item < end ? (uint32_t)(rows - 1) * (uint32_t)a.g.ldw + (uint32_t)a.g.K : 0u);
        q.lane = (uint32_t)min(r, rows - 1) * (uint32_t)a.g.ldw + (uint32_t)(p * 16);
        q.u = b * kHeld;
        return q;
    };
    // half h of the j-th unit held: past the row's end it reads the next row's
    // codes (or zero), which meet zeros of x
    auto load_weight = [&](const Source &q, int j, int h) {
        const int u = q.u + j;
        const uint32_t at = (uint32_t)((first + u * KS) * kUnit + h * 64);
        return __builtin_bit_cast(i32x4, load16(q.rsrc, u < mine ? q.lane + at : 0x80000000u, 0));
    };

    i32x4 w[kHeld][2];
    {
        const Source q = source(it, 0);
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[j][h] = load_weight(q, j, h);
    }
    switch (a.x_type) {
    case DGW4_F32: codes_from<float>(a, s_codes, s_xs); break;
    case DGW4_F16: codes_from<_Float16>(a, s_codes, s_xs); break;
    case DGW4_BF16: codes_from<__bf16>(a, s_codes, s_xs); break;
    default: codes_copied(a, s_codes, s_xs);
    }
    __syncthreads();
    const bool vec = rows_in_fours<Ty>(a.g);
    const char *xp[TB];
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
        xp[tb] = s_codes + min(tb * 16 + r, a.g.T - 1) * stride + p * 16;
    int buf = 0;
    i32x4 acc[TB];
    for (int b = 0; it < end;) {
        const bool last = b == batches - 1;
        const int nit = last ? it + 1 : it, nb = last ? 0 : b + 1;
        const Source q = source(nit, nb);
        if (b == 0) {
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
                acc[tb] = i32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            // past the wave's last unit the weights are zero
            const int at = min(first + (b * kHeld + j) * KS, units - 1) * kUnit;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb)
                    acc[tb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                        w[j][h], *reinterpret_cast<const i32x4 *>(xp[tb] + at + h * 64), acc[tb], 0, 0, 0);
                w[j][h] = load_weight(q, j, h);    // the next step's, into the registers just read
            }
        }
        if (last) {
            const int n0 = it * 16;
            if constexpr (KS == 1) {
                const f32x4 ws = channel_scales(a.g, n0 + 4 * p);
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) {
                    const int t = tb * 16 + r;
                    if (t < a.g.T)
                        store4<Ty>((Ty *)a.g.y + (size_t)t * a.g.ldy, n0 + 4 * p, a.g.N, vec, acc[tb], s_xs[t], ws);
                }
            } else {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb)
                    s_red[buf][wave][tb][lane] = acc[tb];
                __syncthreads();
                // one output per thread: token i, channel c
                for (int o = threadIdx.x; o < a.g.T * 16; o += kI8Threads) {
                    const int i = o >> 4, c = o & 15;
                    if (n0 + c < a.g.N) {
                        int sum = 0;
#pragma unroll
                        for (int v = 0; v < kI8Waves; ++v)
                            sum += s_red[buf][v][i >> 4][(c >> 2) * 16 + (i & 15)][c & 3];
                        ((Ty *)a.g.y)[(size_t)i * a.g.ldy + n0 + c] = scaled<Ty>(sum, s_xs[i], a.g.ws[n0 + c]);
                    }
                }
                buf ^= 1;
            }
        }
        it = nit;
        b = nb;
    }
}

template <int TB, int KS, class Ty>
hipError_t run(const I8FewArgs &a, hipStream_t st)
{
    static size_t allowed = 24 * 1024;
    const size_t lds = (size_t)a.g.T * code_stride(a.g.K);
    const hipError_t err = allow_lds(i8_few_kernel<TB, KS, Ty>, lds, allowed);
    if (err != hipSuccess)
        return err;
    const int items = (a.g.N + 15) / 16;
    const int groups = KS == 1 ? (items + kI8Waves - 1) / kI8Waves : items;
    const int most = lds <= 24 * 1024 ? 1024 : lds <= 56 * 1024 ? 512 : 256;     // resident at once
    i8_few_kernel<TB, KS, Ty><<<dim3(groups < most ? groups : most), dim3(kI8Threads), lds, st>>>(a);
    return hipGetLastError();
}

template <class Ty>
hipError_t pick(const I8FewArgs &a, hipStream_t st)
{
    const bool wide = a.g.N >= kI8FewWideN;
    if (a.g.T <= 16)
        return wide ? run<1, 1, Ty>(a, st) : run<1, 8, Ty>(a, st);
    return wide ? run<2, 1, Ty>(a, st) : run<2, 8, Ty>(a, st);
}

}  // namespace

bool i8_few_fits(int T, int K)
{
    return T <= kI8FewTokens && (size_t)T * code_stride(K) <= 120 * 1024;
}

hipError_t launch_i8_few(const I8FewArgs &a, hipStream_t stream)
{
    return a.g.type == DGW4_F32   ? pick<float>(a, stream)
           : a.g.type == DGW4_F16 ? pick<_Float16>(a, stream)
                                  : pick<__bf16>(a, stream);
}

}  // namespace dgw4
