// The product straight from a few tokens' activations (up to 6), y[t, n] = xs[t]
// ws[n] sum_k xq wq, xs and xq quantised on the way.
//
// The weights, read once, are all the work. Every workgroup quantises the
// tokens into LDS, rows 16 bytes off the bank period so that the 16 rows of an
// MFMA fragment fall on all banks, zero past K. It takes 16 channels at a time,
// its eight waves every eighth 128 bytes of K each; a wave holds six fragments
// of weights (16 channels x 64 bytes) and refills each with the next step's as
// soon as it has been used. v_mfma_i32_16x16x64_i8 takes the channels as its row
// operand; the waves' sums meet in LDS (integers: their order is of no matter).
//
// The workgroups running at one time read neighbouring rows (turn i goes to
// workgroup i % grid). At 262144 channels of K = 2816 one token takes 126 us,
// 5.9 TB/s of weights, five 135; giving each workgroup one contiguous run of
// channels took 133 us, more loads in flight (8 or 12 fragments a wave) or
// copies into LDS in whole lines changed nothing, and non-temporal loads cost
// 12 us. Codes at hand go through the tiles (int8_gemm.hip): from 9 tokens, or
// with short rows, those are as fast or faster (25 tokens, 32768 channels, K
// 1024: 8.7 us against 12.1 here), with fewer and K = 2816 within half a
// microsecond.
#include "int8_common.hpp"
#include "int8_quant.hpp"

namespace dgw4 {
namespace {

constexpr int kI8Threads = 512, kI8Waves = kI8Threads / 64;
constexpr int kUnit = 128;               // bytes of K a wave takes at a time (whole cache lines)
constexpr int kHeld = 3;                 // units in flight per wave

__host__ __device__ constexpr int code_stride(int K) { return (K + kUnit - 1) / kUnit * kUnit + 16; }

// The tokens' codes into LDS, zero from K to the end of its last unit, and the
// scales: quantised from activations of type Tx by the whole workgroup, eight
// values a thread at a time. The codes' rows are whole 128 bytes, so sixteen
// neighbouring threads always share a row; the first kKeep vectors of a thread
// stay in registers between the rows' maxima and the codes.
template <class Tx>
__device__ inline void codes_from(const I8FewArgs &a, char *codes, float *s_xs, uint32_t *s_top, RowScale *s_rs)
{
    constexpr int kKeep = 4;
    const int stride = code_stride(a.g.K), pieces = (stride - 16) / 8;
    const int total = a.g.T * pieces;
    if ((int)threadIdx.x < a.g.T)
        s_top[threadIdx.x] = 0u;
    __syncthreads();
    typename Vec8<Tx>::type v[kKeep];
    // i / pieces, exact for i * pieces < 2^32: i < total <= 2400 here
    auto row_of = [&](int i) { return (int)__umulhi((uint32_t)i, a.row_magic); };
    auto load = [&](int i) {
        const int t = row_of(i), k = (i - t * pieces) * 8;
        return load8<Tx>(reinterpret_cast<const Tx *>(a.x) + (size_t)t * a.ld, k, a.k_x);
    };
    auto rank = [&](typename Vec8<Tx>::type q, int i) {
        uint32_t top = top8(q);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            top = max(top, (uint32_t)__shfl_xor((int)top, o));
        if ((threadIdx.x & 15) == 0)
            atomicMax(&s_top[row_of(i)], top);
    };
    // total is a multiple of 16: a group of 16 threads is in or out together
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int i = (int)threadIdx.x + j * kI8Threads;
        if (i < total)
            v[j] = load(i);
    }
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int i = (int)threadIdx.x + j * kI8Threads;
        if (i < total)
            rank(v[j], i);
    }
    for (int i = (int)threadIdx.x + kKeep * kI8Threads; i < total; i += kI8Threads)
        rank(load(i), i);
    __syncthreads();
    if ((int)threadIdx.x < a.g.T) {
        s_rs[threadIdx.x] = row_scales(s_top[threadIdx.x]);
        s_xs[threadIdx.x] = s_rs[threadIdx.x].s;
    }
    __syncthreads();
    auto emit = [&](typename Vec8<Tx>::type q, int i) {
        const int t = row_of(i), k = (i - t * pieces) * 8;
        *reinterpret_cast<uint2 *>(codes + t * stride + k) = codes8<Tx>(q, s_rs[t]);
    };
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int i = (int)threadIdx.x + j * kI8Threads;
        if (i < total)
            emit(v[j], i);
    }
    for (int i = (int)threadIdx.x + kKeep * kI8Threads; i < total; i += kI8Threads)
        emit(load(i), i);
}

template <class Ty>
__global__ void __launch_bounds__(kI8Threads, 4) i8_few_kernel(I8FewArgs a)
{
    __shared__ float s_xs[kI8FewTokens];
    __shared__ uint32_t s_top[kI8FewTokens];
    __shared__ RowScale s_rs[kI8FewTokens];
    __shared__ i32x4 s_red[2][kI8Waves][64];
    extern __shared__ __attribute__((aligned(16))) char s_codes[];    // [T][code_stride(K)]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r = lane & 15, p = lane >> 4;
    const int stride = code_stride(a.g.K);
    const int units = (a.g.K + kUnit - 1) / kUnit;
    const int items = (a.g.N + 15) / 16;                   // of 16 channels
    const int mine = (units - wave + kI8Waves - 1) / kI8Waves;    // this wave's units: wave, wave + 8, ... (maybe none)
    const int batches = (units + kI8Waves * kHeld - 1) / (kI8Waves * kHeld);
    int it = (int)blockIdx.x * a.run;

    struct Source {
        rsrc_t rsrc;
        uint32_t lane;
        int u;
    };
    // one step's weights (past the last item: none, zeros are read)
    auto source = [&](int item, int b) {
        const int i = min(item, items - 1);
        const int rows = min(16, a.g.N - i * 16);
        Source q;
        q.rsrc = make_rsrc(a.g.wq + (size_t)i * 16 * a.g.ldw,
                           item < items ? (uint32_t)(rows - 1) * (uint32_t)a.g.ldw + (uint32_t)a.g.K : 0u);
        q.lane = (uint32_t)min(r, rows - 1) * (uint32_t)a.g.ldw + (uint32_t)(p * 16);
        q.u = b * kHeld;
        return q;
    };
    // half h of the j-th unit held: past the row's end it reads the next row's
    // codes (or zero), which meet zeros of x
    auto load_weight = [&](const Source &q, int j, int h) {
        const int u = q.u + j;
        const uint32_t at = (uint32_t)((wave + u * kI8Waves) * kUnit + h * 64);
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
    case DGW4_F32: codes_from<float>(a, s_codes, s_xs, s_top, s_rs); break;
    case DGW4_F16: codes_from<_Float16>(a, s_codes, s_xs, s_top, s_rs); break;
    default: codes_from<__bf16>(a, s_codes, s_xs, s_top, s_rs);
    }
    __syncthreads();
    const char *xp = s_codes + min(r, a.g.T - 1) * stride + p * 16;
    int buf = 0;
    i32x4 acc;
    for (int b = 0; it < items;) {
        const bool last = b == batches - 1;
        const int nit = !last ? it : (it + 1) % a.run ? it + 1 : it + 1 + ((int)gridDim.x - 1) * a.run;
        const int nb = last ? 0 : b + 1;
        const Source q = source(nit, nb);
        // the scale of the channel this thread stores, ahead of the next weights
        float ws = a.g.ws[min(it * 16 + (int)(threadIdx.x & 15), a.g.N - 1)];
        asm volatile("" : : : "memory");
        if (b == 0)
            acc = i32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            // past the wave's last unit the weights are zero
            const int at = min(wave + (b * kHeld + j) * kI8Waves, units - 1) * kUnit;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                    w[j][h], *reinterpret_cast<const i32x4 *>(xp + at + h * 64), acc, 0, 0, 0);
                w[j][h] = load_weight(q, j, h);    // the next step's, into the registers just read
            }
        }
        asm volatile("" : "+v"(ws));     // waited for here, where the count of loads after it is known
        if (last) {
            s_red[buf][wave][lane] = acc;
            __syncthreads();
            // one output per thread: token i, channel c
            const int i = threadIdx.x >> 4, c = threadIdx.x & 15, n = it * 16 + c;
            if (i < a.g.T && n < a.g.N) {
                int sum = 0;
#pragma unroll
                for (int v = 0; v < kI8Waves; ++v)
                    sum += s_red[buf][v][(c >> 2) * 16 + i][c & 3];
                ((Ty *)a.g.y)[(size_t)i * a.g.ldy + n] = scaled<Ty>(sum, s_xs[i], ws);
            }
            // one barrier lies between a buffer's reads and its next writes: the
            // next item's, which no thread passes before all have read this one
            buf ^= 1;
        }
        it = nit;
        b = nb;
    }
}

template <class Ty>
hipError_t run(I8FewArgs a, hipStream_t st)
{
    const size_t lds = (size_t)a.g.T * code_stride(a.g.K);
    const int items = (a.g.N + 15) / 16;
    const int resident = 512;                    // two workgroups a compute unit
    // with many turns to share out, two neighbouring blocks of channels a turn: a
    // row's stores then fill whole cache lines in one L2 (5 tokens, 262144
    // channels of fp32: 135 -> 133.5 us; at 131072 channels the coarser turns cost 1)
    a.run = items >= 32 * resident ? 2 : 1;
    const int turns = (items + a.run - 1) / a.run;
    i8_few_kernel<Ty><<<dim3(turns < resident ? turns : resident), dim3(kI8Threads), lds, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_few(I8FewArgs a, hipStream_t stream)
{
    const uint32_t pieces = (uint32_t)(code_stride(a.g.K) - 16) / 8;
    a.row_magic = (uint32_t)(((1ull << 32) + pieces - 1) / pieces);
    return a.g.type == DGW4_F32   ? run<float>(a, stream)
           : a.g.type == DGW4_F16 ? run<_Float16>(a, stream)
                                  : run<__bf16>(a, stream);
}

}  // namespace dgw4
