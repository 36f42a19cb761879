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
// a group, lane (p, r) holds a quarter of channel r's: its 16 (or 8) bytes are
// two nibbles a byte in K order, eight nibbles a dword. The group's MFMA sum begins
// at -(16 + z) sum_k x, with sum_k x formed once when x goes to LDS, and meets the
// scale in one fma.
//
// At few tokens the weights' read is all the work. A wave holds 512 columns of 16
// channels and refills each register with the next 512's as soon as it is used;
// scales and zero points come with one load each for four groups, a lane's quarter
// saying which, and are spread by a permute (a load of two bytes for each group
// took 84 us where this takes 68: 1 token, 262144 channels, K = 2816, 392 MB;
// without any scales 61). The weights' buffer resources are forced into scalar
// registers (74 -> 68 us without per-lane loops around the loads). K is split over
// 1 to 16 waves of a workgroup by an estimate, rounds of the chip times groups a
// wave; their sums meet in LDS. Larger batches held (8 groups a wave) were slower
// at small sizes and level at the LM head.
//
// Up to 16 tokens whose x fits LDS whole (w4_whole_kernel): tiled weights, g 128,
// fp16, in a graph over rotated matrices (medians): 1 token x 4096 channels x 2816
// 5.0 us, 16 x 11264 x 4096 11.6 (the activations' way into every workgroup's LDS,
// 131 KB, is part of it; 176 workgroups of 64 channels, so 80 of the chip's 256
// compute units have none), LM head 1 / 5 / 16 tokens 64 / 68 / 82 us (6.1 / 5.8 /
// 4.8 TB/s). Else x goes through LDS in chunks (w4_chunk_kernel): 2 x 4096 x 65536
// 32 us, LM head 32 / 64 tokens 106 / 155 us, where unpacking, the scales' fma and
// the MFMA share the time (a chunk of 512 columns of 64 tokens takes a workgroup
// 2.2 us, 0.8 for each group's products of a wave, the rest the staging of x, again
// for each turn of channels).
#include "gemm_common.hpp"
#include "step_end.hpp"
#include "w4_few_plan.hpp"

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

// Eight values in the codes' order.
__device__ inline uint4 in_code_order(uint4 v)
{
    return make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                      __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u));
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

// Groups of 64 go in pairs: 128 columns are a wave's unit in any case.
template <int G>
constexpr int kPair = 128 / G;

// The group of K that is a wave's i-th, as one of 1 << split waves.
template <int G>
__device__ inline int group_of(int i, int parts, int part)
{
    return i / kPair<G> * kPair<G> * parts + part * kPair<G> + i % kPair<G>;
}

// The quarter of a group that a lane holds: its own, or, in groups of 64, the one
// that row-major weights leave it after their exchange (see load_codes), in both
// layouts, whose results then have the same bits.
template <int G>
__device__ inline int quarter(int lane)
{
    const int p = lane >> 4;
    return G == 64 ? (p & 1) * 2 + (p >> 1) : p;
}

// Eight values of a token at column k8 * 8, at any alignment of the element.
template <class Tx>
__device__ inline uint4 get_x(const W4FewArgs &a, int t, int k8)
{
    uint4 v;
    __builtin_memcpy(&v, (const char *)a.x + (size_t)t * a.ldx * sizeof(Tx) + (uint32_t)k8 * 16u, 16);
    return v;
}

// The two values of a word onto s, exact products with one (subnormals count).
template <class Tx>
__device__ inline float pair_sum(uint32_t w, float s)
{
    typedef Tx pair __attribute__((ext_vector_type(2)));
    const pair one = {(Tx)1.0f, (Tx)1.0f}, v = __builtin_bit_cast(pair, w);
    if constexpr (Codes<Tx>::kTop == 6)
        return __builtin_amdgcn_fdot2(v, one, s, false);
    else
        return __builtin_amdgcn_fdot2_f32_bf16(v, one, s, false);
}

// The call of this workgroup's tokens alone.
__device__ inline W4FewArgs own_tokens(W4FewArgs a, int tokens)
{
    const int t0 = (int)blockIdx.y * tokens;
    a.x = (const char *)a.x + (size_t)t0 * a.ldx * 2;
    a.y = (char *)a.y + (size_t)t0 * a.ldy * (a.y_type == DGW4_F32 ? 4 : 2);
    a.T = min(tokens, a.T - t0);
    return a;
}

template <int CTRL>
__device__ inline float dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// The sum of a group's values, eight of them in each of G / 8 neighbouring lanes.
template <class Tx, int G>
__device__ inline float group_sum(uint4 v)
{
    float s = pair_sum<Tx>(v.y, pair_sum<Tx>(v.x, 0.0f)) + pair_sum<Tx>(v.w, pair_sum<Tx>(v.z, 0.0f));
    s += dpp<0xB1>(s);                           // quad_perm: the neighbour
    s += dpp<0x4E>(s);                           // quad_perm: the other pair
    s += dpp<0x141>(s);                          // row_half_mirror: the other four of eight
    if constexpr (G == 128)
        s += dpp<0x140>(s);                      // row_mirror: the other eight of sixteen
    return s;
}

// A wave's weights of 16 CB channels from n0 on, and which of its groups a batch begins with.
template <int G, bool TL, int CB>
struct Weights {
    rsrc_t q, s, z;
    int first, parts, part;     // groups group_of(first + j, parts, part)

    __device__ Weights(const W4FewArgs &a, int n0, bool live, int first_, int parts_, int part_)
        : first(first_), parts(parts_), part(part_)
    {
        // in scalar registers, which the compiler does not see by itself
        n0 = __builtin_amdgcn_readfirstlane(n0);
        const int rows = __builtin_amdgcn_readfirstlane(live ? max(0, min(16 * CB, a.N - n0)) : 0);
        const uint32_t groups = (uint32_t)a.K / G;
        q = make_rsrc(a.q + (size_t)n0 * (a.K / 2), (uint32_t)rows * (uint32_t)(a.K / 2));
        s = make_rsrc(a.s + (size_t)n0 * groups, (uint32_t)rows * groups * 2u);
        z = make_rsrc(a.z + (size_t)n0 * groups, (uint32_t)rows * groups * 2u);
    }
};

// The batch's groups j .. j + kPair - 1 of channel block c: past K or past the last
// channel, zeros. Row-major groups of 64 have 32 bytes a row; a lane reads 16 of
// the pair's 64, so that a row's lanes read them in one piece, and the lanes of
// the two groups exchange halves when they are used (paired()).
template <int G, bool TL, int CB, int H>
__device__ inline void load_codes(const W4FewArgs &a, const Weights<G, TL, CB> &w, Frag<G> (&to)[H][CB], int c, int j,
                                  int lane)
{
    const int u = group_of<G>(w.first + j, w.parts, w.part), groups = a.K / G;
    const int half = a.K / 2, r = lane & 15, p = lane >> 4;
    if constexpr (G == 64 && !TL) {
        const uint32_t past = u + (p >> 1) < groups ? 0u : 0x80000000u;
        const uint32_t at = (uint32_t)((c * 16 + r) * half + p * 16) + (uint32_t)u * (G / 2u);
        const uint4 v = load16(w.q, at | past, 0);
        to[j][c].v = make_uint2(v.x, v.y);
        to[j + 1][c].v = make_uint2(v.z, v.w);
    } else {
#pragma unroll
        for (int i = 0; i < kPair<G>; ++i) {
            const uint32_t past = u + i < groups ? 0u : 0x80000000u;
            const uint32_t at = TL ? (uint32_t)(c * 16 * half + (quarter<G>(lane) * 16 + r) * (G / 8)) +
                                         (uint32_t)(u + i) * (8u * G)
                                   : (uint32_t)((c * 16 + r) * half + p * (G / 8)) + (uint32_t)(u + i) * (G / 2u);
            to[j + i][c] = load_frag<G, TL>(w.q, at | past, 0);
        }
    }
}

// Two row-major groups of 64 as they were loaded: lanes 0 .. 31 hold the first's 32
// bytes of each row, lanes 32 .. 63 the second's. The upper lanes' first halves
// against the lower lanes' second ones, and each register is of one group.
__device__ inline void paired(Frag<64> &a, Frag<64> &b)
{
    const auto x = __builtin_amdgcn_permlane32_swap(a.v.x, b.v.x, false, false);
    const auto y = __builtin_amdgcn_permlane32_swap(a.v.y, b.v.y, false, false);
    a.v = make_uint2(x[0], y[0]);
    b.v = make_uint2(x[1], y[1]);
}

// The same for the groups j and j + 1 of a batch, where they are such.
template <int G, bool TL, int H, int CB>
__device__ inline void pair_up(Frag<G> (&w)[H][CB], int j)
{
    if constexpr (G == 64 && !TL) {
        if (j % 2 == 0) {
#pragma unroll
            for (int c = 0; c < CB; ++c)
                paired(w[j][c], w[j + 1][c]);
        }
    }
}

// Scale and zero point of channel r of block c in the batch's group j + p, in
// one word: of four groups with one load each, a lane's quarter p saying which.
template <int G, bool TL, int CB>
__device__ inline uint32_t load_scales(const W4FewArgs &a, const Weights<G, TL, CB> &w, int c, int j, int lane)
{
    const int groups = a.K / G, u = group_of<G>(w.first + j + (lane >> 4), w.parts, w.part);
    const uint32_t at = u < groups ? (uint32_t)(((c * 16 + (lane & 15)) * groups + u) * 2) : 0x80000000u;
    const uint32_t s = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(w.s, at, 0, 0);
    const uint32_t z = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(w.z, at, 0, 0);
    return s | z << 16;
}

// The word of group j for all quarters.
__device__ inline uint32_t spread(uint32_t v, int j, int lane)
{
    return (uint32_t)__builtin_amdgcn_ds_bpermute(((j & 3) * 16 + (lane & 15)) * 4, (int)v);
}

// One group: its sums of 16 TB tokens by 16 CB channels, scaled, onto acc. x: the
// lane's first vector of each token block in LDS; sums: the group's sums of x. The
// MFMA sums begin at -(16 + z) sum x.
template <class Tx, int G, int TB, int CB>
__device__ inline void add_group(f32x4 (&acc)[TB][CB], const Frag<G> (&w)[CB], const uint32_t (&scales)[CB],
                                 const char *const (&x)[TB], const float *sums, uint32_t base)
{
    typedef typename Codes<Tx>::vec vec;
    f32x4 sum[TB][CB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        const f32x4 xs = *reinterpret_cast<const f32x4 *>(sums + t * 16);
#pragma unroll
        for (int c = 0; c < CB; ++c)
            sum[t][c] = (-16.0f - half_bits((uint16_t)(scales[c] >> 16))) * xs;
    }
#pragma unroll
    for (int i = 0; i < G / 32; ++i) {
        vec q[CB];
#pragma unroll
        for (int c = 0; c < CB; ++c)
            q[c] = codes8<Tx>(frag_word<G>(w[c], i), base);
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const vec v = *reinterpret_cast<const vec *>(x[t] + i * 16);
#pragma unroll
            for (int c = 0; c < CB; ++c)
                sum[t][c] = mfma(v, q[c], sum[t][c]);
        }
    }
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int c = 0; c < CB; ++c)
            acc[t][c] += half_bits((uint16_t)scales[c]) * sum[t][c];
}

// A turn's results from its waves' sums. With waves that share channels these
// meet in LDS, AT token blocks at a time, and are added in the waves' order.
template <class Ty, int WAVES, int AT, int TB, int CB>
__device__ inline void finish_as(const W4FewArgs &a, int split, int turn, const f32x4 (&acc)[TB][CB],
                                 f32x4 (*s_red)[AT][CB][64])
{
    const int lane = threadIdx.x & 63, r = lane & 15, p = lane >> 4;
    const int wave = (int)threadIdx.x >> 6, sets = WAVES >> split;
    Ty *y = (Ty *)a.y;
    if (split == 0) {
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int c = 0; c < CB; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = t * 16 + p * 4 + i, n = ((turn * sets + wave) * CB + c) * 16 + r;
                    if (tok < a.T && n < a.N)
                        y[(size_t)tok * a.ldy + n] = (Ty)acc[t][c][i];
                }
        return;
    }
#pragma unroll
    for (int t0 = 0; t0 < TB; t0 += AT) {
        __syncthreads();
#pragma unroll
        for (int t = 0; t < AT; ++t)
#pragma unroll
            for (int c = 0; c < CB; ++c)
                s_red[wave][t][c][lane] = acc[t0 + t][c];
        __syncthreads();
        // one output at a time per thread: token i of a block, channel ch of a block
        for (int o = threadIdx.x; o < AT * sets * CB * 256; o += WAVES * 64) {
            const int ch = o & 15, i = (o >> 4) & 15, c = (o >> 8) % CB, set = (o >> 8) / CB % sets;
            const int t = (o >> 8) / CB / sets, tok = (t0 + t) * 16 + i;
            const int n = ((turn * sets + set) * CB + c) * 16 + ch;
            if (tok < a.T && n < a.N) {
                float v = 0.0f;
                for (int k = 0; k < 1 << split; ++k)
                    v += s_red[(set << split) + k][t][c][(i >> 2) * 16 + ch][i & 3];
                y[(size_t)tok * a.ldy + n] = (Ty)v;
            }
        }
    }
    __syncthreads();
}

template <int WAVES, int AT, int TB, int CB>
__device__ inline void finish(const W4FewArgs &a, int split, int turn, const f32x4 (&acc)[TB][CB],
                              f32x4 (*s_red)[AT][CB][64])
{
    switch (a.y_type) {
    case DGW4_F32: finish_as<float, WAVES>(a, split, turn, acc, s_red); break;
    case DGW4_F16: finish_as<_Float16, WAVES>(a, split, turn, acc, s_red); break;
    default: finish_as<__bf16, WAVES>(a, split, turn, acc, s_red);
    }
}

// All activations in LDS, once: rows 16 bytes off the bank period, so that the 16
// rows of a fragment fall on all banks.
template <class Tx, int G, bool TL, int WAVES, int TB, int CB>
__global__ void __launch_bounds__(WAVES * 64, 4) w4_whole_kernel(W4FewArgs all, Plan pl)
{
    const W4FewArgs a = own_tokens(all, pl.tokens);
    constexpr int H = kHeld<G>;
    extern __shared__ __attribute__((aligned(16))) char lds[];     // [T][row], then [K/G][16 TB] sums
    __shared__ f32x4 s_red[WAVES][1][CB][64];
    static_assert(sizeof s_red <= kLdsStatic, "the LDS allowance counts on it");
    const int lane = threadIdx.x & 63, r = lane & 15, p = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int parts = 1 << pl.split, part = wave & (parts - 1), set = wave >> pl.split, sets = WAVES >> pl.split;
    const int groups = a.K / G, row = a.K * 2 + 16;
    float *sums = reinterpret_cast<float *>(lds + a.T * row);
    uint32_t base = Codes<Tx>::kBase;
    asm("" : "+v"(base));
    auto source = [&](int turn, int b) {
        const bool live = turn < pl.turns;
        return Weights<G, TL, CB>(a, live ? (turn * sets + set) * 16 * CB : 0, live, b * H, parts, part);
    };

    int turn = blockIdx.x;
    Frag<G> w[H][CB];
    uint32_t scales[H / 4][CB];
    {
        const auto q = source(turn, 0);
#pragma unroll
        for (int c = 0; c < CB; ++c) {
#pragma unroll
            for (int j = 0; j < H / 4; ++j)
                scales[j][c] = load_scales(a, q, c, j * 4, lane);
#pragma unroll
            for (int j = 0; j < H; j += kPair<G>)
                load_codes(a, q, w, c, j, lane);
        }
    }
    constexpr int kAhead = 4;        // vectors of x a thread has on their way at once
    const int wide = a.K / 8, total = a.T * wide;
    for (int i0 = threadIdx.x; i0 < total; i0 += kAhead * WAVES * 64) {
        uint4 v[kAhead];
        int t[kAhead], k8[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * WAVES * 64;
            t[j] = (int)__umulhi((uint32_t)i, pl.magic);
            k8[j] = i - t[j] * wide;
            if (i < total)
                v[j] = get_x<Tx>(a, t[j], k8[j]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (i0 + j * WAVES * 64 < total) {
                const float s = group_sum<Tx, G>(v[j]);
                *reinterpret_cast<uint4 *>(lds + t[j] * row + k8[j] * 16) = in_code_order(v[j]);
                if (k8[j] % (G / 8) == 0)
                    sums[k8[j] / (G / 8) * (TB * 16) + t[j]] = s;
            }
        }
    }
    __syncthreads();
    const char *x0[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t)
        x0[t] = lds + min(t * 16 + r, a.T - 1) * row + quarter<G>(lane) * (G / 2);
    f32x4 acc[TB][CB];
    for (int b = 0; turn < pl.turns;) {
        const bool last = b == pl.batches - 1;
        const int next_turn = last ? turn + (int)gridDim.x : turn, next_b = last ? 0 : b + 1;
        const auto q = source(next_turn, next_b);
        if (b == 0) {
#pragma unroll
            for (int t = 0; t < TB; ++t)
#pragma unroll
                for (int c = 0; c < CB; ++c)
                    acc[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        uint32_t next[H / 4][CB];
#pragma unroll
        for (int j = 0; j < H / 4; ++j)
#pragma unroll
            for (int c = 0; c < CB; ++c)
                next[j][c] = load_scales(a, q, c, j * 4, lane);
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const int u = group_of<G>(b * H + j, parts, part);
            pair_up<G, TL>(w, j);
            if (u < groups) {
                const char *x[TB];
                uint32_t sc[CB];
#pragma unroll
                for (int t = 0; t < TB; ++t)
                    x[t] = x0[t] + u * (G * 2);
#pragma unroll
                for (int c = 0; c < CB; ++c)
                    sc[c] = spread(scales[j / 4][c], j, lane);
                add_group<Tx, G>(acc, w[j], sc, x, sums + u * (TB * 16) + p * 4, base);
            }
            if (j % kPair<G> == kPair<G> - 1) {
#pragma unroll
                for (int c = 0; c < CB; ++c)
                    load_codes(a, q, w, c, j - j % kPair<G>, lane);
            }
        }
#pragma unroll
        for (int j = 0; j < H / 4; ++j)
#pragma unroll
            for (int c = 0; c < CB; ++c)
                scales[j][c] = next[j][c];
        if (last)
            finish<WAVES>(a, pl.split, turn, acc, s_red);
        turn = next_turn;
        b = next_b;
    }
}

// The activations M x 512 columns at a time, in two halves of LDS: while one is
// worked on, the next columns are on their way into registers.
template <class Tx, int G, bool TL, int WAVES, int TB, int CB, int M, int SPLIT>
__global__ void __launch_bounds__(WAVES * 64, WAVES == 16 ? 4 : 2) w4_chunk_kernel(W4FewArgs all, Plan pl)
{
    const W4FewArgs a = own_tokens(all, pl.tokens);
    constexpr int H = kHeld<G>, kWide = 64 * M, kRow = kWide * 16 + 16, kMine = TB * 16 * M / WAVES;
    constexpr int parts = 1 << SPLIT, sets = WAVES >> SPLIT, kEach = H * M >> SPLIT;   // a wave's groups of a chunk
    static_assert(kEach >= kPair<G>, "a wave has 128 columns of each chunk");
    extern __shared__ __attribute__((aligned(16))) char lds[];     // 2 x ([T][kRow], then [H M][16 TB] sums)
    const int lane = threadIdx.x & 63, r = lane & 15, p = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int part = wave & (parts - 1), set = wave >> SPLIT;
    const int groups = a.K / G, bytes = a.T * kRow + H * M * TB * 64;
    uint32_t base = Codes<Tx>::kBase;
    asm("" : "+v"(base));
    auto source = [&](int turn, int b) {
        const bool live = turn < pl.turns;
        return Weights<G, TL, CB>(a, live ? (turn * sets + set) * 16 * CB : 0, live, b * H, parts, part);
    };
    // This thread's vectors of a chunk: 64 neighbouring ones of a row per wave. Where
    // a batch takes several chunks, those of two lie ready, in turn: an even number of
    // chunks, the last one maybe past K, keeps the turns in step with the batches.
    constexpr int kDepth = kEach * 2 <= H ? 2 : 1;
    uint4 held[kDepth][kMine];
    const int chunks = ((groups + H * M - 1) / (H * M) + kDepth - 1) / kDepth * kDepth;
    auto row_of = [&](int i) { return (i * WAVES + wave) / M; };
    const int mine = wave % M * 64 + lane;           // its column of vectors, the same in each row: M divides WAVES
    auto fetch = [&](int chunk, uint4 (&to)[kMine]) {
        const int k8 = min(chunk * kWide + mine, a.K / 8 - 1);      // past K: not met by a group
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            if (row_of(i) < a.T)
                to[i] = get_x<Tx>(a, row_of(i), k8);
    };
    auto store = [&](char *at, const uint4 (&from)[kMine]) {
        float *sums = reinterpret_cast<float *>(at + a.T * kRow);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int t = row_of(i);
            if (t < a.T) {
                const float s = group_sum<Tx, G>(from[i]);
                *reinterpret_cast<uint4 *>(at + t * kRow + mine * 16) = in_code_order(from[i]);
                if (lane % (G / 8) == 0)
                    sums[mine / (G / 8) * (TB * 16) + t] = s;
            }
        }
    };

    int turn = blockIdx.x, chunk = kDepth - 1, side = 0;
    Frag<G> w[H][CB];
    uint32_t scales[H / 4][CB];
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        fetch(d, held[d]);
    {
        const auto q = source(turn, 0);
#pragma unroll
        for (int c = 0; c < CB; ++c) {
#pragma unroll
            for (int j = 0; j < H / 4; ++j)
                scales[j][c] = load_scales(a, q, c, j * 4, lane);
#pragma unroll
            for (int j = 0; j < H; j += kPair<G>)
                load_codes(a, q, w, c, j, lane);
        }
    }
    f32x4 acc[TB][CB];
    for (int b = 0; turn < pl.turns;) {
        const bool last = b == pl.batches - 1;
        const int next_turn = last ? turn + (int)gridDim.x : turn, next_b = last ? 0 : b + 1;
        const auto q = source(next_turn, next_b);
        if (b == 0) {
#pragma unroll
            for (int t = 0; t < TB; ++t)
#pragma unroll
                for (int c = 0; c < CB; ++c)
                    acc[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        uint32_t next[H / 4][CB];
#pragma unroll
        for (int j = 0; j < H / 4; ++j)
#pragma unroll
            for (int c = 0; c < CB; ++c)
                next[j][c] = load_scales(a, q, c, j * 4, lane);
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const int i = b * H + j;
            if (i % kEach == 0 && i / kEach < chunks) {
                // the chunk's columns, which the loads have brought, into the half
                // that was read last before the barrier before this one
                uint4 (&these)[kMine] = held[j / kEach % kDepth];
                side ^= 1;
                store(lds + side * bytes, these);
                chunk = chunk + 1 < chunks ? chunk + 1 : 0;
                fetch(chunk, these);
                __syncthreads();
            }
            const int u = group_of<G>(i, parts, part);
            pair_up<G, TL>(w, j);
            if (u < groups) {
                const char *half = lds + side * bytes;
                const int at = group_of<G>(i % kEach, parts, part);
                const char *x[TB];
                uint32_t sc[CB];
#pragma unroll
                for (int t = 0; t < TB; ++t)
                    x[t] = half + min(t * 16 + r, a.T - 1) * kRow + quarter<G>(lane) * (G / 2) + at * (G * 2);
#pragma unroll
                for (int c = 0; c < CB; ++c)
                    sc[c] = spread(scales[j / 4][c], j, lane);
                add_group<Tx, G>(acc, w[j], sc, x,
                                 reinterpret_cast<const float *>(half + a.T * kRow) + at * (TB * 16) + p * 4, base);
            }
            if (j % kPair<G> == kPair<G> - 1) {
#pragma unroll
                for (int c = 0; c < CB; ++c)
                    load_codes(a, q, w, c, j - j % kPair<G>, lane);
            }
        }
#pragma unroll
        for (int j = 0; j < H / 4; ++j)
#pragma unroll
            for (int c = 0; c < CB; ++c)
                scales[j][c] = next[j][c];
        if (last)
            finish<WAVES>(a, SPLIT, turn, acc, reinterpret_cast<f32x4 (*)[TB][CB][64]>(lds));
        turn = next_turn;
        b = next_b;
    }
}

template <class Kern>
hipError_t start(Kern kern, LdsAllowed &allowed, const W4FewArgs &a, const Plan &pl, const Form &f, size_t lds,
                 hipStream_t st)
{
    const hipError_t err = allow_lds_here(kern, lds, allowed);
    if (err != hipSuccess)
        return err;
    const dim3 grid(pl.turns < f.resident ? pl.turns : f.resident, (a.T + pl.tokens - 1) / pl.tokens);
    kern<<<grid, dim3(f.waves * 64), lds, st>>>(a, pl);
    return hipGetLastError();
}

template <class Tx, int G, bool TL, int F>
hipError_t whole(const W4FewArgs &a, int tokens, hipStream_t st)
{
    static LdsAllowed allowed;
    constexpr Form f = kForms[F];
    const Plan pl = plan_of(f, tokens, a.K, a.N);
    return start(w4_whole_kernel<Tx, G, TL, f.waves, f.tb, f.cb>, allowed, a, pl, f, lds_of(f, tokens, a.K, G), st);
}

template <class Tx, int G, bool TL, int F>
hipError_t chunked(const W4FewArgs &a, int tokens, hipStream_t st)
{
    static LdsAllowed allowed[3];
    constexpr Form f = kForms[F];
    static_assert(f.max_split == 2 * f.step, "one instance each");
    const Plan pl = plan_of(f, tokens, a.K, a.N);
    const size_t lds = lds_of(f, tokens, a.K, G);
    switch (pl.split / f.step) {
    case 0: return start(w4_chunk_kernel<Tx, G, TL, f.waves, f.tb, f.cb, f.m, 0>, allowed[0], a, pl, f, lds, st);
    case 1: return start(w4_chunk_kernel<Tx, G, TL, f.waves, f.tb, f.cb, f.m, f.step>, allowed[1], a, pl, f, lds, st);
    default:
        return start(w4_chunk_kernel<Tx, G, TL, f.waves, f.tb, f.cb, f.m, 2 * f.step>, allowed[2], a, pl, f, lds, st);
    }
}

template <class Tx, int G, bool TL>
hipError_t by_tokens(const W4FewArgs &a, hipStream_t st)
{
    int tokens;
    switch (form_of(a.T, a.K, a.N, G, tokens)) {
    case kWhole8: return whole<Tx, G, TL, kWhole8>(a, tokens, st);
    case kWhole16: return whole<Tx, G, TL, kWhole16>(a, tokens, st);
    case kLongK: return chunked<Tx, G, TL, kLongK>(a, tokens, st);
    case kBlocks2: return chunked<Tx, G, TL, kBlocks2>(a, tokens, st);
    default: return chunked<Tx, G, TL, kBlocks4>(a, tokens, st);
    }
}

template <class Tx>
hipError_t by_layout(const W4FewArgs &a, int g, hipStream_t st)
{
    if (g == 128)
        return a.tiled ? by_tokens<Tx, 128, true>(a, st) : by_tokens<Tx, 128, false>(a, st);
    return a.tiled ? by_tokens<Tx, 64, true>(a, st) : by_tokens<Tx, 64, false>(a, st);
}

}  // namespace

hipError_t launch_w4_few(const W4FewArgs &a, int g, hipStream_t stream)
{
    return a.x_type == DGW4_F16 ? by_layout<_Float16>(a, g, stream) : by_layout<__bf16>(a, g, stream);
}

}  // namespace dgw4
