// Products of 8-bit rows, y[t, n] = xs[t] ws[n] sum_k xq wq,
// in LDS tiles.
//
// A workgroup takes BN channels x BT tokens and walks K in stages of 128
// bytes, ST stages deep in LDS; with few tiles KS groups of its waves take every
// KS-th stage each and add their sums through LDS (a stage costs a barrier and
// the LDS's latency whatever its size). A stage's rows (BN of W, then BT of X, 128
// bytes each, whole cache lines) are copied from global memory straight into
// LDS, 16 bytes a lane, without passing through registers; one barrier per
// stage. Position c of a row's eight 16-byte pieces holds piece c ^ (row % 8),
// chosen by the lane that loads it, so that the 16 rows one MFMA fragment
// reads at the same K fall on all banks. A lane's offset past K reads as zero
// (buffer bounds), and rows past T or N repeat the last row, their outputs not
// stored. A lane stores four channels at once at any alignment: with odd row
// lengths element stores took 65 us where this takes 37 (1690 tokens, 18679
// channels of bf16, K = 160), and 313 against 255 at 256 x 262143 x 2816.
//
// v_mfma_i32_16x16x64_i8 takes the channels as its row operand: a lane ends
// with four consecutive channels of one token. The sums are exact, so their
// order is of no matter.
//
// The 256 x 256 tile reaches 1.9 POP/s at T = 4096, K = 2816, N = 11264 (132 us;
// 704 tiles are 2.75 rounds of the chip) and 2.2 to 2.37 at K = 8192 (T = 2048, N
// = 8192). Registers-only MFMA chains on such codes run at 3.2 to 3.4 POP/s on
// the same card and 4.5 on zeros, the clock falling to 1.9 to 2.2 GHz in the
// products: the power the chip may draw bounds them, and deeper pipelines (four
// stages of 64 bytes), fragments held a half stage ahead, waves that only copy
// (with the tiles of a run overlapping their stores) and smaller tiles two to
// a CU all measured the same or slower. That is of the largest tile: the smaller
// ones' stages were not made deeper.
#include "int8_common.hpp"
#include "int8_tiles.hpp"

namespace dgw4 {
namespace {

template <int BN, int BT, int WN, int WT, int ST, int KS, class Ty>
__global__ void __launch_bounds__(KS *(BN / WN) * (BT / WT) * 64) i8_gemm_kernel(I8Args a, int tiles_n, int tiles_t)
{
    constexpr int kWaves = (BN / WN) * (BT / WT);
    constexpr int kLoadsW = BN / 8 / kWaves, kLoadsX = BT / 8 / kWaves;   // copies per wave and stage, 8 rows each
    constexpr int kLoads = kLoadsW + kLoadsX;
    constexpr int kStage = (BN + BT) * kStageK;
    constexpr int NA = WN / 16, NB = WT / 16;
    static_assert(BN % (8 * kWaves) == 0 && BT % (8 * kWaves) == 0, "whole copies for each wave");
    extern __shared__ char s_mem[];
    const int lane = threadIdx.x & 63;
    const int wave_id = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wave = wave_id % kWaves, part = wave_id / kWaves;           // part: its stages are part, part + KS, ...
    const int r = lane & 15, p = lane >> 4;

    // workgroup -> tile: an XCD (workgroups i, i + 8, ...) takes a contiguous run
    // of tiles, in groups of 8 token tiles so that the tiles in flight share
    // both their weights and their tokens in the XCD's L2
    const int total = tiles_n * tiles_t;
    const int per = total / kXcds, rest = total % kXcds;
    const int x = blockIdx.x % kXcds, i0 = blockIdx.x / kXcds;
    const int id = x * per + min(x, rest) + i0;
    const int group = id / (8 * tiles_n);
    const int gt = min(8, tiles_t - group * 8);
    const int in = id - group * 8 * tiles_n;
    const int n0 = in / gt * BN, t0 = (group * 8 + in % gt) * BT;

    // this wave's copies: 8 rows each of W, then of X
    const int rows_w = min(BN, a.N - n0), rows_x = min(BT, a.T - t0);
    const rsrc_t rw = make_rsrc(a.wq + (size_t)n0 * a.ldw, (uint32_t)(rows_w - 1) * (uint32_t)a.ldw + (uint32_t)a.K);
    const rsrc_t rx = make_rsrc(a.xq + (size_t)t0 * a.ldx, (uint32_t)(rows_x - 1) * (uint32_t)a.ldx + (uint32_t)a.K);
    const uint32_t kl = (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);      // this lane's piece of K
    uint32_t off[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        off[i] = i < kLoadsW
                     ? (uint32_t)min((wave * kLoadsW + i) * 8 + (lane >> 3), rows_w - 1) * (uint32_t)a.ldw + kl
                     : (uint32_t)min((wave * kLoadsX + i - kLoadsW) * 8 + (lane >> 3), rows_x - 1) * (uint32_t)a.ldx + kl;
    char *const s_part = s_mem + part * (ST * kStage);
    const uint32_t lds0 = lds_offset(s_part);
    const uint32_t lds_w = lds0 + (uint32_t)(wave * kLoadsW * 1024);
    const uint32_t lds_x = lds0 + (uint32_t)(BN * kStageK + wave * kLoadsX * 1024);

    const int stages = (a.K + KS * kStageK - 1) / (KS * kStageK);         // of each part; past K they read zeros
    auto issue = [&](int st, int buf) {
        const uint32_t k0 = (uint32_t)(st * KS + part) * kStageK;
        const bool in_k = k0 + kl < (uint32_t)a.K;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            copy_to_lds(i < kLoadsW ? rw : rx, in_k ? off[i] + k0 : kPast,
                        (i < kLoadsW ? lds_w + (uint32_t)(i * 1024) : lds_x + (uint32_t)((i - kLoadsW) * 1024)) +
                            (uint32_t)(buf * kStage));
    };

    i32x4 acc[NA][NB];
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[i][j] = i32x4{0, 0, 0, 0};

    const int wn = wave % (BN / WN) * WN, wt = wave / (BN / WN) * WT;
    const uint32_t fa = (uint32_t)((wn + r) * kStageK + (p ^ (r & 7)) * 16);
    const uint32_t fb = fa + (uint32_t)((BN + wt - wn) * kStageK);
#pragma unroll
    for (int st = 0; st < ST - 1; ++st)
        issue(st, st);
    int buf = 0, nbuf = ST - 1;
    for (int st = 0; st < stages; ++st) {
        stage_barrier<kLoads * (ST - 2)>();
        issue(st + ST - 1, nbuf);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            i32x4 fw[NA], fx[NB];
            // piece 4 kk + p of the row: the two halves' positions differ in bit 2
            const char *ra = s_part + ((fa + (uint32_t)(buf * kStage)) ^ (uint32_t)(kk * 64));
            const char *rb = s_part + ((fb + (uint32_t)(buf * kStage)) ^ (uint32_t)(kk * 64));
#pragma unroll
            for (int i = 0; i < NA; ++i)
                fw[i] = *reinterpret_cast<const i32x4 *>(ra + i * 16 * kStageK);
#pragma unroll
            for (int j = 0; j < NB; ++j)
                fx[j] = *reinterpret_cast<const i32x4 *>(rb + j * 16 * kStageK);
#pragma unroll
            for (int i = 0; i < NA; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[i], fx[j], acc[i][j], 0, 0, 0);
        }
        buf = buf + 1 == ST ? 0 : buf + 1;
        nbuf = nbuf + 1 == ST ? 0 : nbuf + 1;
    }
    stage_barrier<0>();                  // no copy may still land when the workgroup ends

    // the parts' sums, over the stages that no wave reads any more
    if constexpr (KS > 1) {
        static_assert((KS - 1) * kWaves * NA * NB * 1024 <= KS * ST * kStage, "the sums fit the stages");
        auto *s_sum = reinterpret_cast<i32x4 *>(s_mem);
        if (part > 0) {
#pragma unroll
            for (int i = 0; i < NA * NB; ++i)
                s_sum[(((part - 1) * kWaves + wave) * NA * NB + i) * 64 + lane] = acc[i / NB][i % NB];
        }
        __syncthreads();
        if (part > 0)
            return;
#pragma unroll
        for (int q = 0; q < KS - 1; ++q)
#pragma unroll
            for (int i = 0; i < NA * NB; ++i)
                acc[i / NB][i % NB] += s_sum[((q * kWaves + wave) * NA * NB + i) * 64 + lane];
    }

    // every scale before the first store: a load behind stores waits for them
    f32x4 ws[NA];
    float xs[NB];
#pragma unroll
    for (int i = 0; i < NA; ++i)
        ws[i] = channel_scales(a, n0 + wn + i * 16 + 4 * p);
#pragma unroll
    for (int j = 0; j < NB; ++j)
        xs[j] = a.xs[min(t0 + wt + j * 16 + r, a.T - 1)];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int t = t0 + wt + j * 16 + r;
        if (t < a.T) {
            Ty *y = (Ty *)a.y + (size_t)t * a.ldy;
#pragma unroll
            for (int i = 0; i < NA; ++i)
                store4<Ty>(y, n0 + wn + i * 16 + 4 * p, a.N, acc[i][j], xs[j], ws[i]);
        }
    }
}

template <int BN, int BT, int WN, int WT, int ST, int KS, class Ty>
hipError_t run(const I8Args &a, hipStream_t st)
{
    static LdsAllowed allowed;
    constexpr size_t lds = (size_t)KS * ST * (BN + BT) * kStageK;
    const hipError_t err = allow_lds_here(i8_gemm_kernel<BN, BT, WN, WT, ST, KS, Ty>, lds, allowed);
    if (err != hipSuccess)
        return err;
    const int tn = (a.N + BN - 1) / BN, tt = (a.T + BT - 1) / BT;
    i8_gemm_kernel<BN, BT, WN, WT, ST, KS, Ty>
        <<<dim3(tn * tt), dim3(KS * (BN / WN) * (BT / WT) * 64), lds, st>>>(a, tn, tt);
    return hipGetLastError();
}

template <class Ty>
hipError_t pick(const I8Args &a, hipStream_t st)
{
    switch (pick_tile(a.T, a.K, a.N)) {
    // one tile of tokens: waves of 128 channels x 64 tokens store longer rows
    // (T = 256, N = 262144, fp32: 244 us against 254); else 64 x 128 is level or
    // 1 to 2% faster
    case 0: return a.T <= 256 ? run<256, 256, 128, 64, 2, 1, Ty>(a, st) : run<256, 256, 64, 128, 2, 1, Ty>(a, st);
    case 1: return run<256, 128, 64, 64, 3, 1, Ty>(a, st);
    case 2: return run<128, 128, 64, 32, 4, 1, Ty>(a, st);
    case 3: return run<64, 128, 32, 64, 3, 2, Ty>(a, st);
    case 4: return run<64, 64, 32, 32, 3, 2, Ty>(a, st);
    case 5: return run<64, 64, 32, 32, 2, 2, Ty>(a, st);
    case 6: return run<64, 32, 32, 16, 3, 2, Ty>(a, st);
    case 7: return run<32, 32, 16, 16, 4, 2, Ty>(a, st);
    default: return run<32, 32, 16, 16, 4, 4, Ty>(a, st);
    }
}

}  // namespace

hipError_t launch_w8a8_linear(const I8Args &a, hipStream_t stream)
{
    return a.type == DGW4_F32 ? pick<float>(a, stream)
           : a.type == DGW4_F16 ? pick<_Float16>(a, stream)
                                : pick<__bf16>(a, stream);
}

}  // namespace dgw4
