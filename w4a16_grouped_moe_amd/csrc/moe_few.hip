// The routed-expert layer for few tokens: at most kFewMaxAssign assignments
// (token, choice), two launches.
//
//   gate_up  H[a, :] = gelu_tanh(x[t] Wg_e^T) * (x[t] Wu_e^T), a = (t, k),
//            e = ids[a]; a workgroup takes 16 columns of H for the (at most
//            16) assignments of one tile and splits d over its eight waves.
//   down     out[t, c] = sum_k w[t, k] (H[a] Wd_e^T)[c], k ascending; a
//            workgroup takes 16 output columns for every assignment, a wave
//            one tile at a time, and keeps the experts' outputs in LDS in
//            fp32 until they are weighted and summed in k order.
//
// The layer is bound by the experts' weights, read once each, so both
// launches split the weights over the whole chip (44 column blocks per expert
// in gate_up, 176 in down at m = 704, d = 2816) where the 32-row-tile kernel
// gives a whole half expert to one workgroup: at one token, eight experts,
// that kernel keeps 16 of the 256 compute units busy.
//
// A tile is up to 16 assignments of one expert (one MFMA row block). Every
// workgroup builds the list of tiles itself from the ids (LDS counters and a
// scan; no launch, no global buffers). All workgroups agree on which
// assignments a tile holds: an expert with up to 16 has one tile, whose row
// order is of no matter (each MFMA row is a sum of its own in a fixed order of
// K); one with more takes its assignments in ascending order, 16 to a tile.
#include "gemm_common.hpp"

namespace dgw4 {
namespace {

constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / 64;

// The tile list of one workgroup: s_row[start .. start + n) of tile i are its
// assignments (low half) with their tokens (high half).
struct FewTiles {
    int count[kMaxExperts];      // assignments of each expert
    uint32_t base[kMaxExperts];  // first tile << 16 | first row of each expert
    uint32_t row[kFewMaxAssign];
    uint32_t tile[kFewMaxAssign];   // expert | start << 10 | rows << 20
    int32_t id[kFewMaxAssign];   // each assignment's expert, -1 if none
    int tiles;
};

__device__ inline int tile_expert_of(uint32_t t) { return (int)(t & 0x3FF); }
__device__ inline int tile_start_of(uint32_t t) { return (int)(t >> 10 & 0x3FF); }
__device__ inline int tile_rows_of(uint32_t t) { return (int)(t >> 20); }

// ids outside [0, E) belong to no tile.
__device__ inline void build_tiles(FewTiles &s, const int32_t *__restrict__ ids, int A, int topk, int E)
{
    const int tid = threadIdx.x;
    for (int e = tid; e < E; e += blockDim.x)
        s.count[e] = 0;
    __syncthreads();
    const int id = tid < A ? ids[tid] : -1;
    const bool live = id >= 0 && id < E;
    int rank = 0;
    if (live)
        rank = atomicAdd(&s.count[id], 1);
    if (tid < A)
        s.id[tid] = live ? id : -1;
    __syncthreads();
    if (live && s.count[id] > 16) {
        // several tiles: the rank by ascending assignment
        rank = 0;
        for (int j = 0; j < tid; ++j)
            rank += s.id[j] == id;
    }
    if (tid < 64) {
        // one wave: `per` consecutive experts per lane, then a wave scan
        const int per = (E + 63) / 64;
        uint32_t sum = 0;
        for (int j = 0; j < per; ++j) {
            const int e = tid * per + j;
            const int c = e < E ? s.count[e] : 0;
            sum += (uint32_t)((c + 15) / 16) << 16 | (uint32_t)c;
        }
        uint32_t inc = sum;
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t v = __shfl_up(inc, o);
            if (tid >= o)
                inc += v;
        }
        uint32_t at = inc - sum;
        for (int j = 0; j < per; ++j) {
            const int e = tid * per + j;
            if (e < E) {
                const int c = s.count[e];
                s.base[e] = at;
                at += (uint32_t)((c + 15) / 16) << 16 | (uint32_t)c;
            }
        }
        if (tid == 63)
            s.tiles = (int)(inc >> 16);
    }
    __syncthreads();
    if (live) {
        const uint32_t b = s.base[id];
        const int start = (int)(b & 0xFFFF);
        s.row[start + rank] = (uint32_t)tid | (uint32_t)(tid / topk) << 16;
        if (rank % 16 == 0)
            s.tile[(b >> 16) + rank / 16] = (uint32_t)id | (uint32_t)(start + rank) << 10 |
                                            (uint32_t)min(16, s.count[id] - rank) << 20;
    }
    __syncthreads();
}

template <int G, bool TL>
__global__ void __launch_bounds__(kFewThreads) few_gate_up_kernel(FewArgs a)
{
    __shared__ FewTiles s;
    __shared__ f32x4 s_red[kFewWaves][2][64];
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int r = lane & 15, p = lane >> 4;
    const int K = a.d;
    const int groups = K / G;
    const int cblocks = a.m / 16;
    build_tiles(s, a.ids, a.A, a.topk, a.E);
    const int items = s.tiles * cblocks;
    const rsrc_t xr = make_rsrc(a.x, (uint32_t)((long long)a.T * K * 2));
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t tile = s.tile[it / cblocks];
        const int cb = it % cblocks;
        const int n = tile_rows_of(tile);
        const size_t e = (size_t)tile_expert_of(tile);
        const rsrc_t wr = make_rsrc(a.gu_q + e * (size_t)a.m * K, (uint32_t)a.m * (uint32_t)K);
        const uint16_t *sp = a.gu_s + (e * 2 * a.m + cb * 16 + r) * (size_t)groups;
        const uint16_t *zp = a.gu_z + (e * 2 * a.m + cb * 16 + r) * (size_t)groups;
        const size_t up_off = (size_t)a.m * groups;
        const uint32_t wg = wq_lane_off<G, TL>(cb * 16 + r, lane, K);
        const uint32_t wu = wq_lane_off<G, TL>(a.m + cb * 16 + r, lane, K);
        const uint32_t xrow = r < n ? (s.row[tile_start_of(tile) + r] >> 16) * (uint32_t)(K * 2) +
                                          (uint32_t)(p * (G / 2))
                                    : kOutOfRange;
        f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        for (int gi = wave; gi < groups; gi += kFewWaves) {
            Frag<G> w[2];
            w[0] = load_frag<G, false>(wr, wg + wq_group_off<G, TL>(gi), 0);
            w[1] = load_frag<G, false>(wr, wu + wq_group_off<G, TL>(gi), 0);
            uint4 xv[G / 32];
#pragma unroll
            for (int t = 0; t < G / 32; ++t)
                xv[t] = load16(xr, xrow == kOutOfRange ? kOutOfRange : xrow + (uint32_t)(gi * G * 2 + t * 16), 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f16x2 c1024, c64;
                zero_point_consts(zp[h * up_off + gi], c1024, c64);
                const float sc = (float)__builtin_bit_cast(_Float16, sp[h * up_off + gi]);
                f32x4 part = {0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < G / 32; ++t)
                    part = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        __builtin_bit_cast(f16x8, permute8(xv[t])),
                        dequant8(frag_word<G>(w[h], t), c1024, c64), part, 0, 0, 0);
                acc[h] += sc * part;
            }
        }
        s_red[wave][0][lane] = acc[0];
        s_red[wave][1][lane] = acc[1];
        __syncthreads();
        if (threadIdx.x < 256) {
            const int i = threadIdx.x >> 4, c = threadIdx.x & 15;   // tile row, column
            if (i < n) {
                const int src = (i >> 2) * 16 + c;
                float g = 0.f, u = 0.f;
#pragma unroll
                for (int v = 0; v < kFewWaves; ++v) {
                    g += s_red[v][0][src][i & 3];
                    u += s_red[v][1][src][i & 3];
                }
                const uint32_t at = s.row[tile_start_of(tile) + i] & 0xFFFF;
                const _Float16 hv = (_Float16)(gelu_tanh(g) * u);
                a.h[(size_t)at * a.m + permuted_col(cb * 16 + c)] = __builtin_bit_cast(uint16_t, hv);
            }
        }
        __syncthreads();
    }
}

template <int G, bool TL>
__global__ void __launch_bounds__(kFewThreads) few_down_kernel(FewArgs a)
{
    __shared__ FewTiles s;
    extern __shared__ float s_y[];     // [A][16]
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int r = lane & 15, p = lane >> 4;
    const int K = a.m;
    const int groups = K / G;
    const int cb = blockIdx.x;
    build_tiles(s, a.ids, a.A, a.topk, a.E);
    const rsrc_t hr = make_rsrc(a.h, (uint32_t)((long long)a.A * K * 2));
    for (int it = wave; it < s.tiles; it += kFewWaves) {
        const uint32_t tile = s.tile[it];
        const int n = tile_rows_of(tile);
        const int start = tile_start_of(tile);
        const size_t e = (size_t)tile_expert_of(tile);
        const rsrc_t wr = make_rsrc(a.dn_q + e * (size_t)a.d * (K / 2), (uint32_t)a.d * (uint32_t)(K / 2));
        const uint16_t *sp = a.dn_s + (e * a.d + cb * 16 + r) * (size_t)groups;
        const uint16_t *zp = a.dn_z + (e * a.d + cb * 16 + r) * (size_t)groups;
        const uint32_t wo = wq_lane_off<G, TL>(cb * 16 + r, lane, K);
        const uint32_t hrow = r < n ? (s.row[start + r] & 0xFFFF) * (uint32_t)(K * 2) + (uint32_t)(p * (G / 2))
                                    : kOutOfRange;
        f32x4 acc = {0, 0, 0, 0};
        for (int gi = 0; gi < groups; ++gi) {
            const Frag<G> w = load_frag<G, false>(wr, wo + wq_group_off<G, TL>(gi), 0);
            uint4 hv[G / 32];
#pragma unroll
            for (int t = 0; t < G / 32; ++t)
                hv[t] = load16(hr, hrow == kOutOfRange ? kOutOfRange : hrow + (uint32_t)(gi * G * 2 + t * 16), 0);
            f16x2 c1024, c64;
            zero_point_consts(zp[gi], c1024, c64);
            const float sc = (float)__builtin_bit_cast(_Float16, sp[gi]);
            f32x4 part = {0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < G / 32; ++t)
                part = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    __builtin_bit_cast(f16x8, hv[t]), dequant8(frag_word<G>(w, t), c1024, c64), part,
                    0, 0, 0);
            acc += sc * part;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * p + i < n)
                s_y[(s.row[start + 4 * p + i] & 0xFFFF) * 16 + r] = acc[i];
    }
    __syncthreads();
    for (int o = threadIdx.x; o < a.T * 16; o += blockDim.x) {
        const int t = o >> 4, c = o & 15;
        float v = 0.f;
        for (int k = 0; k < a.topk; ++k) {
            const int id = a.ids[t * a.topk + k];
            if (id >= 0 && id < a.E)
                v = __fadd_rn(v, __fmul_rn(a.w[t * a.topk + k], s_y[(t * a.topk + k) * 16 + c]));
        }
        a.out[(size_t)t * a.d + cb * 16 + c] = __builtin_bit_cast(uint16_t, (_Float16)v);
    }
}

template <int G, bool TL>
hipError_t run_gate_up(const FewArgs &a, hipStream_t st)
{
    const int items = a.A * (a.m / 16);
    few_gate_up_kernel<G, TL><<<dim3(items < 512 ? items : 512), dim3(kFewThreads), 0, st>>>(a);
    return hipGetLastError();
}

template <int G, bool TL>
hipError_t run_down(const FewArgs &a, hipStream_t st)
{
    few_down_kernel<G, TL><<<dim3(a.d / 16), dim3(kFewThreads), (size_t)a.A * 64, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few(const FewArgs &a, int gu_g, int dn_g, hipStream_t stream)
{
    hipError_t err;
    if (gu_g == 128)
        err = a.gu_tiled ? run_gate_up<128, true>(a, stream) : run_gate_up<128, false>(a, stream);
    else
        err = a.gu_tiled ? run_gate_up<64, true>(a, stream) : run_gate_up<64, false>(a, stream);
    if (err != hipSuccess)
        return err;
    if (dn_g == 128)
        return a.dn_tiled ? run_down<128, true>(a, stream) : run_down<128, false>(a, stream);
    return a.dn_tiled ? run_down<64, true>(a, stream) : run_down<64, false>(a, stream);
}

}  // namespace dgw4
