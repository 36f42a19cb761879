// The routed-expert layer for few tokens: at most kFewMaxAssign assignments
// (token, choice).
//
//   gate_up  H[a, :] = gelu_tanh(x[t] Wg_e^T) * (x[t] Wu_e^T), a = (t, k),
//            e = ids[a]; a workgroup takes 16 columns of H for the (at most
//            16) assignments of one tile at a time and splits d over its
//            eight waves.
//   down     out[t, c] = sum_k w[t, k] (H[a] Wd_e^T)[c], k ascending. With
//            few assignments (few_keeps_outputs says no) a workgroup takes 16
//            output columns for all of them, keeps the experts' outputs in LDS
//            in fp32 and sums them itself: two launches in all. Else runs of
//            (tile, 16 columns) leave them in fp32 in the workspace and a third
//            launch sums: at 64 tokens, top-8, a workgroup with 16 columns of every
//            expert read 2.2 TB/s (64 us), runs of neighbouring columns 4.5
//            (32 us).
//
// Each product's fp32 accumulators are rounded once to fp16 where H is stored
// (16-bit activations, as everywhere in this library's layer).
//
// The layer is bound by the experts' weights, read once for each tile of up to
// 16 assignments (once each, where no expert has more), so the launches split
// them over the whole chip (44 column blocks per expert in gate_up at m = 704,
// 176 in down at d = 2816) where the 32-row-tile kernel gives a whole half
// expert to one workgroup: at one token, eight experts, that kernel keeps 16 of
// the 256 compute units busy (64 us; 16.5 here).
// Tiled weights are read non-temporally, also by an expert's second and later
// tiles: at 128 experts most have one (64 tokens 84 us, 93 without). 8 experts,
// top-2, take 17.9 us at 16 tokens and 50 at 256, four tiles or more an expert,
// where one read of their weights is 5.
// Measured at 128 experts, top-8, d = 2816, m = 704, tiled weights, back to
// back in a graph: 1 token 16.5 us (gate_up 10.6, down 6.8 alone), 4 tokens
// 34, 16 tokens 61, 64 tokens 83 (gate_up 46, down 32, the sum 4: gate_up reads
// 5.8 TB/s, a whole-chip read of contiguous memory 6.6). With one token the
// time is latency: 1 us to the list, 2.5 to the weights, the gap between the
// launches, the same again.
//
// A tile is up to 16 assignments of one expert (one MFMA row block). Every
// workgroup of the first launch builds the list of tiles itself from the ids
// (no launch before it); its first workgroup leaves the list in the workspace
// for the second launch. All workgroups agree on which assignments a tile holds: an
// expert with up to 16 has one tile, whose row order is of no matter (each
// MFMA row is a sum of its own in a fixed order of K); one with more takes its
// assignments in ascending order, 16 to a tile.
#include "gemm_common.hpp"
#include "router_keys.hpp"

#include <cmath>

namespace dgw4 {
namespace {

constexpr int kUpThreads = 512, kUpWaves = kUpThreads / 64;
constexpr int kDownThreads = 1024, kDownWaves = kDownThreads / 64;
constexpr int kSmallAssign = 64;         // assignments that one wave sorts
constexpr int kFewRouteExperts = 256;    // experts that one wave routes over in registers
// Tokens that every workgroup of gate_up routes itself, one a wave: 1.0 to 1.4
// us at 128 experts, top-8. Two a wave cost 3.9 us, what a router launch takes.
constexpr int kFewRouteTokens = kUpWaves;
constexpr uint32_t kFewPast = 0x80000000u;   // an offset past every buffer here, small additions included

// Columns of K that one lane-load of packed weights covers are a group G; a
// wave holds up to this many groups of weights and activations at once. The
// kernels' NB is the least of 1, 2, 3 and so on up to it that holds a wave's
// share of K: a group past the end costs its arithmetic all the same (26
// tokens, top-5 of 232, d = 320, m = 1152, g = 64 and 128: 61 -> 31 us; the bits
// are the same, a wave's groups keep their order).
template <int G>
constexpr int kBatch = G == 128 ? 3 : 6;
template <int G>
constexpr int kItemBatch = G == 128 ? 6 : 11;    // in few_down_items_kernel

// The tile list: tile i holds the assignments row[start .. start + n) (low half,
// their tokens in the high half).
struct FewList {
    uint32_t row[16 * kSmallAssign];
    uint32_t tile[kFewMaxAssign];        // expert | start << 10 | n << 20
    int tiles;
    int pad[3];
};
static_assert(sizeof(FewList) == kFewListBytes && sizeof(FewList) % 16 == 0, "copied in 16-byte pieces");

// What a workgroup builds its list with.
struct FewBuild {
    int32_t id[kFewMaxAssign];           // each assignment's expert, -1 if none
    int count[kMaxExperts];              // assignments of each expert
    uint32_t base[kMaxExperts];          // first tile << 16 | first row of each expert
};
static_assert(16 * kSmallAssign >= kFewMaxAssign, "the row list holds either form");

// Keeps the loads before it ahead of those after it (everything else may
// cross): loads return in order, and a wait counts the ones issued since, so
// the order in which a step's loads go out has to be the order of their use.
__device__ inline void keep_load_order() { __builtin_amdgcn_sched_barrier(0x38F); }

// A value that every lane of the wave holds, as a scalar.
__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <class P>
__device__ inline const P *uniform(const P *p)
{
    const uint64_t v = (uint64_t)p;
    return (const P *)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}

__device__ inline uint32_t tile_at(const FewList &s, int i) { return (uint32_t)uniform((int)s.tile[i]); }
__device__ inline int tile_expert_of(uint32_t t) { return (int)(t & 0x3FF); }
__device__ inline int tile_start_of(uint32_t t) { return (int)(t >> 10 & 0x3FF); }
__device__ inline int tile_rows_of(uint32_t t) { return (int)(t >> 20); }

// The list from b.id (A entries, written before the last barrier), for up to
// 64 assignments: lane a of the first wave gathers the mask of the
// assignments with its expert. 16 row slots per tile.
__device__ inline void build_tiles_small(FewList &s, const FewBuild &b, int A, int topk)
{
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        const int id = lane < A ? b.id[lane] : -1;
        uint64_t same = 0;
        for (int i = 0; i < A; ++i)
            same |= (uint64_t)(id == __builtin_amdgcn_readlane(id, i)) << i;
        const bool live = id >= 0;
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const uint64_t heads = __ballot(live && rank % 16 == 0);
        // the tile of this lane's rank: its head is the expert's assignment of
        // rank rank - rank % 16
        uint64_t m = same;
        for (int i = 0; i < rank / 16 * 16; ++i)
            m &= m - 1;
        const int head = __ffsll((unsigned long long)m) - 1;
        const int tile = live ? __popcll(heads & ((1ull << head) - 1)) : 0;
        if (live) {
            s.row[tile * 16 + rank % 16] = (uint32_t)lane | (uint32_t)(lane / topk) << 16;
            if (rank % 16 == 0)
                s.tile[tile] = (uint32_t)id | (uint32_t)(tile * 16) << 10 |
                               (uint32_t)min(16, __popcll(same) - rank) << 20;
        }
        if (lane == 0)
            s.tiles = __popcll(heads);
    }
    __syncthreads();
}

// The list for any number of assignments: LDS counters and a scan over the
// experts.
__device__ inline void build_tiles_any(FewList &s, FewBuild &b, int A, int topk, int E)
{
    const int tid = threadIdx.x;
    for (int e = tid; e < E; e += blockDim.x)
        b.count[e] = 0;
    __syncthreads();
    const int id = tid < A ? b.id[tid] : -1;
    const bool live = id >= 0;
    int rank = 0;
    if (live)
        rank = atomicAdd(&b.count[id], 1);
    __syncthreads();
    if (live && b.count[id] > 16) {
        // several tiles: the rank by ascending assignment
        rank = 0;
        for (int j = 0; j < tid; ++j)
            rank += b.id[j] == id;
    }
    if (tid < 64) {
        // one wave: `per` consecutive experts per lane, then a wave scan
        const int per = (E + 63) / 64;
        uint32_t sum = 0;
        for (int j = 0; j < per; ++j) {
            const int e = tid * per + j;
            const int c = e < E ? b.count[e] : 0;
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
                const int c = b.count[e];
                b.base[e] = at;
                at += (uint32_t)((c + 15) / 16) << 16 | (uint32_t)c;
            }
        }
        if (tid == 63)
            s.tiles = (int)(inc >> 16);
    }
    __syncthreads();
    if (live) {
        const uint32_t at = b.base[id];
        const int start = (int)(at & 0xFFFF);
        s.row[start + rank] = (uint32_t)tid | (uint32_t)(tid / topk) << 16;
        if (rank % 16 == 0)
            s.tile[(at >> 16) + rank / 16] = (uint32_t)id | (uint32_t)(start + rank) << 10 |
                                            (uint32_t)min(16, b.count[id] - rank) << 20;
    }
    __syncthreads();
}

// The list from b.id, ids outside [0, E) as -1: they belong to no tile.
__device__ inline void build_tiles(FewList &s, FewBuild &b, int A, int topk, int E)
{
    __syncthreads();
    if (A <= kSmallAssign)
        build_tiles_small(s, b, A, topk);
    else
        build_tiles_any(s, b, A, topk, E);
}

// The first launch's list for the second (building it again takes 1 to 2.2 us).
__device__ inline void publish_list(const FewList &s, void *to)
{
    for (int i = threadIdx.x; i < (int)sizeof(FewList) / 16; i += blockDim.x)
        static_cast<uint4 *>(to)[i] = reinterpret_cast<const uint4 *>(&s)[i];
}

__device__ inline void read_list(FewList &s, const void *from)
{
    for (int i = threadIdx.x; i < (int)sizeof(FewList) / 16; i += blockDim.x)
        reinterpret_cast<uint4 *>(&s)[i] = static_cast<const uint4 *>(from)[i];
    __syncthreads();
}

// The largest of a wave's values, in every lane: within rows of 16 lanes by
// DPP shifts, then across the rows by the two row broadcasts.
__device__ inline uint32_t wave_max(uint32_t v)
{
#define DGW4_DPP_MAX(ctrl) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xF, 0xF, true))
    DGW4_DPP_MAX(0x111);   // row_shr:1
    DGW4_DPP_MAX(0x112);   // row_shr:2
    DGW4_DPP_MAX(0x114);   // row_shr:4
    DGW4_DPP_MAX(0x118);   // row_shr:8
    DGW4_DPP_MAX(0x142);   // row_bcast:15
    DGW4_DPP_MAX(0x143);   // row_bcast:31
#undef DGW4_DPP_MAX
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// One token's choices by one wave: dgw4_router's ids and weights. Lane l holds
// the logits of experts l + 64 j; each round takes the largest key (the
// logit's bits in order, see router_keys.hpp), among equal ones the lowest id.
template <int PER>
__device__ inline void route_token(const float *__restrict__ l, int E, int topk, int32_t *ids_lds,
                                   int32_t *__restrict__ ids, float *__restrict__ w, bool publish)
{
    const int lane = threadIdx.x & 63;
    float v[PER];
    uint32_t key[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane + 64 * j;
        v[j] = e < E ? l[e] : 0.0f;
        key[j] = e < E ? order_key(v[j]) : 0u;
    }
    float mine = 0.0f;                   // lane k: the k-th choice's logit
    float top = 0.0f;
    int id = 0;
    for (int k = 0; k < topk; ++k) {
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            best = max(best, key[j]);
        best = wave_max(best);
        bool found = false;
        float lv = 0.0f;
        int e = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint64_t hit = __ballot(key[j] == best);
            if (!found && hit) {
                const int at = __ffsll((unsigned long long)hit) - 1;
                e = at + 64 * j;
                lv = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v[j]), at));
                if (lane == at)
                    key[j] = 0u;
                found = true;
            }
        }
        if (k == 0)
            top = lv;
        if (lane == k) {
            mine = lv;
            id = e;
        }
    }
    const float x = lane < topk ? expf(mine - top) : 0.0f;
    float den = 0.0f;
    for (int k = 0; k < topk; ++k)
        den = __fadd_rn(den, __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), k)));
    if (lane < topk) {
        ids_lds[lane] = id < E ? id : -1;
        if (publish) {
            ids[lane] = id;
            w[lane] = __fdiv_rn(x, den);
        }
    }
}

// gate_up. The (tile, 16 columns) items are dealt to the workgroups in
// contiguous runs, so a workgroup mostly stays within one tile and keeps its
// activation fragments in registers from item to item. The eight waves take
// every eighth group of d; each weight fragment's registers take the next
// step's load as soon as it has been used. The scales are staged through LDS,
// one 16-byte load per thread covers the next item's.
template <int G, bool TL, bool ROUTED, bool MULTI, int NB>
__global__ void __launch_bounds__(kUpThreads, 4) few_gate_up_kernel(FewArgs a)
{
    constexpr int W = G / 32;
    __shared__ FewList s;
    __shared__ union {
        FewBuild build;                  // until the list is done
        f32x4 red[2][kUpWaves][2][64];   // after the barrier ahead of the items
    } s_u;
    auto &s_red = s_u.red;
    static_assert(sizeof(s) + sizeof(s_u) <= kLdsStatic &&
                      2 * 8 * kFewMaxUpGroups * sizeof(uint4) <= kLdsDynamicUnasked,
                  "launched without an allowance");
    extern __shared__ uint4 s_sc[];      // [2][8 * groups]: s and z of the 16 gate, then of the 16 up rows
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int r = lane & 15, p = lane >> 4;
    const int K = a.d;
    const int groups = K / G;
    const int cblocks = a.m / 16;
    if constexpr (ROUTED) {
        for (int t = wave; t < a.T; t += kUpWaves) {
            const float *l = a.logits + (size_t)t * a.E;
            int32_t *ids = a.rids + t * a.topk;
            float *w = a.rw + t * a.topk;
            if (a.E <= 128)
                route_token<2>(l, a.E, a.topk, s_u.build.id + t * a.topk, ids, w, blockIdx.x == 0);
            else
                route_token<kFewRouteExperts / 64>(l, a.E, a.topk, s_u.build.id + t * a.topk, ids, w, blockIdx.x == 0);
        }
    } else if (tid < a.A) {
        const int id = a.ids[tid];
        s_u.build.id[tid] = id >= 0 && id < a.E ? id : -1;
    }
    build_tiles(s, s_u.build, a.A, a.topk, a.E);
    if (blockIdx.x == 0)
        publish_list(s, a.list);
    const int items = uniform(s.tiles) * cblocks;
    const int per = items / gridDim.x, rest = items % gridDim.x;
    const int first = uniform((int)blockIdx.x * per + min((int)blockIdx.x, rest));
    const int count = uniform(per + ((int)blockIdx.x < rest ? 1 : 0));
    if (count == 0)
        return;                          // the whole workgroup: no barrier below is missed
    const int batches = (groups + kUpWaves * NB - 1) / (kUpWaves * NB);
    const rsrc_t xr = make_rsrc(a.x, (uint32_t)((long long)a.T * K * 2));
    const int n_sc = 2 * groups;         // 16-byte pieces of one array's 16 rows
    const int sc_part = tid / n_sc, sc_piece = tid - sc_part * n_sc;

    // an item: tile, column block and how many are left with it
    struct Item {
        int tile, cb, left;
    };
    auto next_item = [&](Item i) {
        const bool wrap = i.cb + 1 == cblocks;
        return Item{i.left > 1 && wrap ? i.tile + 1 : i.tile, i.left > 1 ? (wrap ? 0 : i.cb + 1) : i.cb, i.left - 1};
    };
    auto load_scales = [&](const Item &i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (tid < 4 * n_sc) {
            const size_t row = (size_t)tile_expert_of(tile_at(s, i.tile)) * 2 * a.m + (sc_part >= 2 ? a.m : 0) + i.cb * 16;
            const uint16_t *src = (sc_part & 1) ? a.gu_z : a.gu_s;
            v = reinterpret_cast<const uint4 *>(src + row * groups)[sc_piece];
        }
        return v;
    };
    // one step's weight loads: its resource (empty past the last item) and lane
    // offsets, then one load per group and half
    struct Source {
        rsrc_t rsrc;
        uint32_t lane[2];
        int b;
    };
    auto source = [&](const Item &i, int b) {
        Source q;
        q.rsrc = make_rsrc(uniform(a.gu_q + (size_t)tile_expert_of(tile_at(s, i.tile)) * a.m * K),
                           i.left > 0 ? (uint32_t)a.m * (uint32_t)K : 0u);
        q.lane[0] = wq_lane_off<G, TL>(i.cb * 16 + r, lane, K);
        q.lane[1] = wq_lane_off<G, TL>(a.m + i.cb * 16 + r, lane, K);
        q.b = b;
        return q;
    };
    auto load_weight = [&](const Source &q, int h, int j) {
        const int gi = wave + kUpWaves * (q.b * NB + j);
        return load_frag<G, TL>(q.rsrc, gi < groups ? q.lane[h] + wq_group_off<G, TL>(gi) : kFewPast, 0);
    };

    // batch b of the tile's activations, then their order that of the weights;
    // rows past the tile's repeat its last one (their sums are not stored)
    uint4 xv[NB][W];
    auto load_x = [&](uint32_t tile, int b) {
        const int row = tile_start_of(tile) + min(r, tile_rows_of(tile) - 1);
        const uint32_t xrow = (s.row[row] >> 16) * (uint32_t)(K * 2) + (uint32_t)(p * (G / 2));
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int gi = wave + kUpWaves * (b * NB + j);
#pragma unroll
            for (int t = 0; t < W; ++t)
                xv[j][t] = load16(xr, (gi < groups ? xrow + (uint32_t)(gi * G * 2) : kFewPast) + (uint32_t)(t * 16), 0);
        }
    };
    auto permute_x = [&]() {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int t = 0; t < W; ++t)
                xv[j][t] = permute8(xv[j][t]);
    };

    Item cur{uniform(first / cblocks), uniform(first % cblocks), count};
    uint4 sc = load_scales(cur);
    keep_load_order();
    int have = cur.tile * batches;
    load_x(tile_at(s, cur.tile), 0);
    keep_load_order();
    Frag<G> w[2][NB];
    {
        const Source q = source(cur, 0);
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[h][j] = load_weight(q, h, j);
                keep_load_order();
            }
    }
    if (tid < 4 * n_sc)
        s_sc[tid] = sc;
    permute_x();
    __syncthreads();
    int buf = 0;
    f32x4 acc[2];
    for (int b = 0; cur.left > 0;) {
        const uint32_t tile = tile_at(s, cur.tile);
        const int n = tile_rows_of(tile), start = tile_start_of(tile);
        // at a change of tile, and at every step where a wave's share of K takes
        // several (MULTI): these loads are behind the step's weights, which the
        // wait for them drains (d = 6144, 64 experts: 25.6 us at one token, 128 at 64)
        if (have != cur.tile * batches + b) {
            have = cur.tile * batches + b;
            load_x(tile, b);
            permute_x();
        }
        const bool last = !MULTI || b == batches - 1;
        const Item nit = last ? next_item(cur) : cur;
        const int nb = last ? 0 : b + 1;
        if (!MULTI || b == 0) {
            sc = load_scales(next_item(cur));
            acc[0] = acc[1] = f32x4{0, 0, 0, 0};
        }
        keep_load_order();
        const Source q = source(nit, nb);
        const uint16_t *sl = reinterpret_cast<const uint16_t *>(s_sc + buf * 4 * n_sc) + r * groups;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int gi = min(wave + kUpWaves * (b * NB + j), groups - 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f16x2 c1024, c64;
                zero_point_consts(sl[(2 * h + 1) * 16 * groups + gi], c1024, c64);
                // past the last group: x is zero there, and the scale a finite one
                const float sv = (float)__builtin_bit_cast(_Float16, sl[2 * h * 16 * groups + gi]);
                f32x4 part = {0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < W; ++t)
                    part = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        __builtin_bit_cast(f16x8, xv[j][t]), dequant8(frag_word<G>(w[h][j], t), c1024, c64),
                        part, 0, 0, 0);
                acc[h] += sv * part;
                w[h][j] = load_weight(q, h, j);        // the next step's, into the registers just read
                keep_load_order();
            }
        }
        if (last) {
            s_red[buf][wave][0][lane] = acc[0];
            s_red[buf][wave][1][lane] = acc[1];
            if (tid < 4 * n_sc)
                s_sc[(buf ^ 1) * 4 * n_sc + tid] = sc;
            __syncthreads();
            const int i = tid >> 4, c = tid & 15;      // tile row, column
            if (i < n) {
                const int src = (i >> 2) * 16 + c;
                float g = 0.f, u = 0.f;
#pragma unroll
                for (int v = 0; v < kUpWaves; ++v) {
                    g += s_red[buf][v][0][src][i & 3];
                    u += s_red[buf][v][1][src][i & 3];
                }
                const uint32_t at = s.row[start + i] & 0xFFFF;
                const _Float16 hv = (_Float16)(gelu_tanh(g) * u);
                a.h[(size_t)at * a.m + permuted_col(cur.cb * 16 + c)] = __builtin_bit_cast(uint16_t, hv);
            }
            buf ^= 1;
        }
        cur = nit;
        b = nb;
    }
}

// down and the weighted sum, for the fewest assignments. All of H goes to LDS
// (rows 16 bytes off the bank period) while the first weights are on their way.
// A unit is one half of m's groups for one tile; a wave takes every sixteenth
// unit, in steps of NB groups, the next step's weights loaded into each
// fragment's registers as soon as it has been used. (One token's eight tiles
// are sixteen units: every load of the kernel goes out at once.) The scales of
// the tile's 16 weight rows are contiguous: one 16-byte load per lane (NS of
// them past 16 groups) into the wave's own slot of LDS. With NS = 2 the compiler
// keeps them in scratch (48 bytes a lane, here and in few_down_items_kernel) and
// each step waits for all its loads: d = m = 2048, 64 experts, 25.8 us at one
// token.
template <int G, bool TL, int NS, int NB>
__global__ void __launch_bounds__(kDownThreads) few_down_kernel(FewArgs a)
{
    constexpr int W = G / 32;
    __shared__ FewList s;
    __shared__ float s_w[kFewSumInside];
    __shared__ bool s_live[kFewSumInside];
    __shared__ float s_y[2][kFewSumInside][16];
    __shared__ uint4 s_sc[kDownWaves][64 * NS];
    static_assert(sizeof(s) + sizeof(s_w) + sizeof(s_live) + sizeof(s_y) + sizeof(s_sc) <= kLdsStatic,
                  "allow_lds_here's limit");
    extern __shared__ __attribute__((aligned(16))) char s_h[];     // [A][2 m + 16]
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int r = lane & 15, p = lane >> 4;
    const int K = a.m;
    const int stride = K * 2 + 16;
    const int groups = K / G;
    const int cb = blockIdx.x;
    if (tid < a.A) {
        const int id = a.ids[tid];
        s_w[tid] = a.w[tid];
        s_live[tid] = id >= 0 && id < a.E;
    }
    read_list(s, a.list);
    const int half_groups = (groups + 1) / 2;
    const int batches = (half_groups + NB - 1) / NB;
    const int units = uniform(s.tiles) * 2;
    const int n_sc = 2 * groups;         // 16-byte pieces of one array's 16 rows (z's follow from 32 NS)

    auto load_scales = [&](uint4 (&v)[NS], int u) {
        const size_t row = (size_t)tile_expert_of(tile_at(s, min(u, units - 1) >> 1)) * a.d + cb * 16;
        const uint16_t *sp = a.dn_s + row * groups, *zp = a.dn_z + row * groups;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int at = lane + 64 * i;
            const bool z = at >= 32 * NS;
            v[i] = reinterpret_cast<const uint4 *>(z ? zp : sp)[min(z ? at - 32 * NS : at, n_sc - 1)];
        }
    };
    // one step's weights (zero past the half's last group)
    struct Source {
        rsrc_t rsrc;
        uint32_t w;
        int left, g0;
    };
    const uint32_t wo = wq_lane_off<G, TL>(cb * 16 + r, lane, K);
    auto source = [&](int u, int b) {
        Source q;
        q.rsrc = make_rsrc(uniform(a.dn_q + (size_t)tile_expert_of(tile_at(s, min(u, units - 1) >> 1)) * a.d * (K / 2)),
                           u < units ? (uint32_t)a.d * (uint32_t)(K / 2) : 0u);
        q.g0 = (u & 1) * half_groups + b * NB;
        q.w = wo + wq_group_off<G, TL>(q.g0);
        q.left = ((u & 1) ? groups : half_groups) - q.g0;
        return q;
    };
    auto load_weight = [&](const Source &q, int j) {
        return load_frag<G, TL>(q.rsrc, j < q.left ? q.w + wq_group_off<G, TL>(j) : kFewPast, 0);
    };

    uint4 sc[NS];
    Frag<G> w[NB];
    Source cur{};
    if (units > 0) {
        load_scales(sc, wave);
        keep_load_order();
        cur = source(wave, 0);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            w[j] = load_weight(cur, j);
            keep_load_order();
        }
    }
    const int pieces = K / 8;
    for (int i = tid; i < a.A * pieces; i += kDownThreads) {
        const int row = i / pieces, c = i - row * pieces;
        // a dead assignment's row was never written: not read either
        if (s_live[row])
            *reinterpret_cast<uint4 *>(s_h + row * stride + c * 16) =
                *reinterpret_cast<const uint4 *>(a.h + (size_t)row * K + c * 8);
    }
    __syncthreads();
    f32x4 acc = {0, 0, 0, 0};
    for (int u = wave, b = 0; u < units;) {
        const bool last = b == batches - 1;
        const int nu = last ? u + kDownWaves : u, nb = last ? 0 : b + 1;
        const Source q = source(nu, nb);
        const uint32_t tile = tile_at(s, u >> 1);
        const int n = tile_rows_of(tile), start = tile_start_of(tile);
        // rows past the tile's repeat its last one (their sums are not stored)
        const char *hp = s_h + (s.row[start + min(r, n - 1)] & 0xFFFF) * stride + p * (G / 2);
        if (b == 0) {
            // the wave's own LDS slot: its earlier reads are done, in order
#pragma unroll
            for (int i = 0; i < NS; ++i)
                s_sc[wave][lane + 64 * i] = sc[i];
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            acc = f32x4{0, 0, 0, 0};
        }
        load_scales(sc, nu);
        keep_load_order();
        const uint16_t *sl = reinterpret_cast<const uint16_t *>(s_sc[wave]) + r * groups;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            // past the half's last group: left out
            const int gi = min(cur.g0 + j, groups - 1);
            const bool in = j < cur.left;
            f16x2 c1024, c64;
            zero_point_consts(sl[32 * NS * 8 + gi], c1024, c64);
            const float sv = (float)__builtin_bit_cast(_Float16, sl[gi]);
            f32x4 part = {0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < W; ++t)
                part = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    *reinterpret_cast<const f16x8 *>(hp + gi * (G * 2) + t * 16),
                    dequant8(frag_word<G>(w[j], t), c1024, c64), part, 0, 0, 0);
            w[j] = load_weight(q, j);
            keep_load_order();
            if (in)
                acc += sv * part;
        }
        if (last) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * p + i < n)
                    s_y[u & 1][s.row[start + 4 * p + i] & 0xFFFF][r] = acc[i];
            __builtin_amdgcn_wave_barrier();
        }
        u = nu;
        b = nb;
        cur = q;
    }
    __syncthreads();
    // T * topk <= 64: one thread per output
    if (tid < a.T * 16) {
        const int t = tid >> 4, c = tid & 15;
        float v = 0.f;
        for (int k = 0; k < a.topk; ++k) {
            const int at = t * a.topk + k;
            if (s_live[at])
                v = __fadd_rn(v, __fmul_rn(s_w[at], __fadd_rn(s_y[0][at][c], s_y[1][at][c])));
        }
        a.out[(size_t)t * a.d + cb * 16 + c] = __builtin_bit_cast(uint16_t, (_Float16)v);
    }
}

// down for more assignments: Y[a, :] = H[a] Wd_e^T in fp32, to be weighted and
// summed by few_combine_kernel. The (tile, 16 columns) items are dealt to the
// workgroups in contiguous runs. A workgroup takes its run tile by tile: the
// tile's activations go to LDS (rows 16 bytes off the bank period), then its
// waves take the tile's column blocks in turn, each streaming all of m past
// them with the next step's weights loaded as soon as a fragment is used.
template <int G, bool TL, int NS, bool MULTI, int NB>
__global__ void __launch_bounds__(kUpThreads, 4) few_down_items_kernel(FewArgs a)
{
    constexpr int W = G / 32;
    __shared__ FewList s;
    __shared__ uint4 s_sc[kUpWaves][64 * NS];
    static_assert(sizeof(s) + sizeof(s_sc) <= kLdsStatic, "allow_lds_here's limit");
    extern __shared__ __attribute__((aligned(16))) char s_h[];     // [16][2 m + 16]
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int r = lane & 15, p = lane >> 4;
    const int K = a.m;
    const int stride = K * 2 + 16;
    const int groups = K / G;
    const int cblocks = a.d / 16;
    read_list(s, a.list);
    const int items = uniform(s.tiles) * cblocks;
    const int per = items / gridDim.x, rest = items % gridDim.x;
    int at = uniform((int)blockIdx.x * per + min((int)blockIdx.x, rest));
    const int end = uniform(at + per + ((int)blockIdx.x < rest ? 1 : 0));
    const int batches = (groups + NB - 1) / NB;
    const int n_sc = 2 * groups;         // 16-byte pieces of one array's 16 rows (z's follow from 32 NS)
    const char *hp = s_h + r * stride + p * (G / 2);
    const uint16_t *sl = reinterpret_cast<const uint16_t *>(s_sc[wave]) + r * groups;

    for (int ti = at / cblocks; at < end; ++ti) {
        const int c0 = uniform(at - ti * cblocks), c1 = uniform(min(cblocks, end - ti * cblocks));
        at = ti * cblocks + c1;
        const uint32_t tile = tile_at(s, ti);
        const int n = tile_rows_of(tile), start = tile_start_of(tile);
        const size_t e = (size_t)tile_expert_of(tile);
        const uint8_t *wq = uniform(a.dn_q + e * a.d * (K / 2));
        const uint16_t *sp = a.dn_s + e * a.d * groups, *zp = a.dn_z + e * a.d * groups;

        // one step (a column block, NB groups): nothing is read past the last block
        auto load_weight = [&](int c, int b, int j) {
            const rsrc_t rs = make_rsrc(wq, c < c1 ? (uint32_t)a.d * (uint32_t)(K / 2) : 0u);
            const uint32_t off = wq_lane_off<G, TL>(c * 16 + r, lane, K) + (uint32_t)b * wq_group_off<G, TL>(NB);
            return load_frag<G, TL>(rs, b * NB + j < groups ? off + wq_group_off<G, TL>(j) : kFewPast, 0);
        };
        auto load_scales = [&](uint4 (&v)[NS], int c) {
            const size_t row = (size_t)min(c, c1 - 1) * 16 * groups;
#pragma unroll
            for (int q = 0; q < NS; ++q) {
                const int i = lane + 64 * q;
                const bool z = i >= 32 * NS;
                v[q] = reinterpret_cast<const uint4 *>((z ? zp : sp) + row)[min(z ? i - 32 * NS : i, n_sc - 1)];
            }
        };
        uint4 sc[NS];
        Frag<G> w[NB];
        load_scales(sc, c0 + wave);
        keep_load_order();
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            w[j] = load_weight(c0 + wave, 0, j);
            keep_load_order();
        }
        // the tile's rows; those past n keep what they hold (their sums are not stored)
        const int pieces = K / 8;
        for (int i = tid; i < n * pieces; i += kUpThreads) {
            const int row = i / pieces, c = i - row * pieces;
            const uint32_t src = s.row[start + row] & 0xFFFF;
            *reinterpret_cast<uint4 *>(s_h + row * stride + c * 16) =
                *reinterpret_cast<const uint4 *>(a.h + (size_t)src * K + c * 8);
        }
        __syncthreads();
        f32x4 acc = {0, 0, 0, 0};
        for (int c = c0 + wave, b = 0; c < c1;) {
            const bool last = !MULTI || b == batches - 1;
            const int nc = last ? c + kUpWaves : c, nb = last ? 0 : b + 1;
            if (!MULTI || b == 0) {
                // the wave's own LDS slot: its earlier reads are done, in order
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    s_sc[wave][lane + 64 * i] = sc[i];
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                acc = f32x4{0, 0, 0, 0};
            }
            load_scales(sc, nc);
            keep_load_order();
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                // past the last group the scale is 0 and the rest in range
                const int gi = MULTI ? min(b * NB + j, groups - 1) : min(j, groups - 1);
                const bool in = MULTI ? b * NB + j < groups : j < groups;
                f16x2 c1024, c64;
                zero_point_consts(sl[32 * NS * 8 + gi], c1024, c64);
                const float sv = in ? (float)__builtin_bit_cast(_Float16, sl[gi]) : 0.0f;
                f32x4 part = {0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < W; ++t)
                    part = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        *reinterpret_cast<const f16x8 *>(hp + gi * (G * 2) + t * 16),
                        dequant8(frag_word<G>(w[j], t), c1024, c64), part, 0, 0, 0);
                w[j] = load_weight(nc, nb, j);    // the next step's, into the registers just read
                keep_load_order();
                if (in)
                    acc += sv * part;
            }
            if (last) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (4 * p + i < n)
                        a.y[(size_t)(s.row[start + 4 * p + i] & 0xFFFF) * a.d + c * 16 + r] = acc[i];
                __builtin_amdgcn_wave_barrier();
            }
            c = nc;
            b = nb;
        }
        __syncthreads();                 // the next tile's rows replace these
    }
}

// out[t, c] = sum_k w[t, k] Y[t topk + k, c], k ascending, four columns a thread.
__global__ void __launch_bounds__(256) few_combine_kernel(FewArgs a)
{
    const int t = blockIdx.y, c = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 4;
    if (c >= a.d)
        return;
    const float *y = a.y + (size_t)t * a.topk * a.d + c;
    f32x4 v = {0, 0, 0, 0};
    for (int k0 = 0; k0 < a.topk; k0 += 8) {
        // eight choices' loads before the first addition; a dead one's slot is
        // read with the others and left out of the sum
        f32x4 yk[8];
        float wk[8];
        bool live[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int at = min(k0 + k, a.topk - 1);
            const int id = a.ids[t * a.topk + at];
            live[k] = k0 + k < a.topk && id >= 0 && id < a.E;
            wk[k] = a.w[t * a.topk + at];
            yk[k] = *reinterpret_cast<const f32x4 *>(y + (size_t)at * a.d);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (live[k])
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = __fadd_rn(v[i], __fmul_rn(wk[k], yk[k][i]));
    }
    *reinterpret_cast<uint2 *>(a.out + (size_t)t * a.d + c) = pack_f16x4(v);
}

template <int G, bool TL, bool MULTI, int NB>
hipError_t run_gate_up(const FewArgs &a, hipStream_t st)
{
    const int items = a.A * (a.m / 16);
    const size_t lds = 2 * 8 * (size_t)(a.d / G) * 16;
    const dim3 grid(items < 512 ? items : 512), block(kUpThreads);
    if (a.logits != nullptr)
        few_gate_up_kernel<G, TL, true, MULTI, NB><<<grid, block, lds, st>>>(a);
    else
        few_gate_up_kernel<G, TL, false, MULTI, NB><<<grid, block, lds, st>>>(a);
    return hipGetLastError();
}

template <int G, bool TL>
hipError_t pick_gate_up(const FewArgs &a, hipStream_t st)
{
    const int share = (a.d / G + kUpWaves - 1) / kUpWaves;     // groups of a wave
    if (share > kBatch<G>)
        return run_gate_up<G, TL, true, kBatch<G>>(a, st);
    if (share == 1)
        return run_gate_up<G, TL, false, 1>(a, st);
    if (share == 2)
        return run_gate_up<G, TL, false, 2>(a, st);
    return share == 3 ? run_gate_up<G, TL, false, 3>(a, st) : run_gate_up<G, TL, false, kBatch<G>>(a, st);
}

template <int G, bool TL, int NS, int NB>
hipError_t run_down(const FewArgs &a, hipStream_t st)
{
    static LdsAllowed allowed;
    const size_t lds = (size_t)a.A * (2 * (size_t)a.m + 16);
    const hipError_t err = allow_lds_here(few_down_kernel<G, TL, NS, NB>, lds, allowed);
    if (err != hipSuccess)
        return err;
    few_down_kernel<G, TL, NS, NB><<<dim3(a.d / 16), dim3(kDownThreads), lds, st>>>(a);
    return hipGetLastError();
}

template <int G, bool TL, int NS, bool MULTI, int NB>
hipError_t run_down_items(const FewArgs &a, hipStream_t st)
{
    static LdsAllowed allowed;
    const size_t lds = 16 * (2 * (size_t)a.m + 16);
    hipError_t err = allow_lds_here(few_down_items_kernel<G, TL, NS, MULTI, NB>, lds, allowed);
    if (err != hipSuccess)
        return err;
    const int items = a.A * (a.d / 16);
    const int groups = (items + kUpWaves - 1) / kUpWaves;
    few_down_items_kernel<G, TL, NS, MULTI, NB><<<dim3(groups < 512 ? groups : 512), dim3(kUpThreads), lds, st>>>(a);
    err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    few_combine_kernel<<<dim3((a.d / 4 + 255) / 256, a.T), dim3(256), 0, st>>>(a);
    return hipGetLastError();
}

template <int G, bool TL>
hipError_t pick_down(const FewArgs &a, hipStream_t st)
{
    const int groups = a.m / G;
    if (a.y != nullptr) {
        constexpr int most = kItemBatch<G>;
        if (groups > most)
            return groups <= 16 ? run_down_items<G, TL, 1, true, most>(a, st)
                                : run_down_items<G, TL, 2, true, most>(a, st);
        if (groups <= 2)
            return run_down_items<G, TL, 1, false, 2>(a, st);
        if (groups <= 4)
            return run_down_items<G, TL, 1, false, 4>(a, st);
        return groups <= 6 ? run_down_items<G, TL, 1, false, 6>(a, st) : run_down_items<G, TL, 1, false, most>(a, st);
    }
    const int share = (groups + 1) / 2;
    if (groups > 16)
        return run_down<G, TL, 2, kBatch<G>>(a, st);
    if (share == 1)
        return run_down<G, TL, 1, 1>(a, st);
    if (share == 2)
        return run_down<G, TL, 1, 2>(a, st);
    return share == 3 ? run_down<G, TL, 1, 3>(a, st) : run_down<G, TL, 1, kBatch<G>>(a, st);
}

}  // namespace

bool few_routes_inside(int T, int E)
{
    return T <= kFewRouteTokens && E <= kFewRouteExperts;
}

// Whether down leaves the experts' outputs in the workspace, to be summed by a
// launch of their own. It does not (and sums inside, a workgroup per 16 columns
// of the output holding all of H in LDS) where H fits and either the columns
// alone fill the chip or the work of a workgroup is small. Measured, us a layer, inside / apart: d 2816, m
// 704, 48 assignments 35.6 / 36.8; d 512, m 704, 16 assignments 15.6 / 16.7, 48
// assignments 26.2 / 20.4; d 1536, m 1408, 16 assignments 30.4 / 24.7.
bool few_keeps_outputs(int A, int d, int m)
{
    if (A > kFewSumInside || (long long)A * (2LL * m + 16) > 96 * 1024)
        return true;
    return d < 2304 && (long long)A * m > 11264 + 4LL * d;
}

hipError_t launch_few(const FewArgs &a, int gu_g, int dn_g, hipStream_t stream)
{
    hipError_t err;
    if (gu_g == 128)
        err = a.gu_tiled ? pick_gate_up<128, true>(a, stream) : pick_gate_up<128, false>(a, stream);
    else
        err = a.gu_tiled ? pick_gate_up<64, true>(a, stream) : pick_gate_up<64, false>(a, stream);
    if (err != hipSuccess)
        return err;
    if (dn_g == 128)
        return a.dn_tiled ? pick_down<128, true>(a, stream) : pick_down<128, false>(a, stream);
    return a.dn_tiled ? pick_down<64, true>(a, stream) : pick_down<64, false>(a, stream);
}

}  // namespace dgw4
