// A batch of requests' rules on its logits (penalties for the tokens that a
// sequence holds, biases, a scale, masks): on their own, and inside the
// sampler's pass.
//
// A workgroup takes one tile of columns of one row, or of neighbouring rows in
// turn. It keeps a word per column in LDS, into which the sequence's biases (the
// last place of a column wins: a maximum) and its tokens (a count: integer
// additions) go, whatever their order: no workspace, no sorting, and the rows
// that share a sequence share the words. Each logit is read once.
//
// The rules' arithmetic costs a lane about thirty instructions, and few columns
// have a word: the wave's lanes take those columns in turns of 64, whoever holds
// them, and the logits go through LDS there and back. (Each lane with its own
// columns, one at a time, waits for the lane that has most: a canvas of 256 rows
// and 4 sequences 84 us against 76, 64 histories of 60000 tokens 70 against 65; in
// place with nothing else changed it was the better by 20 us to 21, with 1000
// tokens a row by 28.6 to 29.4.)
//
// A wave's part of a row (the maximum, its first place, sums of exp relative to
// it, the best score) goes to the workspace; a second kernel joins a row's parts.
// Every order is fixed, so results are bitwise reproducible.
//
// Bounds (all figures of this file: replays of a graph over logits that change from
// call to call, medians, 262144 columns of fp32 where nothing else is said): adjusting is
// a copy, 256 rows 101 us (5.3 TB/s; fp16 to itself 57, 4.7 TB/s). In place with
// nothing changed but a few columns it is not: 64 rows of 1000 tokens 21 us, of
// which a few columns' lines would be one; each of 4096 workgroups clears its words
// and reads the row's tokens. The sampler without rules reads 256 rows in 48 us (44
// at best, 6.1 TB/s); history costs half or more on top, in the steps that make the
// words (64 rows of own sequences of 1000 tokens, greedy: 16 -> 29 us) and in the
// columns with words and the registers they take (256 rows of 4 sequences of 8000
// tokens: 48 -> 65 us, 76 with masks): with history and 16 columns a thread the
// sampler keeps 62 of its scalars, the rules' pointers among them, in lanes of
// vector registers, adjusting 30 to 34.
#include "element_types.hpp"
#include "logit_cut.hpp"
#include "logit_rules.hpp"
#include "sampler_common.hpp"

#include <climits>
#include <type_traits>

namespace dgw4 {
namespace {

constexpr int kJoin = 256;           // threads that join a row's parts

// v of all lanes joined: the lanes of a row of 16 by DPP, then the four rows.
template <class T, class F>
__device__ inline T across(T v, F f)
{
    auto step = [&](auto ctrl) {
        const int o = __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF, 0xF, true);
        v = f(v, __builtin_bit_cast(T, o));
    };
    step(std::integral_constant<int, 0xB1>{});       // quad_perm: the neighbour
    step(std::integral_constant<int, 0x4E>{});       // quad_perm: the other pair
    step(std::integral_constant<int, 0x141>{});      // row_half_mirror
    step(std::integral_constant<int, 0x140>{});      // row_mirror
    auto row = [&](int lane) {
        return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
    };
    return f(f(row(0), row(16)), f(row(32), row(48)));
}

__device__ inline float across_max(float v)
{
    return across(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ inline float across_sum(float v)
{
    return across(v, [](float a, float b) { return a + b; });
}
__device__ inline int across_min(int v)
{
    return across(v, [](int a, int b) { return min(a, b); });
}

// The words of columns c0 .. of sequence seq, by the whole workgroup. The first
// tokens are on their way while the words are cleared.
template <int kThreads, int TILE>
__device__ inline void enter(const dgw4_logit_rules &u, int seq, int c0, uint32_t *words)
{
    constexpr int kAhead = 4, kStep = kThreads * 4;  // loads of four tokens a thread has on their way
    const int32_t *tok = u.tokens + (long long)max(seq, 0) * u.ld_tokens;
    int n = 0, p = 0;
    if (u.tokens && seq >= 0) {
        n = min(max(u.lengths[seq], 0), u.max_tokens);
        p = u.prompt_lengths ? u.prompt_lengths[seq] : 0;
    }
    int4 t[kAhead];
    auto load = [&](int i0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            t[j] = make_int4(-1, -1, -1, -1);
            if (i0 + j * kStep + 3 < n)
                __builtin_memcpy(&t[j], tok + i0 + j * kStep, 16);
        }
    };
    const int i0 = (int)threadIdx.x * 4;
    load(i0);
    // the last tokens, fewer than four
    const int rest = (n & ~3) + (int)threadIdx.x;
    const int last = rest < n ? tok[rest] : -1;
    __syncthreads();
    for (int i = threadIdx.x * 4; i < TILE; i += kStep)
        *reinterpret_cast<uint4 *>(words + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (u.n_bias > 0 && seq >= 0) {
        const int32_t *ids = u.bias_ids + (long long)seq * u.ld_bias;
        for (int j = threadIdx.x; j < u.n_bias; j += kThreads) {
            const uint32_t c = (uint32_t)ids[j] - (uint32_t)c0;
            if (c < (uint32_t)TILE)
                atomicMax(&words[c], (uint32_t)(j + 1) << kPlaceBit);
        }
        __syncthreads();
    }
    // a token outside the tile, or none (-1), has no word
    auto prompt = [&](int token) {
        const uint32_t c = (uint32_t)token - (uint32_t)c0;
        if (c < (uint32_t)TILE)
            atomicOr(&words[c], kPrompt);
    };
    auto generated = [&](int token) {
        const uint32_t c = (uint32_t)token - (uint32_t)c0;
        if (c < (uint32_t)TILE)
            atomicAdd(&words[c], 1u);
    };
    auto either = [&](int token, int i) { i < p ? prompt(token) : generated(token); };
    const int wave0 = __builtin_amdgcn_readfirstlane(i0);
    for (int step = 0; wave0 + step < n; step += kAhead * kStep) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (wave0 + step + j * kStep >= n)
                break;
            const int i = i0 + step + j * kStep;
            if (i >= p) {
                generated(t[j].x);
                generated(t[j].y);
                generated(t[j].z);
                generated(t[j].w);
            } else if (i + 3 < p) {
                prompt(t[j].x);
                prompt(t[j].y);
                prompt(t[j].z);
                prompt(t[j].w);
            } else {
                either(t[j].x, i);
                either(t[j].y, i + 1);
                either(t[j].z, i + 2);
                either(t[j].w, i + 3);
            }
        }
        load(i0 + step + kAhead * kStep);
    }
    either(last, rest);
    __syncthreads();
}

// W neighbouring logits at any alignment of their element, read or written once.
template <class T>
struct Wide {
    static constexpr int W = 16 / sizeof(T);
    typedef T vec __attribute__((ext_vector_type(W), aligned(sizeof(T))));
};

template <class T>
__device__ inline typename Wide<T>::vec read_wide(const T *row, int c, int V)
{
    constexpr int W = Wide<T>::W;
    typedef typename Wide<T>::vec vec;
    if (c + W <= V)
        return __builtin_nontemporal_load(reinterpret_cast<const vec *>(row + c));
    vec v;
#pragma unroll
    for (int i = 0; i < W; ++i)
        v[i] = c + i < V ? row[c + i] : (T)0.0f;
    return v;
}

// A thread's N vectors, `step` columns apart from c on; inside: the tile ends before V does.
template <class T, int N>
__device__ inline void read_all(typename Wide<T>::vec (&x)[N], const T *row, int c, int step, int V, bool inside)
{
    typedef typename Wide<T>::vec vec;
    if (inside) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            x[k] = __builtin_nontemporal_load(reinterpret_cast<const vec *>(row + c + k * step));
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
            x[k] = read_wide(row, c + k * step, V);
    }
}

// The mask's bits of columns c .. c + W - 1 (c a multiple of W) in the low bits; past V: anything.
template <int W>
__device__ inline uint32_t allowed(const uint32_t *mask, int c, int V)
{
    return mask && c < V ? mask[c >> 5] >> (c & 31) : ~0u;
}

// l where bit i of bits is set, else -inf.
__device__ inline float kept(float l, uint32_t bits, int i)
{
    const uint32_t all = (uint32_t)((int32_t)(bits << (31 - i)) >> 31);
    return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, l) & all) | (0xFF800000u & ~all));
}

// The largest of three. (fmaxf would have the compiler quiet each logit first.)
__device__ inline float max3(float a, float b, float c)
{
    float v;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(v) : "v"(a), "v"(b), "v"(c));
    return v;
}

// Which of a thread's columns have a word: bit k * W + i for column i of vector k,
// whose words lie from words + k * step on.
template <int W, int N>
__device__ inline uint32_t with_words(const uint32_t *words, int step)
{
    uint32_t need = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i)
            need |= min(words[k * step + i], 1u) << (k * W + i);
    return need;
}

// A wave's columns with words, dealt out over its lanes: lane i has the i-th of each
// 64, its place in the tile's words and its word. Two turns: one sends the waves of
// long histories the other way (64 of 60000 tokens: 72 us against 66), three or four
// take registers from all (canvas of 256 rows in fp16: 103 and 107 us against 97).
constexpr int kDealt = 2;

struct Dealt {
    int count;                                   // more than kDealt * 64: not dealt out
    uint32_t at[kDealt], word[kDealt];
};

// What the wave's lanes have written to LDS, before any of them reads it.
__device__ inline void within_wave()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// need: this thread's columns with a word, as with_words() has them, the first at
// words[own]; list: kDealt * 64 places of the wave's own.
template <int W, int N>
__device__ inline void deal(Dealt &d, uint32_t need, const uint32_t *words, int own, int step, uint16_t *list)
{
    const int lane = threadIdx.x & 63, n = __builtin_popcount(need);
    int place = 0;
    d.count = 0;
#pragma unroll
    for (int b = 0; 1 << b <= N * W; ++b) {
        const uint64_t some = __ballot(n >> b & 1);
        place += (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(some >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)some, 0))
                 << b;
        d.count += __builtin_popcountll(some) << b;
    }
    if (d.count > kDealt * 64)
        return;
    for (; need; need &= need - 1) {
        const int at = __builtin_ctz(need);
        list[place++] = (uint16_t)(own + at / W * step + at % W);
    }
    within_wave();
#pragma unroll
    for (int j = 0; j < kDealt; ++j)
        if (j * 64 + lane < d.count) {
            d.at[j] = list[j * 64 + lane];
            d.word[j] = words[d.at[j]];
        }
    within_wave();
}

// A thread's N vectors of W logits after their sequence's rules. The wave's logits
// change places with its words, which d holds, and each lane takes the columns
// dealt to it; where too many have a word, every lane takes all of its own.
template <int W, int N>
__device__ inline void follow_rules(float (&l)[N * W], const Dealt &d, uint32_t *words, int own, int step,
                                    const Sequence &q)
{
    const int lane = threadIdx.x & 63;
    if (d.count > kDealt * 64) {
#pragma unroll
        for (int e = 0; e < N * W; ++e) {
            const uint32_t word = words[own + e / W * step + e % W];
            if (word)
                l[e] = adjusted(l[e], word, q);
        }
    } else if (d.count > 0) {
#pragma unroll
        for (int e = 0; e < N * W; e += 4)
            *reinterpret_cast<uint4 *>(words + own + e / W * step + e % W) =
                make_uint4(__builtin_bit_cast(uint32_t, l[e]), __builtin_bit_cast(uint32_t, l[e + 1]),
                           __builtin_bit_cast(uint32_t, l[e + 2]), __builtin_bit_cast(uint32_t, l[e + 3]));
        within_wave();
#pragma unroll
        for (int j = 0; j < kDealt; ++j)
            if (j * 64 + lane < d.count) {
                const float v = __builtin_bit_cast(float, words[d.at[j]]);
                words[d.at[j]] = __builtin_bit_cast(uint32_t, adjusted(v, d.word[j], q));
            }
        within_wave();
#pragma unroll
        for (int e = 0; e < N * W; e += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(words + own + e / W * step + e % W);
            l[e] = __builtin_bit_cast(float, v.x);
            l[e + 1] = __builtin_bit_cast(float, v.y);
            l[e + 2] = __builtin_bit_cast(float, v.z);
            l[e + 3] = __builtin_bit_cast(float, v.w);
        }
        within_wave();
    }
#pragma unroll
    for (int e = 0; e < N * W; ++e)
        l[e] = rounded_product(l[e], q.scale);
}

// E columns a thread; SPARSE: in place and no scale, so only what changes is read and
// written. Five waves a SIMD for 16-bit logits hide the words' making (48 rows of
// 100003 bf16 with every rule 15.3 -> 12.0 us), though a canvas of shared words goes
// better with four (256 rows of fp16 to fp32 90 us against 96, to fp16 56 against
// 58): out of place with history and 16 columns, fp16 spills two vector registers
// under five, 12 bytes of scratch a lane.
template <class Tx, class Ty, int kThreads, int E, bool HIST, bool SPARSE>
__global__ void __launch_bounds__(kThreads, sizeof(Tx) == 2 ? 5 : 4) adjust_kernel(LogitArgs a, int tiles, int rows)
{
    constexpr int W = Wide<Tx>::W, N = E / W;        // columns of a vector, vectors of a thread
    constexpr int kTile = tile_of(kThreads, E);
    __shared__ __attribute__((aligned(16))) uint32_t words[HIST ? kTile : 4];
    const int tile = (int)(blockIdx.x % (uint32_t)tiles), r0 = (int)(blockIdx.x / (uint32_t)tiles) * rows;
    const int c0 = tile * kTile;
    __shared__ uint16_t list[HIST ? kThreads / 64 : 1][kDealt * 64];
    const int own = HIST ? (int)threadIdx.x * W : 0, wave = (int)threadIdx.x >> 6;   // own: the first vector's words
    constexpr uint32_t kAll = (1u << W) - 1;
    const int mine = c0 + (int)threadIdx.x * W, end = r0 + min(rows, a.R - r0);
    const bool inside = c0 + kTile <= a.V;
    const Tx *row = (const Tx *)a.logits + (long long)r0 * a.ld;
    Ty *out = (Ty *)a.out + (long long)r0 * a.ld_out;
    typename Wide<Tx>::vec x[N];
    if (!SPARSE)
        read_all<Tx, N>(x, row, mine, kThreads * W, a.V, inside);
    int seq = -2;
    uint32_t needs = 0;
    Dealt d;
    d.count = 0;
    for (int r = r0; r < end; ++r, row += a.ld, out += a.ld_out) {
        const int s = sequence_of(a.rules, r);
        const uint32_t *mask = mask_of(a.rules, r);
        uint32_t bits[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
            bits[k] = allowed<W>(mask, mine + k * kThreads * W, a.V);
        if (HIST && s != seq) {
            enter<kThreads, kTile>(a.rules, s, c0, words);
            needs = with_words<W, N>(words + own, kThreads * W);
            deal<W, N>(d, needs, words, own, kThreads * W, list[wave]);
        }
        seq = s;
        const Sequence q = sequence(a.rules, s);
        if (SPARSE) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int c = mine + k * kThreads * W;
                if (c < a.V && ((needs >> (k * W) & kAll) || (bits[k] & kAll) != kAll))
                    x[k] = read_wide(row, c, a.V);
            }
        }
        float l[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            l[e] = to_f32(x[e / W][e % W]);
        // the next row's, behind this one's arithmetic
        if (!SPARSE && r + 1 < end)
            read_all<Tx, N>(x, row + a.ld, mine, kThreads * W, a.V, inside);
        follow_rules<W, N>(l, d, words, own, kThreads * W, q);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int c = c0 + (k * kThreads + (int)threadIdx.x) * W;
            if (c >= a.V || (SPARSE && !(needs >> (k * W) & kAll) && (bits[k] & kAll) == kAll))
                continue;
            typedef Ty vec __attribute__((ext_vector_type(W), aligned(sizeof(Ty))));
            vec y;
#pragma unroll
            for (int i = 0; i < W; ++i)
                y[i] = from_f32<Ty>(kept(l[k * W + i], bits[k], i));
            if (c + W <= a.V) {
                if constexpr (SPARSE)
                    *reinterpret_cast<vec *>(out + c) = y;
                else
                    __builtin_nontemporal_store(y, reinterpret_cast<vec *>(out + c));
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (c + i < a.V)
                        out[c + i] = y[i];
            }
        }
    }
}

// exp(d), d <= 0. Below -200 fp32 holds nothing of it; taken there so that d times
// it is zero also where d is infinite.
__device__ inline float bounded(float d) { return fmaxf(d, -200.0f); }

template <class Tx, int kThreads, int E, bool HIST>
__global__ void __launch_bounds__(kThreads, !HIST ? 6 : sizeof(Tx) == 2 ? 5 : 4)
    sample_adjusted_kernel(LogitArgs a, int tiles, int rows)
{
    constexpr int W = Wide<Tx>::W, N = E / W, kTile = tile_of(kThreads, E), kWaves = kThreads / 64;
    __shared__ __attribute__((aligned(16))) uint32_t words[HIST ? kTile : 4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int tile = (int)(blockIdx.x % (uint32_t)tiles), r0 = (int)(blockIdx.x / (uint32_t)tiles) * rows;
    const int c0 = tile * kTile, first = wave * part_of(E);       // the tile's and, in it, the wave's columns
    __shared__ uint16_t list[HIST ? kWaves : 1][kDealt * 64];
    const int own = HIST ? first + lane * W : 0;                  // where this lane's first vector's words are
    const int mine = c0 + first + lane * W, end = r0 + min(rows, a.R - r0);
    const bool inside = c0 + kTile <= a.V;
    const Tx *row = (const Tx *)a.logits + (long long)r0 * a.ld;
    typename Wide<Tx>::vec x[N];
    read_all<Tx, N>(x, row, mine, 64 * W, a.V, inside);
    int seq = -2;
    Dealt d;
    d.count = 0;
    for (int r = r0; r < end; ++r, row += a.ld) {
        const int s = sequence_of(a.rules, r);
        const uint32_t *mask = mask_of(a.rules, r);
        uint32_t bits[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int c = mine + k * 64 * W;
            bits[k] = allowed<W>(mask, c, a.V);
            if (!inside && c + W > a.V)
                bits[k] &= c < a.V ? (1u << (a.V - c)) - 1 : 0u;
        }
        if (HIST && s != seq) {
            enter<kThreads, kTile>(a.rules, s, c0, words);
            deal<W, N>(d, with_words<W, N>(words + own, 64 * W), words, own, 64 * W, list[wave]);
        }
        seq = s;
        const Sequence q = sequence(a.rules, s);
        float l[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            l[e] = to_f32(x[e / W][e % W]);
        // the next row's, behind this one's arithmetic
        if (r + 1 < end)
            read_all<Tx, N>(x, row + a.ld, mine, 64 * W, a.V, inside);
        follow_rules<W, N>(l, d, words, own, 64 * W, q);
        if (mask || !inside) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                l[e] = kept(l[e], bits[e / W], e % W);
        }
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < E; e += 2)
            top = max3(top, l[e], l[e + 1]);
        Partial p;
        p.m = across_max(top);
        const float m = p.m > -INFINITY ? p.m : 0.0f;
        p.z = p.m > -INFINITY ? 1.0f : 0.0f;
        p.s = 0.0f;
        if (a.entropy) {
            float z = 0.0f, sum = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float d = bounded(l[e] - m), ex = __expf(d);
                z += ex;
                sum += ex * d;
            }
            p.z = across_sum(z);
            p.s = across_sum(sum);
        }
        // the first column that holds the maximum
        int at = INT_MAX;
        if (top == p.m) {
#pragma unroll
            for (int e = E - 1; e >= 0; --e)
                at = l[e] == p.m ? (e / W * 64 + lane) * W + e % W : at;
        }
        p.av = p.m;
        p.ai = across_min(at) + c0 + first;
        p.sv = -INFINITY;
        p.si = INT_MAX;
        if (a.sample) {
            float best = -INFINITY;
            int where = INT_MAX;
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const int c = c0 + first + (e / W * 64 + lane) * W + e % W;
                // (not known ahead of the rows: its first products would wait for
                // them in registers)
                uint32_t w[4], block = (uint32_t)c >> 2;
                asm volatile("" : "+v"(block));
                philox4x32_10(block, (uint32_t)r, 0u, 0u, a.k0, a.k1, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float v = l[e + j] + gumbel(w[j]);
                    const bool g = v > best;
                    best = g ? v : best;
                    where = g ? c + j : where;
                }
                __builtin_amdgcn_sched_barrier(0);   // one block at a time: its registers
            }
            p.sv = across_max(best);
            p.si = across_min(best == p.sv ? where : INT_MAX);
        }
        p.pad = 0;
        if (lane == 0)
            ((Partial *)a.parts)[((size_t)r * tiles + tile) * kWaves + wave] = p;
    }
}

// A workgroup for a row's parts: their maximum, then the sums relative to it.
__global__ void __launch_bounds__(kJoin) join_kernel(LogitArgs a, int parts)
{
    __shared__ float s_m[kJoin / 64], s_v[kJoin / 64], s_z[kJoin / 64], s_s[kJoin / 64];
    __shared__ int s_a[kJoin / 64], s_i[kJoin / 64];
    const int lane = threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    for (long long r = blockIdx.x; r < a.R; r += gridDim.x) {
        const Partial *part = (const Partial *)a.parts + (size_t)r * parts;
        float m = -INFINITY, v = -INFINITY;
        for (int k = threadIdx.x; k < parts; k += kJoin) {
            m = fmaxf(m, part[k].m);
            v = fmaxf(v, part[k].sv);
        }
        m = across_max(m);
        v = across_max(v);
        if (lane == 0) {
            s_m[wave] = m;
            s_v[wave] = v;
        }
        __syncthreads();
        m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
        v = fmaxf(fmaxf(s_v[0], s_v[1]), fmaxf(s_v[2], s_v[3]));
        const bool none = !(m > -INFINITY);
        float z = 0.0f, s = 0.0f;
        int ai = INT_MAX, si = INT_MAX;
        for (int k = threadIdx.x; k < parts; k += kJoin) {
            const Partial p = part[k];
            const float d = none ? 0.0f : bounded(p.m - m), e = __expf(d);
            z += e * p.z;
            s += e * (p.s + d * p.z);
            ai = p.m == m ? min(ai, p.ai) : ai;
            si = p.sv == v ? min(si, p.si) : si;
        }
        z = across_sum(z);
        s = across_sum(s);
        ai = across_min(ai);
        si = across_min(si);
        if (lane == 0) {
            s_z[wave] = z;
            s_s[wave] = s;
            s_a[wave] = ai;
            s_i[wave] = si;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            z = (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]);
            s = (s_s[0] + s_s[1]) + (s_s[2] + s_s[3]);
            if (a.entropy)
                a.entropy[r] = none ? 0.0f : __logf(z) - s / z;
            if (a.sample)
                a.sample[r] = none ? -1 : min(min(s_i[0], s_i[1]), min(s_i[2], s_i[3]));
            if (a.argmax)
                a.argmax[r] = none ? -1 : min(min(s_a[0], s_a[1]), min(s_a[2], s_a[3]));
        }
        __syncthreads();
    }
}

bool has_history(const dgw4_logit_rules &u) { return u.tokens || u.n_bias > 0; }
bool has_long_history(const dgw4_logit_rules &u) { return u.tokens && u.max_tokens >= kLongHistory; }

template <class Tx, class Ty, int T, int E, bool HIST>
hipError_t adjust(const LogitArgs &a, hipStream_t st)
{
    const Cut c = cut(a.R, a.V, tile_of(T, E), HIST && a.rules.row_seq);
    if constexpr (sizeof(Tx) == sizeof(Ty)) {
        if (a.logits == a.out && !a.rules.scale) {
            adjust_kernel<Tx, Ty, T, E, HIST, true><<<dim3(c.groups), dim3(T), 0, st>>>(a, c.tiles, c.rows);
            return hipGetLastError();
        }
    }
    adjust_kernel<Tx, Ty, T, E, HIST, false><<<dim3(c.groups), dim3(T), 0, st>>>(a, c.tiles, c.rows);
    return hipGetLastError();
}

template <class Tx, class Ty, int E>
hipError_t adjust_with(const LogitArgs &a, hipStream_t st)
{
    return !has_history(a.rules)       ? adjust<Tx, Ty, kNarrow, E, false>(a, st)
           : has_long_history(a.rules) ? adjust<Tx, Ty, kBroad, E, true>(a, st)
                                       : adjust<Tx, Ty, kNarrow, E, true>(a, st);
}

template <class Tx, class Ty>
hipError_t adjust_sized(const LogitArgs &a, hipStream_t st)
{
    return per_thread(a.R, a.V) == kMany ? adjust_with<Tx, Ty, kMany>(a, st) : adjust_with<Tx, Ty, kFew>(a, st);
}

template <class Tx, int T, int E, bool HIST>
hipError_t sample(const LogitArgs &a, hipStream_t st)
{
    const Cut c = cut(a.R, a.V, tile_of(T, E), HIST && a.rules.row_seq);
    sample_adjusted_kernel<Tx, T, E, HIST><<<dim3(c.groups), dim3(T), 0, st>>>(a, c.tiles, c.rows);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    join_kernel<<<dim3(a.R < (1 << 20) ? a.R : 1 << 20), dim3(kJoin), 0, st>>>(a, c.tiles * (T / 64));
    return hipGetLastError();
}

template <class Tx, int E>
hipError_t sample_with(const LogitArgs &a, hipStream_t st)
{
    return !has_history(a.rules)       ? sample<Tx, kNarrow, E, false>(a, st)
           : has_long_history(a.rules) ? sample<Tx, kBroad, E, true>(a, st)
                                       : sample<Tx, kNarrow, E, true>(a, st);
}

template <class Tx>
hipError_t sample_sized(const LogitArgs &a, hipStream_t st)
{
    return per_thread(a.R, a.V) == kMany ? sample_with<Tx, kMany>(a, st) : sample_with<Tx, kFew>(a, st);
}

}  // namespace

hipError_t launch_adjust_logits(const LogitArgs &a, hipStream_t stream)
{
    switch (a.type) {
    case DGW4_F32: return adjust_sized<float, float>(a, stream);
    case DGW4_F16:
        return a.out_type == DGW4_F32 ? adjust_sized<_Float16, float>(a, stream)
                                      : adjust_sized<_Float16, _Float16>(a, stream);
    default:
        return a.out_type == DGW4_F32 ? adjust_sized<__bf16, float>(a, stream)
                                      : adjust_sized<__bf16, __bf16>(a, stream);
    }
}

// The parts of the rows at the wider workgroup, which has the more.
size_t sample_adjusted_workspace_bytes(int R, int V)
{
    const int tile = tile_of(kBroad, per_thread(R, V));
    return (size_t)R * (size_t)((V + tile - 1) / tile) * (kBroad / 64) * sizeof(Partial);
}

hipError_t launch_sample_adjusted(const LogitArgs &a, hipStream_t stream)
{
    switch (a.type) {
    case DGW4_F32: return sample_sized<float>(a, stream);
    case DGW4_F16: return sample_sized<_Float16>(a, stream);
    default: return sample_sized<__bf16>(a, stream);
    }
}

}  // namespace dgw4
