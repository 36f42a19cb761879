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
// On their own the logits meet the words as they pass. Inside the sampler, where
// the arithmetic counts, a wave first lists the few columns whose word is not
// zero; the pass over its columns takes them like masked ones (one bit a column)
// and the listed ones follow, a lane each.
//
// A wave's part of a row (the maximum, its first place, sums of exp relative to
// it, the best score) goes to the workspace; a second kernel joins a row's parts.
// Every order is fixed, so results are bitwise reproducible.
#include "element_types.hpp"
#include "logit_rules.hpp"
#include "sampler_common.hpp"

#include <climits>
#include <type_traits>

namespace dgw4 {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// Columns of a workgroup's tile whose threads take E columns each, and of its waves.
template <int E>
constexpr int kTile = kThreads * E;
template <int E>
constexpr int kPart = 64 * E;

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

// The words of columns c0 .. of sequence seq, by the whole workgroup.
template <int TILE>
__device__ inline void enter(const dgw4_logit_rules &u, int seq, int c0, uint32_t *words)
{
    __syncthreads();
    for (int i = threadIdx.x * 4; i < TILE; i += kThreads * 4)
        *reinterpret_cast<uint4 *>(words + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (seq < 0)
        return;
    if (u.n_bias > 0) {
        const int32_t *ids = u.bias_ids + (long long)seq * u.ld_bias;
        for (int j = threadIdx.x; j < u.n_bias; j += kThreads) {
            const uint32_t c = (uint32_t)ids[j] - (uint32_t)c0;
            if (c < (uint32_t)TILE)
                atomicMax(&words[c], (uint32_t)(j + 1) << kPlaceBit);
        }
        __syncthreads();
    }
    if (u.tokens) {
        const int32_t *tok = u.tokens + (long long)seq * u.ld_tokens;
        const int n = min(max(u.lengths[seq], 0), u.max_tokens);
        const int p = u.prompt_lengths ? u.prompt_lengths[seq] : 0;
        auto one = [&](int t, int i) {
            const uint32_t c = (uint32_t)t - (uint32_t)c0;
            if (c < (uint32_t)TILE) {
                if (i < p)
                    atomicOr(&words[c], kPrompt);
                else
                    atomicAdd(&words[c], 1u);
            }
        };
        constexpr int kAhead = 4;                    // loads of four tokens a thread has on their way
        int i = threadIdx.x * 4;
        for (; i + (kAhead - 1) * kThreads * 4 + 3 < n; i += kAhead * kThreads * 4) {
            int4 t[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                __builtin_memcpy(&t[j], tok + i + j * kThreads * 4, 16);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int at = i + j * kThreads * 4;
                one(t[j].x, at);
                one(t[j].y, at + 1);
                one(t[j].z, at + 2);
                one(t[j].w, at + 3);
            }
        }
        for (; i < n; i += kThreads * 4)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k < n)
                    one(tok[i + k], i + k);
        __syncthreads();
    }
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

// The mask's bits of columns c .. c + W - 1 (c a multiple of W) in the low bits; past V: anything.
template <int W>
__device__ inline uint32_t allowed(const uint32_t *mask, int c, int V)
{
    return mask && c < V ? mask[c >> 5] >> (c & 31) : ~0u;
}

// E columns a thread; SPARSE: in place and no scale, so only what changes is read and written.
template <class Tx, class Ty, int E, bool HIST, bool SPARSE>
__global__ void __launch_bounds__(kThreads) adjust_kernel(LogitArgs a, int tiles, int rows)
{
    constexpr int W = Wide<Tx>::W, N = E / W;        // columns of a vector, vectors of a thread
    __shared__ __attribute__((aligned(16))) uint32_t words[HIST ? kTile<E> : 4];
    const int tile = (int)(blockIdx.x % (uint32_t)tiles), r0 = (int)(blockIdx.x / (uint32_t)tiles) * rows;
    const int c0 = tile * kTile<E>;
    int seq = -2;
    for (int r = r0; r < min(r0 + rows, a.R); ++r) {
        const int s = sequence_of(a.rules, r);
        const uint32_t *mask = mask_of(a.rules, r);
        if (HIST && s != seq)
            enter<kTile<E>>(a.rules, s, c0, words);
        seq = s;
        const Sequence q = sequence(a.rules, s);
        const Tx *row = (const Tx *)a.logits + (long long)r * a.ld;
        Ty *out = (Ty *)a.out + (long long)r * a.ld_out;
        typename Wide<Tx>::vec x[N];
        uint32_t bits[N], any[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int c = c0 + (k * kThreads + (int)threadIdx.x) * W;
            bits[k] = allowed<W>(mask, c, a.V);
            any[k] = 0;
            if (HIST) {
                const uint32_t *w = words + c - c0;
#pragma unroll
                for (int i = 0; i < W; ++i)
                    any[k] |= w[i];
            }
            if (c < a.V && (!SPARSE || any[k] || (bits[k] & ((1u << W) - 1)) != (1u << W) - 1))
                x[k] = read_wide(row, c, a.V);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int c = c0 + (k * kThreads + (int)threadIdx.x) * W;
            if (c >= a.V || (SPARSE && !any[k] && (bits[k] & ((1u << W) - 1)) == (1u << W) - 1))
                continue;
            float l[W];
#pragma unroll
            for (int i = 0; i < W; ++i)
                l[i] = to_f32(x[k][i]);
            if (HIST && any[k]) {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    l[i] = adjusted(l[i], words[c - c0 + i], q);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    l[i] = rounded_product(l[i], q.scale);
            }
            typedef Ty vec __attribute__((ext_vector_type(W), aligned(sizeof(Ty))));
            vec y;
#pragma unroll
            for (int i = 0; i < W; ++i)
                y[i] = from_f32<Ty>(bits[k] >> i & 1 ? l[i] : -INFINITY);
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

// A part of a row in a wave, the same in all lanes.
struct Part {
    float m, z, s;              // max, sum exp(l - m), sum exp(l - m) * (l - m)
    int ai;                     // the first place of m
    float sv;                   // the best score and its first place
    int si;
};

template <class Tx, int E, bool HIST>
__global__ void __launch_bounds__(kThreads, 4) sample_adjusted_kernel(LogitArgs a, int tiles, int rows)
{
    constexpr int W = Wide<Tx>::W, N = E / W;
    __shared__ __attribute__((aligned(16))) uint32_t words[HIST ? kTile<E> : 4];
    __shared__ uint32_t touched[HIST ? kTile<E> / 32 : 4];
    __shared__ uint16_t listed[HIST ? kWaves : 1][HIST ? kPart<E> : 2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int tile = (int)(blockIdx.x % (uint32_t)tiles), r0 = (int)(blockIdx.x / (uint32_t)tiles) * rows;
    const int c0 = tile * kTile<E>, first = wave * kPart<E>;       // the tile's and, in it, the wave's columns
    int seq = -2, count = 0;
    for (int r = r0; r < min(r0 + rows, a.R); ++r) {
        const int s = sequence_of(a.rules, r);
        const uint32_t *mask = mask_of(a.rules, r);
        const Tx *row = (const Tx *)a.logits + (long long)r * a.ld;
        const Sequence q = sequence(a.rules, s);
        typename Wide<Tx>::vec x[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int c = c0 + first + (k * 64 + lane) * W;
            if (c < a.V)
                x[k] = read_wide(row, c, a.V);
        }
        if (HIST && s != seq) {
            enter<kTile<E>>(a.rules, s, c0, words);
            // the wave's columns with a word, in ascending order
            count = 0;
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const bool is = words[first + k * 64 + lane] != 0;
                const uint64_t all = __ballot(is);
                if (lane == 0) {
                    touched[(first + k * 64) / 32] = (uint32_t)all;
                    touched[(first + k * 64) / 32 + 1] = (uint32_t)(all >> 32);
                }
                if (is)
                    listed[wave][count + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32),
                                                                   __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0))] =
                        (uint16_t)(first + k * 64 + lane);
                count += __popcll(all);
            }
            // other lanes of the wave read them
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        seq = s;
        // the first of the listed, ahead of the columns' arithmetic
        int lc = 0;
        float ll = -INFINITY;
        auto get_listed = [&](int at) {
            ll = -INFINITY;
            lc = INT_MAX;
            if (at + lane < count) {
                const int c = listed[wave][at + lane];
                lc = c0 + c;
                if (lc < a.V && (allowed<1>(mask, lc, a.V) & 1))
                    ll = adjusted(to_f32(row[lc]), words[c], q);
            }
        };
        if (HIST)
            get_listed(0);

        float l[E];
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int c = c0 + first + (k * 64 + lane) * W;
            uint32_t bits = allowed<W>(mask, c, a.V);
            if (HIST)
                bits &= ~(touched[(c - c0) >> 5] >> (c & 31));
            if (c + W > a.V)
                bits &= c < a.V ? (1u << (a.V - c)) - 1 : 0u;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                l[k * W + i] = bits >> i & 1 ? rounded_product(to_f32(x[k][i]), q.scale) : -INFINITY;
                top = fmaxf(top, l[k * W + i]);
            }
        }
        Part p;
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
        p.ai = across_min(at) + c0 + first;
        p.sv = -INFINITY;
        p.si = INT_MAX;
        if (a.sample) {
            float best = -INFINITY;
            int where = INT_MAX;
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const int c = c0 + first + (e / W * 64 + lane) * W + e % W;
                uint32_t w[4];
                philox4x32_10((uint32_t)c >> 2, (uint32_t)r, 0u, 0u, a.k0, a.k1, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float v = l[e + j] + gumbel(w[j]);
                    const bool g = v > best;
                    best = g ? v : best;
                    where = g ? c + j : where;
                }
            }
            p.sv = across_max(best);
            p.si = across_min(best == p.sv ? where : INT_MAX);
        }
        for (int i = 0; HIST && i < count; i += 64) {
            if (i > 0)
                get_listed(i);
            const float lm = across_max(ll);
            if (!(lm > -INFINITY))
                continue;
            const int la = across_min(ll == lm ? lc : INT_MAX);
            p.ai = lm > p.m ? la : lm == p.m ? min(la, p.ai) : p.ai;
            const float nm = fmaxf(lm, p.m), d = bounded(p.m - nm), shrink = p.z > 0.0f ? __expf(d) : 0.0f;
            const float ld = bounded(ll - nm), le = __expf(ld);
            p.s = shrink * (p.s + d * p.z) + across_sum(le * ld);
            p.z = shrink * p.z + across_sum(le);
            p.m = nm;
            if (a.sample) {
                uint32_t w[4];
                philox4x32_10((uint32_t)lc >> 2, (uint32_t)r, 0u, 0u, a.k0, a.k1, w);
                const uint32_t word = lc & 2 ? lc & 1 ? w[3] : w[2] : lc & 1 ? w[1] : w[0];
                const float v = ll + gumbel(word), best = across_max(v);
                const int where = across_min(v == best ? lc : INT_MAX);
                p.si = best > p.sv ? where : best == p.sv ? min(where, p.si) : p.si;
                p.sv = fmaxf(best, p.sv);
            }
        }
        if (lane == 0) {
            const Partial out = {p.m, p.z, p.s, p.m, p.ai, p.sv, p.si, 0};
            ((Partial *)a.parts)[((size_t)r * tiles + tile) * kWaves + wave] = out;
        }
    }
}

// A workgroup for a row's parts: their maximum, then the sums relative to it.
__global__ void __launch_bounds__(kThreads) join_kernel(LogitArgs a, int parts)
{
    __shared__ float s_m[kWaves], s_v[kWaves], s_z[kWaves], s_s[kWaves];
    __shared__ int s_a[kWaves], s_i[kWaves];
    const int lane = threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    for (long long r = blockIdx.x; r < a.R; r += gridDim.x) {
        const Partial *part = (const Partial *)a.parts + (size_t)r * parts;
        float m = -INFINITY, v = -INFINITY;
        for (int k = threadIdx.x; k < parts; k += kThreads) {
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
        for (int k = threadIdx.x; k < parts; k += kThreads) {
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

// Columns a thread takes: few where that makes too few waves for the chip.
constexpr int kFew = 8, kMany = 16;

int per_thread(int R, int V)
{
    return (long long)R * ((V + kPart<kMany> - 1) / kPart<kMany>) >= 4096 ? kMany : kFew;
}

// Tiles of a row, and the rows that a workgroup takes in turn: those of a
// sequence lie next to each other where rows share sequences, and the words are
// entered once for them.
struct Cut {
    int tiles, rows;
    uint32_t groups;
};

Cut cut(const LogitArgs &a, int e, bool shared)
{
    Cut c;
    c.tiles = (a.V + kThreads * e - 1) / (kThreads * e);
    const long long pairs = (long long)a.R * c.tiles, resident = 2048, most = 1 << 23;
    long long rows = shared ? (pairs + resident - 1) / resident : 1;
    rows = rows > 32 ? 32 : rows;
    if (pairs / rows > most)                         // a launch has at most 2^32 threads
        rows = (pairs + most - 1) / most;
    c.rows = (int)rows;
    c.groups = (uint32_t)((a.R + rows - 1) / rows * c.tiles);
    return c;
}

bool has_history(const dgw4_logit_rules &u) { return u.tokens || u.n_bias > 0; }

template <class Tx, class Ty, int E>
hipError_t adjust(const LogitArgs &a, hipStream_t st)
{
    const bool hist = has_history(a.rules), sparse = a.logits == a.out && !a.rules.scale;
    const Cut c = cut(a, E, hist && a.rules.row_seq);
    const dim3 grid(c.groups), block(kThreads);
    if constexpr (sizeof(Tx) == sizeof(Ty)) {
        if (sparse) {
            if (hist)
                adjust_kernel<Tx, Ty, E, true, true><<<grid, block, 0, st>>>(a, c.tiles, c.rows);
            else
                adjust_kernel<Tx, Ty, E, false, true><<<grid, block, 0, st>>>(a, c.tiles, c.rows);
            return hipGetLastError();
        }
    }
    if (hist)
        adjust_kernel<Tx, Ty, E, true, false><<<grid, block, 0, st>>>(a, c.tiles, c.rows);
    else
        adjust_kernel<Tx, Ty, E, false, false><<<grid, block, 0, st>>>(a, c.tiles, c.rows);
    return hipGetLastError();
}

template <class Tx, class Ty>
hipError_t adjust_sized(const LogitArgs &a, hipStream_t st)
{
    return per_thread(a.R, a.V) == kMany ? adjust<Tx, Ty, kMany>(a, st) : adjust<Tx, Ty, kFew>(a, st);
}

template <class Tx, int E>
hipError_t sample(const LogitArgs &a, hipStream_t st)
{
    const bool hist = has_history(a.rules);
    const Cut c = cut(a, E, hist && a.rules.row_seq);
    if (hist)
        sample_adjusted_kernel<Tx, E, true><<<dim3(c.groups), dim3(kThreads), 0, st>>>(a, c.tiles, c.rows);
    else
        sample_adjusted_kernel<Tx, E, false><<<dim3(c.groups), dim3(kThreads), 0, st>>>(a, c.tiles, c.rows);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    join_kernel<<<dim3(a.R < (1 << 20) ? a.R : 1 << 20), dim3(kThreads), 0, st>>>(a, c.tiles * kWaves);
    return hipGetLastError();
}

template <class Tx>
hipError_t sample_sized(const LogitArgs &a, hipStream_t st)
{
    return per_thread(a.R, a.V) == kMany ? sample<Tx, kMany>(a, st) : sample<Tx, kFew>(a, st);
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

size_t sample_adjusted_workspace_bytes(int R, int V)
{
    const int tile = kThreads * per_thread(R, V);
    return (size_t)R * (size_t)((V + tile - 1) / tile) * kWaves * sizeof(Partial);
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
