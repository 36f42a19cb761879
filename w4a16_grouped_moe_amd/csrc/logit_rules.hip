// A batch of requests' rules on its logits (penalties for the tokens that a
// sequence holds, biases, a scale, masks): on their own, and inside the
// sampler's pass.
//
// A workgroup takes one tile of columns of one row. It keeps a word per column
// in LDS, which the sequence's biases (the last place of a column wins: a
// maximum) and then its tokens (a count: integer additions) are entered into
// whatever their order, and meets the logits with those words.
#include "element_types.hpp"
#include "logit_rules.hpp"
#include "sampler_common.hpp"

#include <climits>

namespace dgw4 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 2048;

// The words of columns c0 .. c0 + kTile - 1 of sequence seq.
__device__ inline void enter(const LogitArgs &a, int seq, int c0, uint32_t *words)
{
    for (int i = threadIdx.x; i < kTile; i += kThreads)
        words[i] = 0;
    __syncthreads();
    if (seq < 0)
        return;
    if (a.rules.n_bias > 0) {
        const int32_t *ids = a.rules.bias_ids + (long long)seq * a.rules.ld_bias;
        for (int j = threadIdx.x; j < a.rules.n_bias; j += kThreads) {
            const uint32_t c = (uint32_t)ids[j] - (uint32_t)c0;
            if (c < (uint32_t)kTile)
                atomicMax(&words[c], (uint32_t)(j + 1) << kPlaceBit);
        }
        __syncthreads();
    }
    if (a.rules.tokens) {
        const int32_t *tok = a.rules.tokens + (long long)seq * a.rules.ld_tokens;
        const int n = min(max(a.rules.lengths[seq], 0), a.rules.max_tokens);
        const int p = a.rules.prompt_lengths ? a.rules.prompt_lengths[seq] : 0;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint32_t c = (uint32_t)tok[i] - (uint32_t)c0;
            if (c < (uint32_t)kTile) {
                atomicOr(&words[c], kSeen);
                if (i >= p)
                    atomicAdd(&words[c], 1u);
            }
        }
        __syncthreads();
    }
}

template <class Tx>
__device__ inline float rule(const LogitArgs &a, const Sequence &q, const uint32_t *mask, const Tx *row, int c, uint32_t word)
{
    const float l = adjusted(to_f32(row[c]), word, q);
    return mask && !(mask[c >> 5] >> (c & 31) & 1) ? -INFINITY : l;
}

template <class Tx, class Ty>
__global__ void __launch_bounds__(kThreads) adjust_kernel(LogitArgs a)
{
    __shared__ uint32_t words[kTile];
    const int r = blockIdx.y, c0 = (int)blockIdx.x * kTile;
    const int seq = sequence_of(a.rules, r);
    const uint32_t *mask = mask_of(a.rules, r);
    enter(a, seq, c0, words);
    const Sequence q = sequence(a.rules, seq);
    const Tx *row = (const Tx *)a.logits + (long long)r * a.ld;
    Ty *out = (Ty *)a.out + (long long)r * a.ld_out;
    for (int i = threadIdx.x; i < kTile && c0 + i < a.V; i += kThreads)
        out[c0 + i] = from_f32<Ty>(rule(a, q, mask, row, c0 + i, words[i]));
}

// p and q joined. A part that vanishes beside the other is left out: its distance
// times z may be infinite (a mask of the type's lowest value).
__device__ inline void join(Partial &p, const Partial &q)
{
    const float top = fmaxf(p.m, q.m);
    const float a = p.z > 0.0f ? __expf(p.m - top) : 0.0f, b = q.z > 0.0f ? __expf(q.m - top) : 0.0f;
    p.s = (a > 0.0f ? a * (p.s + (p.m - top) * p.z) : 0.0f) + (b > 0.0f ? b * (q.s + (q.m - top) * q.z) : 0.0f);
    p.z = a * p.z + b * q.z;
    p.m = top;
    take_best(p.av, p.ai, q.av, q.ai);
    take_best(p.sv, p.si, q.sv, q.si);
}

template <class Tx>
__global__ void __launch_bounds__(kThreads) sample_adjusted_kernel(LogitArgs a)
{
    __shared__ uint32_t words[kTile];
    __shared__ Partial parts[kThreads];
    const int r = blockIdx.y, c0 = (int)blockIdx.x * kTile;
    const int seq = sequence_of(a.rules, r);
    const uint32_t *mask = mask_of(a.rules, r);
    enter(a, seq, c0, words);
    const Sequence q = sequence(a.rules, seq);
    const Tx *row = (const Tx *)a.logits + (long long)r * a.ld;
    Partial p = {-INFINITY, 0.0f, 0.0f, -INFINITY, INT_MAX, -INFINITY, INT_MAX, 0};
    for (int i = threadIdx.x; i < kTile && c0 + i < a.V; i += kThreads) {
        const int c = c0 + i;
        const float l = rule(a, q, mask, row, c, words[i]);
        if (l == -INFINITY)
            continue;
        Partial one = {l, 1.0f, 0.0f, l, c, -INFINITY, INT_MAX, 0};
        if (a.sample) {
            uint32_t w[4];
            philox4x32_10((uint32_t)c >> 2, (uint32_t)r, 0u, 0u, a.k0, a.k1, w);
            one.sv = l + gumbel(w[c & 3]);
            one.si = c;
        }
        join(p, one);
    }
    parts[threadIdx.x] = p;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if ((int)threadIdx.x < o)
            join(parts[threadIdx.x], parts[threadIdx.x + o]);
        __syncthreads();
    }
    if (threadIdx.x == 0)
        ((Partial *)a.parts)[(size_t)r * gridDim.x + blockIdx.x] = parts[0];
}

__global__ void __launch_bounds__(64) merge_adjusted_kernel(LogitArgs a, int parts)
{
    const int r = blockIdx.x * 64 + (int)threadIdx.x;
    if (r >= a.R)
        return;
    const Partial *part = (const Partial *)a.parts + (size_t)r * parts;
    Partial p = part[0];
    for (int k = 1; k < parts; ++k)
        join(p, part[k]);
    const bool none = p.z == 0.0f;
    if (a.entropy)
        a.entropy[r] = none ? 0.0f : __logf(p.z) - p.s / p.z;
    if (a.sample)
        a.sample[r] = none ? -1 : p.si;
    if (a.argmax)
        a.argmax[r] = none ? -1 : p.ai;
}

int tiles_of(int V) { return (V + kTile - 1) / kTile; }

template <class Tx, class Ty>
hipError_t adjust(const LogitArgs &a, hipStream_t st)
{
    adjust_kernel<Tx, Ty><<<dim3(tiles_of(a.V), a.R), dim3(kThreads), 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adjust_logits(const LogitArgs &a, hipStream_t stream)
{
    switch (a.type) {
    case DGW4_F32: return adjust<float, float>(a, stream);
    case DGW4_F16:
        return a.out_type == DGW4_F32 ? adjust<_Float16, float>(a, stream) : adjust<_Float16, _Float16>(a, stream);
    default: return a.out_type == DGW4_F32 ? adjust<__bf16, float>(a, stream) : adjust<__bf16, __bf16>(a, stream);
    }
}

size_t sample_adjusted_workspace_bytes(int R, int V)
{
    return (size_t)R * (size_t)tiles_of(V) * sizeof(Partial);
}

hipError_t launch_sample_adjusted(const LogitArgs &a, hipStream_t stream)
{
    const dim3 grid(tiles_of(a.V), a.R);
    switch (a.type) {
    case DGW4_F32: sample_adjusted_kernel<float><<<grid, dim3(kThreads), 0, stream>>>(a); break;
    case DGW4_F16: sample_adjusted_kernel<_Float16><<<grid, dim3(kThreads), 0, stream>>>(a); break;
    default: sample_adjusted_kernel<__bf16><<<grid, dim3(kThreads), 0, stream>>>(a);
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    merge_adjusted_kernel<<<dim3((a.R + 63) / 64), dim3(64), 0, stream>>>(a, (int)grid.x);
    return hipGetLastError();
}

}  // namespace dgw4
