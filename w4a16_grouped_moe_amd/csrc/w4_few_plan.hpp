// How a few-token W4A16 call is cut up (not part of the ABI). Plain C++, which a
// host program can ask too.
#pragma once

#include <climits>
#include <cstddef>
#include <cstdint>

namespace dgw4 {
namespace {

// How a call is cut up. A turn is what a workgroup takes at a time: its waves in
// sets of 1 << split, each set 16 CB channels, the waves of a set every
// (1 << split)-th 128 columns of K.
struct Plan {
    int split, turns, batches;
    int tokens;                 // of a workgroup: blockIdx.y says which
    uint32_t magic;             // of the division by the vectors of a row (whole K in LDS)
};

// Groups of a batch: what a wave holds of the weights, each refilled with the
// next batch's as soon as it has been used.
template <int G>
constexpr int kHeld = 512 / G;

// The kernels' forms: waves of a workgroup, blocks of 16 tokens and of 16 channels
// that a wave takes, x's chunk in units of 512 columns (0: x whole), workgroups
// that run at once, the most waves that share channels and the step between such
// numbers (logarithms).
struct Form {
    int waves, tb, cb, m, resident, max_split, step;
};
constexpr int kWhole8 = 0, kWhole16 = 1, kLongK = 2, kBlocks2 = 3, kBlocks4 = 4;
constexpr Form kForms[] = {
    {8, 1, 1, 0, 512, 3, 1}, {16, 1, 1, 0, 256, 4, 1}, {16, 1, 1, 4, 256, 4, 2},
    {16, 2, 1, 1, 256, 2, 1}, {8, 4, 2, 1, 256, 2, 1},
};

constexpr size_t kLds = 160 * 1024;

// Dynamic LDS of a workgroup of `tokens` tokens: rows of x 16 bytes off the bank
// period and each group's sums of 16 tb tokens, two halves of both for chunks,
// where the waves' sums meet in the same place.
inline size_t lds_of(const Form &f, int tokens, int K, int g)
{
    if (f.m == 0)
        return (size_t)tokens * (K * 2 + 16) + (size_t)(K / g) * 64;
    const size_t x = 2 * ((size_t)tokens * (64 * f.m * 16 + 16) + 512 / g * f.m * f.tb * 64);
    const size_t sums = (size_t)f.waves * f.tb * f.cb * 1024;
    return x > sums ? x : sums;
}

// The form for T tokens, and how many of them a workgroup takes.
//
// More than 16 tokens share each weight's unpacking in one workgroup, unless there
// are so few channels that workgroups of 16 or of 32 tokens each (which read the
// same weights, from the caches but for one of them) still run all at once. In a
// graph, us in blocks of 16 / of 32 / whole:
//   64 tokens, K 2816: 1024 channels 7.0 / 11.3 / 17.8, 8192 26 / 12.4 / 18.5,
//     16384 35 / 25 / 20
//   64 tokens, K 8192: 1024 channels 11 / 23 / 38, 8192 69 / 26 / 39, 16384 80 / 55 / 43
//   32 tokens, K 1408: 2048 channels 5.2 / 8.2 / 10, 8192 12 / 8.5 / 10
// Just past a border the form before it would still be the faster for some: 32
// tokens, K 1408, 2064 channels 6.6 / 8.2, 20 tokens, K 8192, 2064 channels 15 / 21
// (of 132 sizes the worst; nine lose more than 15%, all within twice a border).
inline int form_of(int T, int K, int N, int g, int &tokens)
{
    constexpr int kChip = 256;
    const long long by16 = (T + 15) / 16 * ((N + 15LL) / 16), by32 = (T + 31) / 32 * ((N + 63LL) / 64);
    if (T <= 16 || by16 <= kChip) {
        tokens = T < 16 ? T : 16;
        if (lds_of(kForms[kWhole8], tokens, K, g) + 8 * 1024 <= kLds / 2)
            return kWhole8;
        return lds_of(kForms[kWhole16], tokens, K, g) + 16 * 1024 <= kLds ? kWhole16 : kLongK;
    }
    if (T <= 32 || by32 <= kChip) {
        tokens = T < 32 ? T : 32;
        return kBlocks2;
    }
    tokens = T;
    return kBlocks4;
}

// The plan whose split takes the least time by an estimate: rounds of the chip times
// what a wave does in one, in quarters of a unit of 128 columns: four a unit, and
// for the turn's beginning and end half a unit, or one and a half where waves join
// in LDS (both set by hand). Against each split by itself, 23 sizes of 1 to 64
// tokens: 5% slower than the best on average, 16% at worst (16 x 8192 x 8192 21 us
// against 18; two timings of one split are up to 10% apart).
inline Plan plan_of(const Form &f, int tokens, int K, int N)
{
    constexpr int held = 4;     // units of 128 columns in a batch
    const int units = (K + 127) / 128;
    Plan pl{};
    long long best = LLONG_MAX;
    for (int split = 0; split <= f.max_split; split += f.step) {
        const int per = (f.waves >> split) * 16 * f.cb;
        const long long turns = ((long long)N + per - 1) / per, rounds = (turns + f.resident - 1) / f.resident;
        const long long each = (units + (1 << split) - 1) >> split;
        const long long cost = rounds * (each * 4 + (split ? 6 : 2));
        if (cost < best) {
            best = cost;
            pl.split = split;
            pl.turns = (int)turns;
            pl.batches = (int)((each + held - 1) / held);
        }
    }
    pl.tokens = tokens;
    pl.magic = (uint32_t)(((1ull << 32) + K / 8 - 1) / (K / 8));
    return pl;
}

}  // namespace
}  // namespace dgw4
