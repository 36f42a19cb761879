// Which tile an 8-bit product runs on (not part of the ABI). Plain C++, which a
// host program can ask too.
#pragma once

#include <cmath>

namespace dgw4 {

constexpr int kStageK = 128;                     // bytes of K per stage

// The tile by the least estimated time, in us past what every launch costs: a
// workgroup takes fixed + stage * (128-byte stages of K), times the rounds of
// the chip's 256 compute units. A workgroup that fills one by its LDS runs in
// whole rounds (per_cu 0); the others share it, per_cu of them in a workgroup's
// time. Fitted to 68 shapes (33 to 4096 tokens, 64 to 65536 channels, K 704 to
// 16384) that every tile was timed on: the choice is within 1% of the best
// tile on average and 11% at worst, where tiles of whole K alone were 20% and
// 117% off. Some, us, 64 x 32 with whole K / the tile taken now:
//   T 252, N 737, K 8544: 17.1 / 10.5 (32 x 32, four parts of K)
//   T 256, N 4096, K 2816: 9.8 / 8.4 (64 x 64, two parts)
//   T 128, N 4096, K 4096: 10.0 / 8.3 (64 x 32, two parts)
struct I8Tile {
    int bn, bt, threads;
    double stage, fixed, per_cu;
};
constexpr I8Tile kTiles[] = {
    {256, 256, 512, 1.80, 8.1, 0.0}, {256, 128, 512, 0.94, 6.1, 0.0}, {128, 128, 512, 0.59, 3.7, 0.0},
    {64, 128, 512, 0.34, 2.8, 0.0},  {64, 64, 512, 0.24, 1.7, 0.0},   {64, 64, 512, 0.30, 0.9, 1.1},
    {64, 32, 512, 0.15, 0.8, 0.8},   {32, 32, 512, 0.11, 0.7, 1.0},   {32, 32, 1024, 0.093, 1.6, 0.0},
};

// The tile for T tokens, K codes a row and N channels, by its place in kTiles.
inline int pick_tile(int T, int K, int N)
{
    const int stages = (K + kStageK - 1) / kStageK;
    int best = 0;
    double least = HUGE_VAL;
    for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
        const I8Tile &t = kTiles[i];
        const double tiles = (double)((N + t.bn - 1) / t.bn) * ((T + t.bt - 1) / t.bt) / 256.0;
        const double rounds = t.per_cu == 0.0 ? std::ceil(tiles) : std::fmax(1.0, tiles / t.per_cu);
        const double us = (t.fixed + t.stage * stages) * rounds;
        // a launch takes fewer than 2^32 threads; the first tile's stay under
        // that for every y that fits the device
        if (us < least && (i == 0 || tiles * 256.0 * t.threads < 4294967296.0)) {
            least = us;
            best = i;
        }
    }
    return best;
}

}  // namespace dgw4
