// How the rows of a batch's logits are cut into workgroups (not part of the ABI).
// Plain C++, which a host program can ask too.
#pragma once

#include <cstdint>

namespace dgw4 {
namespace {

// Threads of a workgroup. Long histories take the wider one: each workgroup reads
// its rows' whole histories, so half as many of them read half as much (64
// sequences of up to 60000 tokens: 81 -> 66 us, of 16000 51 -> 48, one of 120000: 37
// -> 25). Short ones take the narrower: more workgroups on a compute unit hide each
// other's steps (a canvas of 4 sequences of 8000: 75 us against 79).
// The tokens' buffer decides, for the host does not know the lengths: a buffer of
// 131072 tokens a sequence with short histories in it takes the wider one too (that
// canvas without masks 67 us against 64, 64 rows of 1000 tokens in place 23.5
// against 21, greedy 30.1 against 29.3, one row of 200 drawn 9.1 against 8.5), which
// a view of the columns in use avoids.
constexpr int kNarrow = 256, kBroad = 512;
constexpr int kLongHistory = 16384;

// Columns of a tile: of a workgroup of `threads` that take E columns each; of a wave.
constexpr int tile_of(int threads, int e) { return threads * e; }
constexpr int part_of(int e) { return 64 * e; }

// Columns a thread takes: few where that makes too few waves for the chip.
constexpr int kFew = 8, kMany = 16;

inline int per_thread(int R, int V)
{
    return (long long)R * ((V + part_of(kMany) - 1) / part_of(kMany)) >= 4096 ? kMany : kFew;
}

// Tiles of a row, and the rows that a workgroup takes in turn: where rows share
// sequences, those of one lie next to each other, and the words are entered once
// for them.
struct Cut {
    int tiles, rows;
    uint32_t groups;
};

inline Cut cut(int R, int V, int tile, bool shared)
{
    Cut c;
    c.tiles = (V + tile - 1) / tile;
    const long long pairs = (long long)R * c.tiles, resident = 2048, most = 1 << 22;
    long long rows = shared ? (pairs + resident - 1) / resident : 1;
    rows = rows > 32 ? 32 : rows;
    if (pairs / rows > most)                         // a launch has at most 2^32 threads
        rows = (pairs + most - 1) / most;
    c.rows = (int)rows;
    c.groups = (uint32_t)((R + rows - 1) / rows * c.tiles);
    return c;
}

}  // namespace
}  // namespace dgw4
