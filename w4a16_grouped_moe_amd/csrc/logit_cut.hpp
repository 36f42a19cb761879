// How the rows of a batch's logits are cut into workgroups (not part of the ABI).
// Plain C++, which a host program can ask too.
#pragma once

#include <cstdint>

namespace dgw4 {
namespace {

// Threads of a workgroup. Long histories take the wider one: each workgroup reads
// its rows' whole histories, so half as many of them read half as much (64
// sequences of 60000 tokens: 80 -> 66 us, one of 120000: 37 -> 24). Short ones
// take the narrower: more workgroups on a compute unit hide each other's steps (a
// canvas of 4 sequences of 8000: 76 us against 80).
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
