// Which form a product in 8-bit blocks takes (host only): rules on its sizes, each with what both
// sides of it measured, us a call on 256 compute units unless stated.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace exl3 {

constexpr int kBlock = 128;                      // elements a scale serves along a row
constexpr int blocks_of(int width) { return (width + kBlock - 1) / kBlock; }

// y[n][m] from x[n][k], a matrix for each of `groups`.
struct BlockCall {
    int64_t n;
    int m, k, groups;
    bool offsets, transposed;
};

// Streamed (block_rows_kernel), with 16-bit rows written as blocks by the workgroups or with
// blocks; else tiles, columns x rows, and how many sets of waves split the contraction (two of
// kTile128x128Twice share a compute unit).
enum BlockForm {
    kOwnRows,
    kFewRows,
    kTile256x256,
    kTile256x128,
    kTile128x128Twice,
    kTile128x128,
    kTile128x64,                                 // two sets
    kTile128x32,                                 // two
    kTile64x32,                                  // four
    kTile32x32,                                  // four
    kNoForm                                      // more tiles than a launch holds
};

// Whether the streaming workgroups write 16-bit rows as blocks themselves, each all that it needs,
// in place of a launch before: up to some 28,000 elements on a compute unit, us with and without:
// 2 rows, 12288 x 4096 (24,576): 13.1, 15.1; 4 rows, 4096 x 4096 (16,384): 7.9, 10.0; 8 rows
// (32,768): 10.6, 10.1; 4 rows, 12288 x 4096 (49,152): 15.4, 14.8.  Counted in whole blocks, and
// with all rows in one group as well (up to 33,000), as nothing says where they go: 16 experts of
// 1408 x 2048, 16 rows: even 12.6 and 13.9, in one 11.9 and 12.0; 32 rows: 13.0 and 14.0, 20.4 and
// 12.3.
// And up to four passes of 16 rows, one after the other, or six over a unit's workgroups: 256 or
// 4,096 columns from 64, 64 rows 9.1 to 9.3 and 11.7, 96 rows 12.4 and 11.3, 437 rows 50 and 12;
// 12,288 columns (three workgroups a unit), 32 rows 9.5 and 11.9, 64 rows 16.5 and 11.6; 64 experts
// of 256 x 256, 64 rows in one: 10.2 and 12.1, 512: 61 and 12.
inline bool takes_own_rows(const BlockCall &c, int n_cu) {
    if (c.transposed) return false;
    const int64_t wide = (int64_t)blocks_of(c.k) * kBlock, one = (c.m + 15) / 16;
    const int64_t rows = (c.n + c.groups - 1) / c.groups, passes = (c.n + 15) / 16;
    return rows * wide * std::max<int64_t>(n_cu, one * c.groups) <= (int64_t)28000 * n_cu &&
           c.n * wide * std::max<int64_t>(n_cu, one) <= (int64_t)33000 * n_cu && passes <= 4 &&
           passes * ((one + n_cu - 1) / n_cu) <= 6;
}

// Whether experts' matrices are streamed through registers for few rows each (up to 16), or go
// through the tiles, whose smallest for them have 128 columns of the result by 32 rows.  A single
// matrix goes through tiles, the smallest of 32 x 32 (or is streamed as above).  Estimates in us,
// of both as measured: 64 experts of 1408 x 2048, 64 rows: 25.4 and 26.7, 256: 36.9 and 41.0, 512:
// 45.8 and 41.8; 16 of 2048 x 1408, 16 rows: 9.8 and 9.4, 64: 13.6 and 11.7.
inline bool takes_few_rows(const BlockCall &c, int n_cu) {
    if (c.transposed || c.groups == 1 || c.n > (int64_t)16 * c.groups) return false;
    const double rows = (double)c.n / c.groups, mb = 1e-6 * c.m * c.k * c.groups;
    const double streamed = 3.5 + mb * (0.16 + 0.01 * rows);
    const double tiles = (c.m + 127) / 128 * (c.n / 32 + 0.5 * c.groups);
    const double steps = (blocks_of(c.k) + 1) / 2;
    const double tiled =
        3.2 + std::max(0.44 * steps * std::max(1.0, tiles / n_cu), mb / 4.9);
    return streamed < tiled;
}

// The tiles, by what a step of a round takes, us (a tile a compute unit, but two of
// kTile128x128Twice; a step is a block for each set), from calls of 4,096 columns from 4,096 with
// 64 rows (32 x 32: 7.4), 128 (64 x 32: 8.5), 200 (128 x 32: 11.3), 512 (128 x 64: 14.2), 1,024
// (128 x 128: 21.9; two rounds of 128 x 64: 27), 2,000 (256 x 128: 33; 128 x 128, two a unit: 36)
// and of 12,288 with 4,096 rows (three rounds of 256 x 256: 167; six of 256 x 128: 199); some 3 us
// of each are not in steps.  The contraction in four sets where tiles are few: 4,096 columns from
// 12,288, 24 rows: 11.8, 128 x 32 in two sets: 23.  Experts' tiles: each group's last is half empty
// on average, and rounds run into one another; none of less than 128 columns (16 of 2048 x 1408, 64
// rows: 128 x 32 11.6, 64 x 32 15.2, 32 x 32 21.7).
inline BlockForm block_tile(const BlockCall &c, int n_cu) {
    struct Tile {
        int bm, bn, sets, places;
        double us;
    };
    const Tile tiles[] = {{256, 256, 1, 1, 1.7}, {256, 128, 1, 1, 1.0}, {128, 128, 1, 2, 1.03},
                          {128, 128, 1, 1, 0.6}, {128, 64, 2, 1, 0.83}, {128, 32, 2, 1, 0.67},
                          {64, 32, 4, 1, 0.78},  {32, 32, 4, 1, 0.5}};
    int best = kNoForm;
    double least = 1e30;
    for (int i = 0; i < 8; ++i) {
        const Tile &t = tiles[i];
        if (c.offsets && t.bm < 128) continue;
        const int64_t m_tiles = (c.m + t.bm - 1) / t.bm, whole = (c.n + t.bn - 1) / t.bn;
        // a launch has fewer than 2^32 lanes, of up to 512 a workgroup
        if (m_tiles * (c.offsets ? c.n / t.bn + c.groups : whole) >= (int64_t)1 << 23) continue;
        const double steps = (blocks_of(c.k) + t.sets - 1) / t.sets, places = t.places * n_cu;
        const double rounds =
            c.offsets ? std::max(1.0, m_tiles * ((double)c.n / t.bn + 0.5 * c.groups) / places)
                      : std::ceil((double)(m_tiles * whole) / places);
        const double cost = t.us * steps * rounds;
        if (cost < least) {
            least = cost;
            best = kTile256x256 + i;
        }
    }
    return (BlockForm)best;
}

// x16: x is 16-bit rows, to be written as blocks in the call.
inline BlockForm block_form(const BlockCall &c, bool x16, int n_cu) {
    if (x16 && takes_own_rows(c, n_cu)) return kOwnRows;
    if (takes_few_rows(c, n_cu)) return kFewRows;
    return block_tile(c, n_cu);
}

}  // namespace exl3
