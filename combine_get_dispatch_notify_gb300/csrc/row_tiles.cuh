// Walk over the tiles of ragged experts: experts in order, then tiles of rows,
// then tiles of columns.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ep_device.cuh"

namespace ep {

constexpr int kRowGroups = 8192 / kWarp;  // most groups of 32 experts

struct RowTile {
    int e, m0, col, rows;  // expert, first row, tile of columns, rows
};

// `first` (shared memory, kRowGroups + 2 words) holds the tiles of rows before each group of 32 experts, and last the binary
// logarithm of a tile's rows; a walk goes on from the expert of its last tile.
//
// Tiles have kTileM rows, or half as many where that takes no more rounds of tiles.  With few tiles an expert of many rows is
// what a call waits for, and its halves go to two places: 24 experts by Zipf popularity (220, 126, 112 rows and fewer),
// 1160 / 520, bf16: gradient through the activation 22.6 -> 16.0 us, rows' gradient 19.6 -> 16.3, gated 19.9 -> 15.7, last
// product 12.9 -> 10.8.  16 experts with 200 rows, 2048 / 1024, where it takes more: last product 19.0 -> 24.4, rows' gradient 33 -> 46.
// Two experts with 256 rows, 7168 / 2048: gated 68 -> 59, but gradient through the activation 48 -> 58.
//
// An expert's last tile has the rest of its rows, or (kEven) all of its tiles about as many, in steps of 32.  A last
// tile of a few rows is bound by its weights' bytes and costs half of a whole one; even tiles have more bytes a row all of them.
// 32 experts, 7168 / 2048, about 512 rows each (1024), half of the experts with a few more: gated 586 us evenly, 625 not
// (1153, 1151), but the rows' gradient 665 and 607 (1322, 1184), the last product 320 and 310 (663, 622).
template <int kTileM, bool kEven>
struct RowTiles {
    const int32_t* count;
    const int* first;
    int E, cap;
    int tiles_n = 1;        // tiles of columns
    int e = 0, before = 0;  // an expert, and the tiles of rows before it
    int shift = kWhole;     // binary logarithm of a tile's rows

    static constexpr int kWhole = kTileM == 256 ? 8 : kTileM == 128 ? 7 : 6;
    static_assert(kTileM == 1 << kWhole, "");

    __device__ __forceinline__ int rows_of(int i) const { return min(max(__ldg(count + i), 0), cap); }

    __device__ __forceinline__ int row_tiles() const { return first[(E + kWarp - 1) / kWarp]; }

    __device__ __forceinline__ int tiles_of(int rows) const { return (rows + (1 << shift) - 1) >> shift; }

    // Fills `to` by the columns of blocks and the pairs of CTAs that share the tiles (one warp).
    __device__ __forceinline__ void fill(int* to, int lane, int columns, int pairs) {
        constexpr int kAhead = 8;  // groups whose counts are asked for together
        const int groups = (E + kWarp - 1) / kWarp;
        const auto ask = [&](int i0, int (&rows)[kAhead]) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int at = (i0 + i) * kWarp + lane;
                rows[i] = at < E ? rows_of(at) : 0;
            }
        };
        int rows[kAhead];
        ask(0, rows);
        if (cap > kTileM / 2) {
            int whole = 0, halves = 0;
            for (int i0 = 0;;) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    whole += (rows[i] + kTileM - 1) / kTileM;
                    halves += (rows[i] + kTileM / 2 - 1) / (kTileM / 2);
                }
                if ((i0 += kAhead) >= groups) break;
                ask(i0, rows);
            }
            whole = __reduce_add_sync(0xffffffffu, whole);
            halves = __reduce_add_sync(0xffffffffu, halves);
            // rounds of tiles: of halves no more than of whole ones?
            const unsigned rounds = (static_cast<unsigned>(whole) * columns + pairs - 1) / pairs;
            if (static_cast<unsigned>(halves) * columns <= rounds * pairs) --shift;
            if (groups > kAhead) ask(0, rows);
        }
        int base = 0;
        for (int i0 = 0;;) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (i0 + i >= groups) break;
                if (lane == 0) to[i0 + i] = base;
                base += static_cast<int>(__reduce_add_sync(0xffffffffu, tiles_of(rows[i])));
            }
            if ((i0 += kAhead) >= groups) break;
            ask(i0, rows);
        }
        if (lane == 0) {
            to[groups] = base;
            to[kRowGroups + 1] = shift;
        }
    }
    // Before tiles are asked for, once `first` is filled.
    __device__ __forceinline__ void start() { shift = first[kRowGroups + 1]; }

    // Tile t, which is below row_tiles() * tiles_n and not before the last one asked for.
    __device__ __forceinline__ RowTile at(int t) {
        const int want = t / tiles_n;
        if (first[e / kWarp + 1] <= want) {
            int group = e / kWarp + 1;
            while (first[group + 1] <= want) ++group;
            e = group * kWarp;
            before = first[group];
        }
        int rows, n;
        for (;;) {
            rows = rows_of(e);
            n = tiles_of(rows);
            if (before + n > want) break;
            before += n;
            ++e;
        }
        const int height = kEven ? ((rows + n - 1) / n + 31) / 32 * 32 : 1 << shift, m0 = (want - before) * height;
        return RowTile{e, m0, t - want * tiles_n, min(height, rows - m0)};
    }
};

// Blocks of a tile for products whose tiles may have two blocks of output columns or one: two, which read the rows half
// as often, unless single ones leave a call's last round of tiles so much fuller that an eighth of the rounds is saved
// (few tiles: one row to each of eight experts, 28 blocks of columns, 76 pairs: 3 rounds of single blocks against
// 2 of double ones).
__device__ __forceinline__ int blocks_of_tiles(int row_tiles, int column_blocks, int pairs) {
    const int one = (row_tiles * column_blocks + pairs - 1) / pairs;
    const int two = (row_tiles * ((column_blocks + 1) / 2) + pairs - 1) / pairs;
    return 8 * one <= 7 * 2 * two ? 1 : 2;
}

}  // namespace ep
