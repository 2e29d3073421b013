// Walk over the tiles of ragged experts: experts in order, then tiles of rows,
// then tiles of columns.  For kernels whose tile height is kTileM for every expert.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ep_device.cuh"

namespace ep {

constexpr int kRowGroups = 8192 / kWarp;  // most groups of 32 experts

struct RowTile {
    int e, m0, col, rows;  // expert, first row, tile of columns, valid rows of the expert from m0 on
};

// `first` (shared memory, kRowGroups + 2 words) holds the tiles before each group of 32 experts; a walk goes on from the
// expert of its last tile.
template <int kTileM>
struct RowTiles {
    const int32_t* count;
    const int* first;
    int E, cap, tiles_n;
    int e = 0, before = 0;  // an expert, and the tiles before it

    __device__ __forceinline__ int rows_of(int i) const { return min(max(__ldg(count + i), 0), cap); }
    __device__ __forceinline__ int tiles_of(int i) const { return (rows_of(i) + kTileM - 1) / kTileM * tiles_n; }

    __device__ __forceinline__ int total() const { return first[(E + kWarp - 1) / kWarp]; }

    // Fills `to` (one warp).
    __device__ __forceinline__ void fill(int* to, int lane) const {
        const int groups = (E + kWarp - 1) / kWarp;
        int base = 0;
        for (int i = 0; i < groups; ++i) {
            if (lane == 0) to[i] = base;
            const int at = i * kWarp + lane;
            base += static_cast<int>(__reduce_add_sync(0xffffffffu, at < E ? tiles_of(at) : 0));
        }
        if (lane == 0) to[groups] = base;
    }

    // Tile t, which is below total() and not before the last one asked for.
    __device__ __forceinline__ RowTile at(int t) {
        if (first[e / kWarp + 1] <= t) {
            int group = e / kWarp + 1;
            while (first[group + 1] <= t) ++group;
            e = group * kWarp;
            before = first[group];
        }
        int rows, n;
        for (;;) {
            rows = rows_of(e);
            n = (rows + kTileM - 1) / kTileM * tiles_n;
            if (before + n > t) break;
            before += n;
            ++e;
        }
        const int local = t - before, m0 = local / tiles_n * kTileM;
        return RowTile{e, m0, local % tiles_n, rows - m0};
    }
};

}  // namespace ep
