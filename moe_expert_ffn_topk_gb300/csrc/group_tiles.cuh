// Tiles of a product whose rows fall into groups, each with its own weights (the offsets of moe_plan or moe_permute): a table in shared
// memory that every role of a kernel finds its tiles in.
#pragma once

#include <stdint.h>

namespace moe {

// tab: tile_off [groups + 1] (the row tiles of the groups before), lo [groups], hi [groups] (the groups' rows). One warp writes it, one
// scan per 32 groups. Offsets are taken into [0, M], and one below an earlier one as that one: the groups' rows never overlap.
// Without offsets there is one group of all rows.
__device__ __forceinline__ void write_group_tiles(const int32_t* offsets, int M, int groups, int tile_rows, int* tab, int lane) {
    int *lo = tab + groups + 1, *hi = lo + groups, carry = 0;
    int last = offsets ? min(max(__ldg(offsets), 0), M) : 0;  // where the groups so far end
    for (int b = 0; b < groups; b += 32) {
        const int g = b + lane;
        int h = M;
        if (offsets) h = g < groups ? min(max(__ldg(offsets + g + 1), 0), M) : 0;
        if (lane == 0) h = max(h, last);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, h, o);
            if (lane >= o) h = max(h, u);
        }
        const int before = __shfl_up_sync(0xffffffffu, h, 1);
        const int l = lane == 0 ? last : before;
        last = __shfl_sync(0xffffffffu, h, 31);
        int v = 0;
        if (g < groups) {
            lo[g] = l;
            hi[g] = h;
            v = h > l ? (h - l - 1) / tile_rows + 1 : 0;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (g < groups) tab[g + 1] = carry + v;
        carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) tab[0] = 0;
}

struct GroupTile {
    int g, n_tile, row0, hi;  // column tile n_tile of group g; rows [row0, hi)
};

// Tile t of (row tiles) x (n_tiles column tiles): group by group, column tile by column tile, row tile by row tile. (A division in 32 bits
// where the numbers fit gained nothing on either product.)
__device__ __forceinline__ GroupTile find_group_tile(int64_t t, const int* tab, int groups, int n_tiles, int tile_rows) {
    const int *off = tab, *lo = tab + groups + 1, *hi = lo + groups;
    int a = 0, b = groups - 1;
    while (a < b) {
        const int mid = (a + b + 1) >> 1;
        if ((int64_t)off[mid] * n_tiles <= t) a = mid; else b = mid - 1;
    }
    const int mt = off[a + 1] - off[a];
    const int64_t local = t - (int64_t)off[a] * n_tiles;
    GroupTile tl;
    tl.g = a;
    tl.n_tile = (int)(local / mt);
    tl.row0 = lo[a] + (int)(local % mt) * tile_rows;
    tl.hi = hi[a];
    return tl;
}

}  // namespace moe
