// Which rows belong to which group, for the kernels of the experts' products.
// The offsets live on the device, so every block builds the table of the
// groups' tiles for itself, in shared memory.
//
// These kernels start while the one before them, which may write any of their
// inputs, ends (common.cuh, programmatic dependent launch).  So none of them
// loads by the read-only path, which is for data that nothing writes as long as
// the kernel runs: offsets, rows, weights, scales and zero points come by plain
// loads behind the wait, or by TMA.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

// first: row ranges are [first[g], first[g+1]) cut to what `rows` holds;
// tiles: exclusive prefix of the groups' row tiles.
struct GroupTable {
    int32_t tiles[kProductMaxG + 1];
    int32_t first[kProductMaxG + 1];
    int32_t last[kProductMaxG + 1];
};

// Rows of a group.  Entries outside [0, rows] are cut to it; a group whose
// end lies before its start has none.
__device__ __forceinline__ int2 group_rows(const int32_t* offsets, int g, int rows) {
    if (!offsets) return make_int2(0, rows);
    const int lo = min(max(offsets[g], 0), rows);
    return make_int2(lo, min(max(offsets[g + 1], lo), rows));
}

// By one converged warp; the block synchronises afterwards.
__device__ __forceinline__ void group_table(GroupTable& t, const int32_t* offsets, int G, int rows, int tile_rows) {
    const int lane = threadIdx.x & 31;
    int base = 0;
#pragma unroll 4
    for (int g0 = 0; g0 < G; g0 += 32) {
        const int g = g0 + lane;
        int n = 0;
        if (g < G) {
            const int2 r = group_rows(offsets, g, rows);
            n = (r.y - r.x + tile_rows - 1) / tile_rows;
            t.first[g] = r.x;
            t.last[g] = r.y;
        }
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (g < G) t.tiles[g] = base + inc - n;
        base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) t.tiles[G] = base;
}

}  // namespace moe
