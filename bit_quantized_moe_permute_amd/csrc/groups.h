// Device-side reading of a group description (moe_group_desc): rows grouped by expert.
#pragma once
#include "common.h"
#include "internal.h"

namespace moe {

// First position of group g, or the end of the last group: whatever the offsets hold, in 0 .. rows.
__device__ __forceinline__ int group_edge(const Groups &g, int i) {
    if (!g.offsets) return i ? g.rows : 0;
    return min(max(g.offsets[i], 0), g.rows);
}

// Row of the input that position p reads, -1 for none.
__device__ __forceinline__ int in_row(const Groups &g, int p, int n_rows) {
    int r = p;
    if (g.in_index) {
        r = g.in_index[p];
        if (r >= 0 && g.in_div > 1) r = (int)((uint32_t)r / (uint32_t)g.in_div);
    }
    return (unsigned)r < (unsigned)n_rows ? r : -1;
}
// Row of the output that position p writes (of dy that it reads), -1 for none.
__device__ __forceinline__ int out_row(const Groups &g, int p, int n_rows) {
    const int r = g.out_index ? g.out_index[p] : p;
    return (unsigned)r < (unsigned)n_rows ? r : -1;
}
// Row of the input's gradient that position p writes, -1 for none.
__device__ __forceinline__ int in_slot(const Groups &g, int p, int n_rows) {
    const int r = g.in_index ? g.in_index[p] : p;
    return (unsigned)r < (unsigned)n_rows ? r : -1;
}

// The positions of a tile: group, first position, end of the tile.
struct Tile {
    int group, begin, end;
};

// Tile number `item` when every group is cut into tiles of up to `height` positions, groups in order; false behind the last.
// Every wave of a workgroup finds it for itself: a lane sums the tiles of a run of groups, a scan over the lanes finds the
// lane whose run holds the item.
__device__ __forceinline__ bool find_tile(const Groups &g, int height, int item, Tile &t) {
    if (!g.offsets) {
        t.group = 0;
        t.begin = item * height;
        t.end = min(t.begin + height, g.rows);
        return t.begin < g.rows;
    }
    const int lane = threadIdx.x & 63, per = (g.n + 63) / 64, g0 = min(lane * per, g.n), g1 = min(g0 + per, g.n);
    int sum = 0, b = group_edge(g, g0);
    for (int i = g0; i < g1; ++i) {
        const int e = group_edge(g, i + 1);
        if (e > b) sum += (e - b + height - 1) / height;
        b = e;
    }
    int upto = sum;
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(upto, o, 64);
        if (lane >= o) upto += v;
    }
    const unsigned long long here = __ballot(item >= upto - sum && item < upto);
    if (!here) return false;
    int left = item - (upto - sum), found[3] = {0, 0, 0};
    b = group_edge(g, g0);
    for (int i = g0; i < g1; ++i) {
        const int e = group_edge(g, i + 1), n = e > b ? (e - b + height - 1) / height : 0;
        if (left >= 0 && left < n) {
            found[0] = i;
            found[1] = b + left * height;
            found[2] = min(found[1] + height, e);
        }
        left -= n;
        b = e;
    }
    const int who = __ffsll(here) - 1;
    t.group = __builtin_amdgcn_readlane(found[0], who);
    t.begin = __builtin_amdgcn_readlane(found[1], who);
    t.end = __builtin_amdgcn_readlane(found[2], who);
    return true;
}

// Tiles that find_tile can have at most: whole ones, and one more for each group with rows.
inline int64_t most_tiles(const Groups &g, int height) {
    return g.offsets ? (int64_t)g.rows / height + (g.n < g.rows ? g.n : g.rows) : ((int64_t)g.rows + height - 1) / height;
}

__device__ __forceinline__ float swiglu(float gate, float up) { return gate / (1.0f + expf(-gate)) * up; }

}  // namespace moe
