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
        if (r >= 0 && g.in_div > 1) r = (int)(__umulhi((uint32_t)r, g.div_mul) >> g.div_shift);
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

// The groups cut into tiles of up to `height` positions, in order. Every wave finds tiles for itself: a lane has the tiles of a
// run of groups, and a scan over the lanes tells whose run holds a tile. Up to 256 groups the edges of a lane's four are loaded
// at once and kept.
struct Tiles {
    int g0, g1, sum, upto, total;        // this lane's groups, their tiles, those up to their end; all tiles, at most `most`
    int edge[5];
};
constexpr int EDGES = 4;
__device__ __forceinline__ int tiles_of(int b, int e, int height) { return e > b ? (e - b + height - 1) / height : 0; }

// most: what most_tiles() says. Offsets that overlap can name more; those behind it are left out.
__device__ __forceinline__ Tiles scan_tiles(const Groups &g, int height, int most) {
    Tiles t;
    if (!g.offsets) {
        t.total = (g.rows + height - 1) / height;
        return t;
    }
    const int lane = threadIdx.x & 63;
    t.sum = 0;
    if (g.n <= 64 * EDGES) {
        t.g0 = lane * EDGES;
#pragma unroll
        for (int i = 0; i <= EDGES; ++i) t.edge[i] = group_edge(g, min(t.g0 + i, g.n));
#pragma unroll
        for (int i = 0; i < EDGES; ++i) t.sum += tiles_of(t.edge[i], t.edge[i + 1], height);
    } else {
        const int per = (g.n + 63) / 64;
        t.g0 = min(lane * per, g.n);
        t.g1 = min(t.g0 + per, g.n);
        int b = group_edge(g, t.g0);
        for (int i = t.g0; i < t.g1; ++i) {
            const int e = group_edge(g, i + 1);
            t.sum += tiles_of(b, e, height);
            b = e;
        }
    }
    t.upto = t.sum;
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(t.upto, o, 64);
        if (lane >= o) t.upto += v;
    }
    t.total = (int)min((uint32_t)__builtin_amdgcn_readlane(t.upto, 63), (uint32_t)most);
    return t;
}

// Tile `item`, 0 <= item < total.
__device__ __forceinline__ Tile tile_at(const Groups &g, const Tiles &t, int height, int item) {
    if (!g.offsets) return Tile{0, item * height, min((item + 1) * height, g.rows)};
    int left = item - (t.upto - t.sum), found[3] = {0, 0, 0};
    const int who = __ffsll(__ballot(left >= 0 && left < t.sum)) - 1;
    auto look = [&](int i, int b, int e) {
        const int n = tiles_of(b, e, height);
        if (left >= 0 && left < n) {
            found[0] = i;
            found[1] = b + left * height;
            found[2] = min(found[1] + height, e);
        }
        left -= n;
    };
    if (g.n <= 64 * EDGES) {
#pragma unroll
        for (int i = 0; i < EDGES; ++i) look(t.g0 + i, t.edge[i], t.edge[i + 1]);
    } else {
        int b = group_edge(g, t.g0);
        for (int i = t.g0; i < t.g1; ++i) {
            const int e = group_edge(g, i + 1);
            look(i, b, e);
            b = e;
        }
    }
    return Tile{__builtin_amdgcn_readlane(found[0], who), __builtin_amdgcn_readlane(found[1], who),
                __builtin_amdgcn_readlane(found[2], who)};
}

// Tiles that there can be at most: whole ones, and one more for each group with rows.
inline int64_t most_tiles(const Groups &g, int height) {
    return g.offsets ? (int64_t)g.rows / height + (g.n < g.rows ? g.n : g.rows) : ((int64_t)g.rows + height - 1) / height;
}

// A workgroup's place: positions of a group, and rows of its matrix from n0 on. XCD-aware order: consecutive workgroups go to
// the eight XCDs in turn; each takes a run of tiles, in blocks of four tiles of positions that read the same weights.
__device__ __forceinline__ bool place(const Groups &g, int height, int rows, int most, int tiles_n, Tile &t, int &n0) {
    const Tiles all = scan_tiles(g, height, most);
    const int total = all.total * tiles_n, per = (total + 7) / 8;
    const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= total) return false;
    const int block = id / (4 * tiles_n), in = id - block * 4 * tiles_n, tiles = min(4, all.total - 4 * block), tn = in / tiles;
    n0 = tn * rows;
    t = tile_at(g, all, height, 4 * block + in - tn * tiles);
    return true;
}

static __device__ const u32x4_t zeros[1] = {};

// 16 bytes at p, or of zeros.
typedef const __attribute__((address_space(1))) u32x4_t *global_u32x4;
__device__ __forceinline__ uint4 load_or_zeros(const uint16_t *p, bool in) {
    const uintptr_t at = in ? reinterpret_cast<uintptr_t>(p) : reinterpret_cast<uintptr_t>(zeros);
    return __builtin_bit_cast(uint4, *reinterpret_cast<global_u32x4>(at));
}

__device__ __forceinline__ f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

// Whether a launch can count its threads (in 32 bits).
inline bool grid_fits(int64_t blocks, int threads) { return blocks * threads < ((int64_t)1 << 32); }

// silu(gate) * up of N values. exp(-gate) as a power of two, times 1 + what the rounding of its exponent lost; the quotient through the
// hardware's reciprocal: some 2 units of the last place, in 12 instructions (library exp and division take 40: for 256 x 256 results
// of a tile a tenth of its whole time). The correction is below 1e-5 where the quotient matters; its bounds keep a gate of 2e7 and
// more, or an infinite one, from making it anything else. Where exp(-gate) passes 2^64, 1 + exp(-gate) is exp(-gate), and what is
// above goes to the other factor as a power of two: the sum would overflow from a gate of -88.7 on and its reciprocal leave the
// normal floats at -87.3, while the product may be any float (from -131 on that factor is below 2^-126, and is 0). A wave goes that way
// only if one of N values of its lanes needs it, the others' bits are the same on either (always: 11709 tokens of 8 among 32 experts 2811
// -> 2830 us, 5374 of 2 among 8 with sums of 368 39.5 -> 41.1).
template <int N> __device__ __forceinline__ void swiglu(const float (&gate)[N], const float (&up)[N], float (&y)[N]) {
#pragma clang fp contract(off)                               // 64 - t is of the rounded t, whose rest is in c
    constexpr float L = 1.44269502f, L_REST = 1.92596299e-8f, LN2 = 0.693147181f;    // log2(e) in two parts
    float t[N], c[N], most = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i] = -gate[i] * L;
        c[i] = __builtin_amdgcn_fmed3f(__fmaf_rn(__fmaf_rn(-gate[i], L_REST, __fmaf_rn(-gate[i], L, -t[i])), LN2, 1.f), 0.99f, 1.01f);
        most = fmaxf(most, t[i]);
    }
    if (__any(most > 64.f)) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float s = __builtin_amdgcn_exp2f(fminf(64.f - t[i], 0.f));
            y[i] = gate[i] * __builtin_amdgcn_rcpf(__fmaf_rn(__builtin_amdgcn_exp2f(fminf(t[i], 64.f)), c[i], 1.f)) * (up[i] * s);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = gate[i] * __builtin_amdgcn_rcpf(__fmaf_rn(__builtin_amdgcn_exp2f(t[i]), c[i], 1.f)) * up[i];
    }
}
__device__ __forceinline__ float swiglu(float gate, float up) {
    const float g[1] = {gate}, u[1] = {up};
    float y[1];
    swiglu<1>(g, u, y);
    return y[0];
}

}  // namespace moe
