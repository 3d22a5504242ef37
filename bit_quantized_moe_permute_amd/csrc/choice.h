// Which kernel a call of the grouped products takes, by its counts and sizes alone. Host code without HIP: the test compiles it
// by itself.
#pragma once
#include <cstdint>

namespace moe {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The positions of a call: groups that can have any, and their mean.
struct Load {
    int64_t used, rows, mean;
    Load(int n_groups, int n_rows) : used(n_groups < n_rows ? n_groups : n_rows), rows(n_rows), mean(ceil_div(n_rows, used)) {}
    // Tiles of up to `height` positions to expect: those of one group; of several, which share the positions unevenly, half a tile
    // to each above whole ones, and one to each at least.
    int64_t tiles(int height) const {
        if (used == 1) return ceil_div(rows, height);
        const int64_t t = rows / height + used / 2;
        return t > used ? t : used;
    }
};

// ---------------------------------------------------------------------------
// moe_q4_linear (q4.h): k_few with 16 weight rows to a workgroup, or k_many with 128 (SwiGLU: 64 of each half) and tiles of 16, 32
// or 64 positions, along all of K or in two halves of it. Calls in us (weights of 4096 columns, one matrix, where nothing else is
// said), the kernel taken first:
//
//   k_few while k_many's workgroups of 16 positions (w16) would be few: its time grows with w16, faster with more rows to a tile,
//     where the other's stands still up to 256. Up to 160 with 4 rows at most: 1 row of 20480 rows of weights (160) 16.6 (halves of
//     16: 18.4), of 24576 (192) 18.4 (few: 19.0), 4 of 20480 19.1 (19.2). Up to 128 with 8: 8 of 16384 (128) 18.4 (19.0), of 24576
//     (192) 19.2 (26.2). Up to 96 with more: 16 of 12288 (96) 18.4 (19.3), 24 of 6144 (96) 18.3 (19.1), 16 of 16384 (128) 19.2
//     (23.5), 64 of 8192 (256) 19.3 (44.3), 256 of 2048 (256) 19.8 (44.3); 16384 columns: 32 of 4096 (64) 44.5 (58), 64 (128) 58
//     (86). Up to 128 where K is too short for halves: 1280 columns 64 of 4096 (128) 8.8 (10.3), 1024 columns 64 of 4096 9.2 (9.2),
//     128 (256) 9.4 (16.4)
//   tiles of 16 while these fit one round of the chip's 256 units, in two halves of K from 16 chunks of 128 columns on: 64 of 8192
//     19.3 (whole: 21.8), 2048 columns 64 of 4096 12.3 (12.9); below them the second half has little or nothing: 1024 columns 128
//     of 4096 whole 9.4 (halves: 11.1), 16384 rows of weights and 24 9.3 (11.0)
//   beyond, up to 512 workgroups of tiles of 64 (w64):
//     tiles of 64 in halves where the groups have 32 rows at most and one round holds them: 24 of 24576 24.9 (16: 29.5, 32: 30.6),
//       24 of 32768 25.5 (16: 29.9)
//     tiles of 16 up to two rounds: 128 of 8192 29.7 (32: 30.2, halves of 64: 36.5), 48 of 16384 29.5 (30.2, 35.6)
//     tiles of 64 in halves in one round: 1024 of 2048 37.7 (32: 42.4, 16: 53.4), 64 of 24576 37.1 (41.8, 40.5)
//     else tiles of 32: 128 of 24576 58.6 (64: 63.2, in halves 71.3, 16: 75.2), 512 tokens of 2 among 8 experts of 2048 rows 56.3
//       (64.4, 73.6, 64.1); 1024 columns 128 of 16384 16.3 (17.4, 19.2, 20.2)
//   from 512 on by the mean of the groups, along all of K (halves: 3 tokens of 8 among 256 experts, 768 workgroups, 58.7 against
//     47.5). Tiles of 16 or 32 leave three waves to a SIMD registers, tiles of 64 two, but they read a group's weights once (the
//     others' second reading comes out of caches). 256 experts of 4096 x 2048, a token's 8 spread unevenly, tiles of 16, 32, 64: mean
//     4 260, 268, 309; 8 327, 319, 398; 16 453, 401, 475; 31 693, 566, 614; 62 1177, 903, 863. One group has just its rows: 16 of
//     65536 rows of weights 38.6 (64: 38.9), 17 44.3 (16: 57.5, 32: 46.1).
// ---------------------------------------------------------------------------
enum Q4Kernel { Q4_FEW, Q4_16_HALVES, Q4_16, Q4_32, Q4_64_HALVES, Q4_64 };

inline Q4Kernel q4_choice(bool swiglu, int n_groups, int n_rows, int N, int K) {
    const Load l(n_groups, n_rows);
    const int64_t tiles_n = ceil_div(N, swiglu ? 64 : 128), w16 = l.tiles(16) * tiles_n, w64 = l.tiles(64) * tiles_n;
    const bool one = l.used == 1, halves = K >= 16 * 128;
    if (w16 <= (l.mean <= 4 ? 160 : l.mean <= 8 || !halves ? 128 : 96)) return Q4_FEW;
    if (w16 <= 256) return halves ? Q4_16_HALVES : Q4_16;
    if (w64 < 512) {
        if (halves && w64 <= 256 && (one ? l.mean : 2 * l.mean) <= 32) return Q4_64_HALVES;
        if (w16 <= 512) return Q4_16;
        return halves && w64 <= 256 ? Q4_64_HALVES : Q4_32;
    }
    if (l.mean < (one ? 17 : 8)) return Q4_16;
    return !one && l.mean <= 32 ? Q4_32 : Q4_64;
}

// ---------------------------------------------------------------------------
// moe_grouped_linear and moe_grouped_dgrad (grouped.hip). Calls in us, the kernel taken first, one matrix of 4096 x 4096 or weights of
// 4096 columns where nothing else is said.
//
//   k_few_rows (16 weight rows to a workgroup, forward only) while its workgroups are few: its time grows with them, where the tiles'
//     stands still until these fill the chip.
//     Below 2048 workgroups for up to 4 rows of one matrix, which are read from the caches all along: 1 row, 16384 rows of weights
//       (1024) 31.5 (tiles: 37), 24576 (1536) 37 (44), 4 rows of 16384 33 (37)
//     Below 1024 for up to 16 rows: 1 row 7.6 (26), 16 rows 9.7 (26), 12288 rows of weights (768) 19 (32), 16 of these 27 (32), 1024 x
//       1024 and one token of 4 among 64 experts 4.4 (9.6). There tiles: 16 rows of 16384 (1024) 38 (few: 41), 16 tokens of 2 among 16
//       experts of 1024 x 1024 10.3 (11.7)
//     Up to 768 for more: 24 rows (512) 16.5 (26.4), 48 (768) 23.4 (27.1), 64 (1024) 27.1 (few: 30.3), 1024 rows of weights and 192 (768)
//       23.3 (27.1), 256 (1024) 27.1 (30.2), 1024 columns 32 rows (512) 6.6 (9.0), 64 (1024) 9.3 (11.1), 16384 columns 32 (512) 66
//       (116), 64 (1024) 123 (121)
//
//   The tiles, by their numbers t128 of 256 x 128 and t256 of 256 x 256 results (SwiGLU: of both halves) against 256 units; one
//   workgroup of 8 waves fills a unit. What is left of several groups' positions counts as half a tile each.
//     256 x 128 or 256 x 256 of 8 waves, from 128 rows a group and 160 tiles of 256 x 128 on, where the rounds of 256 workgroups are
//       fewer, one of 256 x 128 counted as 0.61 of one of 256 x 256 (63 us; 111 for one, 96 each of two, sums of 4096): forward, one matrix of 4096 x
//       4096, 2048 rows (1 round, 1) 63 (256 x 256: 80), 2560 (2, 1) 87 (256 x 128: 109), 4096 (2, 1) 111 (125), 6144 (3, 2) 190 (192),
//       8192 (4, 2) 224 (255); input's gradient the same to 3%. 2048 tokens of 8 among 32 experts, input's gradient of 4096 -> 2048
//       (9, 5) 321 (342), of 2048 -> 4096 (5, 3) 348 (334), 1024 tokens of that (3, 2) 206 (228). 4096 tokens of 4
//       among 16 experts of 520 x 1000 (2, 1) 32 (37). Less than 160: 1024 rows (128) 43.7 with 128 x 64 (256 x 128: 46); from there:
//       1280 (160) 50 (69).
//     Several groups of 128 to 255 rows have most in one tile of 256: 512 tokens of 8 among 32 experts, input's gradient, 4096 ->
//       2048 139 (256 x 128: 144), 2048 -> 4096 116 (146), 768 of these 157 (170) and 132 (145), forward 144 (153; SwiGLU 280 and 272),
//       4096 tokens of 8 among 256 experts with SwiGLU 1939 (2307; 256 x 128 of 4 waves 2554)
//     256 x 128 of 4 waves, two workgroups to a unit, from 256 tiles on, forward from 48 rows a group: 2048 tokens of 8 among 256
//       experts with SwiGLU 1737 (8 waves 1782, 128 x 64 1910), 1024 of these (32 rows) 1737 with 128 x 64 (256 x 128 1810). The input's
//       gradient from 1 row on if its sum is long: one token's row in each of 32 experts, 4096 -> 2048 99 (128 x 64: 130), 4 tokens of 8
//       among 256, 2048 -> 4096, 91 (100), 128 of 8 among 32 103 (135), 256 experts 797 (838); sums of 512: 16 tokens of 4 among 64
//       experts of 512 x 1024 10.7 (256 x 128: 12.2), 256 of these 13.8 (14.7)
//     128 x 64 else: 300 x 4 rows of 16 experts 11 (128 x 128 13, 256 x 128 14 to 24)
// ---------------------------------------------------------------------------
inline bool few_rows_choice(bool swiglu, int n_groups, int n_rows, int n_out) {
    const Load l(n_groups, n_rows);
    const int64_t workgroups = l.tiles(16) * ceil_div(n_out, 16) * (swiglu ? 2 : 1);         // (in SwiGLU's each has twice the weights)
    return workgroups < (l.used == 1 && l.mean <= 4 ? 2048 : l.mean <= 16 ? 1024 : 769);
}

enum GroupedKernel { TILE_128_64, TILE_256_128_4, TILE_256_128_8, TILE_256_256, FEW_ROWS };

// dgrad: the input's gradient
inline GroupedKernel grouped_choice(bool dgrad, bool swiglu, int n_groups, int n_rows, int n_out, int n_in) {
    const Load l(n_groups, n_rows);
    const int64_t tiles_p = ceil_div(dgrad ? n_in : swiglu ? 2 * n_out : n_out, 256);
    const int64_t t128 = l.tiles(128) * tiles_p, t256 = l.tiles(256) * tiles_p;
    if (l.mean >= 128 && t128 >= 160) {
        if (l.used > 1 && l.mean < 256) return TILE_256_256;
        return 61 * ceil_div(t128, 256) < 100 * ceil_div(t256, 256) ? TILE_256_128_8 : TILE_256_256;
    }
    if (t128 >= 256 && (l.mean >= 48 || (dgrad && n_out >= 1024))) return TILE_256_128_4;
    return !dgrad && few_rows_choice(swiglu, n_groups, n_rows, n_out) ? FEW_ROWS : TILE_128_64;
}

// ---------------------------------------------------------------------------
// moe_grouped_wgrad: tiles of 256 x 256 of 8 waves from half of the chip's units on, 128 x 128 of 8 waves where these would be fewer.
// Calls in us, fp32 results, by the number of 256 x 256: 64, one matrix of 2048 x 2048, 512 rows 11.1 (256 x 256: 20.2), 8192 92 (179);
// 128, 2048 x 4096, 64 rows 10.8 (11.7), 512 20.7 (21.7), 2048 54.3 (54.1), 8192 195 (191); 160, 4096 x 2560, 64 rows 12.7 (128 x 128:
// 14.5), 8192 189 (258); 196, 3584 x 3584, 512 rows 25 (35), 8192 218 (336); 256, 4096 x 4096, 8192 rows 248 (395); 192, 12 experts of
// 1024 x 1024, 64 rows of 2 14.1 (16.5), 8192 43.5 (57.4); 300 x 2, 300 experts of 264 x 136 24.5 to 31.7 either way. (Of 32 experts of
// 4096 x 4096, 2048 tokens of 8, 256 x 256 939, 256 x 128 two workgroups to a unit 961; 8192 rows of one matrix 240 and 279.)
// ---------------------------------------------------------------------------
inline bool wgrad_256(int n_groups, int n_out, int n_in) { return ceil_div(n_out, 256) * ceil_div(n_in, 256) * n_groups > 128; }

}  // namespace moe
