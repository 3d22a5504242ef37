// Which kernel a call of the grouped products takes, by its counts and sizes alone. Host code without HIP: the test compiles it
// by itself.
//
// The rules were made from the times of every kernel at some 2000 calls: the shapes given below, and random ones over the whole range
// (1 to 256 groups, 1 to 32768 rows, 32 to 32768 weight rows, 64 to 16384 columns, even and uneven groups). At 690 other random calls
// the kernel taken needs on average 3.5% (4-bit), 1.5% (forward), 1.8% (input's gradient) and 0.2% (weights' gradient) more than the
// fastest, at 3% of them more than a fifth, at none more than 1.4 times as much. Times are whole calls in us on one MI355X.
#pragma once
#include <algorithm>
#include <cmath>
#include <cstdint>

namespace moe {

constexpr int64_t UNITS = 256;                               // of the chip: a round of workgroups that fill a unit each

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The positions of a call: groups that have some, where positions fall on them at random (64 positions leave 23 of 64 groups without),
// and their mean.
struct Load {
    int64_t used, rows, mean;
    Load(int n_groups, int n_rows)
        : used((int64_t)std::ceil(-n_groups * std::expm1(-(double)n_rows / n_groups))), rows(n_rows), mean(ceil_div(n_rows, used)) {}
    // Tiles of up to `height` positions to expect: those of one group; of several, which share the positions unevenly, half a tile
    // to each above whole ones, and one to each at least.
    int64_t tiles(int height) const { return used == 1 ? ceil_div(rows, height) : std::max(rows / height + used / 2, used); }
};

// ---------------------------------------------------------------------------
// moe_q4_linear (q4.h): k_few with 16 weight rows to a workgroup, or k_many with 128 (SwiGLU: 64 of each half) and tiles of 16, 32
// or 64 positions, along all of K or in two halves of it. w16 and w64 are k_many's workgroups with tiles of 16 and 64.
//
// k_few's time grows with its workgroups, k_many's stands still up to one round; where the two meet depends on K and on the rows of
// a tile. So their times are estimated, by the chunks of 128 columns (k_few takes 16 at a time, a half of k_many 8), fitted to the calls
// above; 9 of 10 lie within a quarter. One matrix, the kernel taken first:
//   4096 columns: 1 row of 20480 rows of weights, few 16.6 (halves of 16: 18.4), of 32768 18.7 (few: 24.8); 8 of 16384 18.4 (19.0), of
//     24576 19.2 (26.2); 16 of 12288 18.4 (19.3), of 16384 19.2 (23.5); 64 of 2048 12.7 (18.9), of 8192 19.3 (44.3); 256 of 2048 19.8 (44)
//   16384 columns: 32 of 4096 44.5 (58), 64 58 (86); 2432 columns, 238 of 872 13.1 (18.1); 1280, 64 of 4096 8.8 (10.3); 1024, 128 of 4096
//     9.4 (16.4); 352, 863 of 300 5.2 (8.9)
//   halves of K or all of it, tiles of 16: 64 of 8192 19.3 (whole: 21.8), 64 of 4096 and 1920 columns 14.6 (16.1); whole: 128 of 4096
//     and 1024 columns 9.4 (halves: 11.1), 1536 11.4 (11.9)
// More than one round of tiles of 16, up to 512 workgroups of tiles of 64:
//   tiles of 64 in halves where the groups have 32 rows at most and one round holds them: 24 of 24576 24.9 (16: 29.5, 32: 30.6)
//   tiles of 16 up to two rounds: 128 of 8192 29.7 (32: 30.2, halves of 64: 36.5), 48 of 16384 29.5 (30.2, 35.6)
//   tiles of 64 in halves in one round: 1024 of 2048 37.7 (32: 42.4, 16: 53.4), 64 of 24576 37.1 (41.8, 40.5)
//   else tiles of 32: 128 of 24576 58.6 (64: 63.2, in halves 71.3, 16: 75.2), 512 tokens of 2 among 8 experts of 2048 rows 56.3 (64.4,
//     73.6, 64.1); 1024 columns 128 of 16384 16.3 (17.4, 19.2, 20.2)
// From there on by the mean of the groups, along all of K (halves: 3 tokens of 8 among 256 experts, 768 workgroups, 58.7 against 47.5).
//   Tiles of 16 or 32 leave three waves to a SIMD registers, tiles of 64 two, but they read a group's weights once (the others'
//   second reading comes out of caches). 256 experts of 4096 x 2048, a token's 8 spread unevenly, tiles of 16, 32, 64: mean 4 260, 268,
//   309; 8 327, 319, 398; 16 453, 401, 475; 31 693, 566, 614; 62 1177, 903, 863. One group has just its rows: 16 of 65536 rows of weights
//   38.6 (64: 38.9), 17 44.3 (16: 57.5, 32: 46.1).
// ---------------------------------------------------------------------------
enum Q4Kernel { Q4_FEW, Q4_16_HALVES, Q4_16, Q4_32, Q4_64_HALVES, Q4_64 };

// group: columns to a scale
inline Q4Kernel q4_choice(bool swiglu, int n_groups, int n_rows, int N, int K, int group) {
    const Load l(n_groups, n_rows);
    const int64_t tiles16 = l.tiles(16), tiles_n = ceil_div(N, swiglu ? 64 : 128), w16 = tiles16 * tiles_n, w64 = l.tiles(64) * tiles_n;
    const int64_t chunks = ceil_div(K, 128), serial = std::min(chunks, 8 * ceil_div(chunks, 16));        // those that a half takes one by one
    const double step = group == 32 ? 1.36 : 1;              // (four scales to a chunk)
    const double few = 1.8 + 0.5 * ceil_div(chunks, 16) + std::max(tiles16 * ceil_div(N, 16) / 512., 0.4) *
                       (1.2 + chunks * (0.146 + 0.0055 * std::min<int64_t>(l.mean, 16)) * (swiglu ? 1.86 : 1));
    const double halves = 5.9 + 0.78 * step * serial, whole = 5.1 + 0.55 * step * chunks;
    const bool one = l.used == 1, long_k = chunks > 12;
    if (w16 <= UNITS) return few < std::min(halves, whole) ? Q4_FEW : halves < whole ? Q4_16_HALVES : Q4_16;
    if (w64 < 2 * UNITS) {
        if (few < whole + 0.36 * chunks * (w16 - UNITS) / UNITS) return Q4_FEW;
        if (long_k && w64 <= UNITS && (one ? l.mean : 2 * l.mean) <= 32) return Q4_64_HALVES;
        if (w16 <= 2 * UNITS) return Q4_16;
        return long_k && w64 <= UNITS ? Q4_64_HALVES : Q4_32;
    }
    if (l.mean < (one ? 17 : 8)) return Q4_16;
    return !one && l.mean <= 32 ? Q4_32 : Q4_64;
}

// ---------------------------------------------------------------------------
// moe_grouped_linear and moe_grouped_dgrad (grouped.hip). One matrix of 4096 x 4096, or weights of 4096 columns, where nothing else is
// said; the kernel taken first.
//
// k_few_rows (16 weight rows to a workgroup, forward only) while its workgroups are few (SwiGLU's count twice): its time grows with them,
// where that of the tiles stands still until these fill the chip.
//   below 2048 for up to 4 rows of one matrix, which are read from the caches all along: 1 row, 16384 rows of weights (1024) 31.5
//     (tiles: 37), 24576 (1536) 37 (44), 4 rows of 16384 33 (37)
//   below 1024 for up to 16 rows of one: 1 row 7.6 (26), 16 9.7 (26), 16 rows, 12288 of weights (768) 27 (32), 16384 (1024) 38 (few: 41)
//   below 896 for more, or of several: 24 rows (512) 16.5 (26.4), 48 (768) 23.4 (27.1), 64 (1024) 27.1 (few: 30.3); 192 rows, 1024 of
//     weights (768) 23.3 (27.1); 16384 columns 32 rows (512) 66 (116), 64 (1024) 123 (121); 13552 columns 242 rows, 424 of weights (432)
//     63 (82); one token of 4 among 64 experts of 1024 x 1024 4.4 (9.6), 4 tokens of 2 among 8 of 2048 rows (768) 18 (27.5), 16 of 2 among
//     16 of 1024 x 1024 (896) 10.3 (11.7)
//
// The tiles, by the numbers t128 of 256 x 128 and t256 of 256 x 256 results (SwiGLU: of both halves); one workgroup of 8 waves fills a unit.
//   8 waves, from 112 rows a group, 152 tiles of 256 x 128 and sums of more than 320 on: 1024 rows (128) 43.7 with 128 x 64 (256 x 128:
//   46), 1280 (160) 50 (69). Short sums are better off with two workgroups to a unit: 4096 tokens of 8 among 32 experts, 256 -> 4096 140
//   (256 x 256: 150), of 512 210 (210).
//     One matrix, and 256 rows and more: where the rounds are fewer, one of 256 x 128 counted as 0.61 of one of 256 x 256 (63; 111 for one,
//       96 each of two). 2048 rows (1 round, 1) 63 (256 x 256: 80), 2560 (2, 1) 87 (256 x 128: 109), 4096 (2, 1) 111 (125), 6144 (3, 2) 190
//       (192), 8192 (4, 2) 224 (255); input's gradient the same to 3%, 2048 tokens of 8 among 32 experts, 4096 -> 2048 (9, 5) 321 (342), 1024
//       tokens, 2048 -> 4096 (3, 2) 206 (228)
//     Several groups of 112 to 255 rows have most in one tile of 256: 512 tokens of 8 among 32 experts, input's gradient, 4096 -> 2048 139
//       (256 x 128: 144), 2048 -> 4096 116 (146), forward 144 (153; SwiGLU 280 and 272), 4096 tokens of 8 among 256 experts with SwiGLU
//       1939 (2307; 4 waves 2554). 256 x 128 where one round (by the estimate, a little more) holds all: 640 tokens of 8 among 32 experts,
//       1024 -> 1024 (224) 21.8 (256 x 256: 26.1, 128 x 64: 25.8), 2645 tokens among 12, input's gradient, 2480 -> 1184 (260) 30 (41)
//   4 waves, 256 x 128, two workgroups to a unit, from 48 rows and 256 tiles on: 2048 tokens of 8 among 256 experts with SwiGLU 1737 (8 waves
//   1782, 128 x 64 1910), 1024 of these (32 rows) 1737 with 128 x 64 (256 x 128 1810). The input's gradient of any number of rows from
//   200 tiles on, with sums of 1024 and more and no half tile of 256 left empty among fewer than 8: 4 tokens of 8 among 256, 2048 -> 4096
//   (248) 91 (128 x 64: 100), 32 of 8 among 32, 4096 -> 2048 (336) 99 (130), 128 (512) 103 (135), 256 experts 797 (838); 128 x 64: 2 tokens of
//   8 among 256 (128) 53 (72), 58 of 2 among 25, 1728 -> 2112 (175) 23.5 (37), 1547 of 4 among 220, 632 -> 4056 249 (284), sums of 512: 16 tokens
//   of 4 among 64 experts of 512 x 1024 10.7 (12.2)
//   128 x 64 else: 300 x 4 rows of 16 experts 11 (128 x 128 13, 256 x 128 14 to 24)
// ---------------------------------------------------------------------------
enum GroupedKernel { TILE_128_64, TILE_256_128_4, TILE_256_128_8, TILE_256_256, FEW_ROWS };

// dgrad: the input's gradient
inline GroupedKernel grouped_choice(bool dgrad, bool swiglu, int n_groups, int n_rows, int n_out, int n_in) {
    const Load l(n_groups, n_rows);
    const bool one = l.used == 1;
    const int64_t results = dgrad ? n_in : swiglu ? 2 * n_out : n_out, sum = dgrad ? n_out : n_in, tiles_p = ceil_div(results, 256);
    const int64_t t128 = l.tiles(128) * tiles_p, t256 = l.tiles(256) * tiles_p;
    if (l.mean >= 112 && t128 >= 152 && sum > 320) {
        if (!one && l.mean < 256) return t128 <= UNITS + UNITS / 8 ? TILE_256_128_8 : TILE_256_256;
        return 61 * ceil_div(t128, UNITS) < 100 * ceil_div(t256, UNITS) ? TILE_256_128_8 : TILE_256_256;
    }
    if (l.mean >= 48 && t128 >= UNITS) return TILE_256_128_4;
    if (dgrad) return sum >= 1024 && t128 >= 200 && (tiles_p >= 8 || ceil_div(results, 128) == 2 * tiles_p) ? TILE_256_128_4 : TILE_128_64;
    const int64_t few = l.tiles(16) * ceil_div(n_out, 16) * (swiglu ? 2 : 1);
    return few < (one && l.mean <= 4 ? 2048 : one && l.mean <= 16 ? 1024 : 896) ? FEW_ROWS : TILE_128_64;
}

// ---------------------------------------------------------------------------
// moe_grouped_wgrad: tiles of 256 x 256 from half of the chip's units on, 128 x 128 where these would be fewer, both of 8 waves. fp32
// results, by the number of 256 x 256: 64, one matrix of 2048 x 2048, 512 rows 11.1 (256 x 256: 20.2), 8192 92 (179); 128, 2048 x 4096, 64
// rows 10.8 (11.7), 2048 54.3 (54.1), 8192 195 (191); 160, 4096 x 2560, 64 rows 12.7 (128 x 128: 14.5), 8192 189 (258); 196, 3584 x 3584,
// 512 rows 25 (35), 8192 218 (336); 256, 4096 x 4096, 8192 rows 248 (395); 192, 12 experts of 1024 x 1024, 64 rows of 2 14.1 (16.5), 8192
// 43.5 (57.4); 600, 300 experts of 264 x 136 24.5 to 31.7 either way. (32 experts of 4096 x 4096, 2048 tokens of 8, 939; 256 x 128, two
// workgroups to a unit, 961; 8192 rows of one matrix 240 and 279.)
// ---------------------------------------------------------------------------
inline bool wgrad_256(int n_groups, int n_out, int n_in) { return ceil_div(n_out, 256) * ceil_div(n_in, 256) * n_groups > UNITS / 2; }

}  // namespace moe
