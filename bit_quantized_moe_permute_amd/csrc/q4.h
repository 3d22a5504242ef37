// Products with 4-bit weights and group scales over rows grouped by expert (moe_q4_linear):
//
//   out[o][n] = sum over groups j of scale[n][j] * sum over k in j of (code[n][k] - zero[n][j]) x[r][k]
//
// on the bf16 matrix cores. (Each group length has a source of its own that instantiates what is here.) A code c becomes the bf16
// number 16 + c by two bit operations (c goes into the mantissa behind the exponent of 16), and a product of x with -(16 + zero),
// also exact in bf16, opens each group's sum:
//
//   sum (16 + c) x + sum -(16 + zero) x = sum (c - zero) x
//
// so that no weight is rounded; the group's sum takes its scale in fp32, and sums over groups are fp32. (Taking the zero point from
// the code would cost two conversions to each pair of codes; the product with the offset is one matrix instruction to 16 rows x 32
// columns, on units that have time.)
//
// What bounds it: one to a few rows, the codes' stream and the latency before it (1 token, 4096 x 4096: 5.2 us; 3 tokens of 8 among
// 256 experts, 207 MB: 47 us, 4.4 TB/s); from 16 rows on, the vector instructions that unpack (512 tokens of 8 among 256 experts of
// 4096 x 2048, groups of 32: 401 to 419 us where codes and rows alone take 272: 180 vector instructions, a third of them unpacking,
// to 16 products; three waves to a SIMD instead of two took it there from 475).
//
// The matrix instruction takes 16 weight rows, 16 rows of x and 32 columns: lane l has weight row (x row) l % 16 and columns
// 8 (l / 16) .. + 7. Codes are loaded 16 bytes (32 columns) to a lane, four lanes to a row; a 4 x 4 exchange of dwords among these
// four gives each instruction 32 consecutive columns, so that any group of 32 or more is whole.
#pragma once
#include "choice.h"
#include "groups.h"

using namespace moe;

namespace {

constexpr int CHUNK = 128;                                   // columns of a row that four lanes load at once

// Dword j of lane group q (lanes 16 q .. + 15) to dword q of lane group j.
__device__ __forceinline__ void exchange(uint32_t (&w)[4]) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false), b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false), d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w[0] = c[0];
    w[1] = c[1];
    w[2] = d[0];
    w[3] = d[1];
}

// The constants of unpack() in registers: an instruction takes no two literals.
struct Unpack {
    uint32_t mask, exponent;
    __device__ __forceinline__ Unpack() {
        asm("s_mov_b32 %0, 0x780078" : "=s"(mask));
        asm("v_mov_b32 %0, 0x41804180" : "=v"(exponent));
    }
    // Eight codes as 16 + code, in the order 0 4 1 5 2 6 3 7.
    __device__ __forceinline__ uint4 operator()(uint32_t w) const {
        return make_uint4((w << 3 & mask) | exponent, (w >> 1 & mask) | exponent, (w >> 5 & mask) | exponent,
                          (w >> 9 & mask) | exponent);
    }
};

// Eight values of x in the same order.
__device__ __forceinline__ uint4 reorder(uint4 v) {
    return make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                      __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u));
}

// 16 rows of a matrix, one to each lane l % 16: the first one's address is the same for all lanes, the others' distance from it a
// 32-bit number, so that loads need no address arithmetic in vector registers.
template <int G, int KIND> struct Rows {
    static constexpr int SB = KIND == Q4_F32 ? 4 : 2;
    const uint8_t *codes, *zero;
    const char *scale;
    uint32_t row, lane_codes;                                // this lane's row behind the first; its 16 bytes of a chunk

    // first: row of the stack, n: this lane's row behind it
    __device__ __forceinline__ void set(const Q4Args &a, int64_t first, int n) {
        codes = a.codes + first * (a.K / 2);
        scale = static_cast<const char *>(a.scale) + first * (a.K / G) * SB;
        zero = a.zero ? a.zero + first * (a.K / G) : nullptr;
        row = n;
        lane_codes = n * (uint32_t)(a.K / 2) + 16 * (threadIdx.x >> 4 & 3);
    }
};

// A chunk of 16 rows: codes, and the scales and zero points of its groups, as they are loaded.
template <int G, int KIND> struct Chunk {
    static constexpr int SB = KIND == Q4_F32 ? 4 : 2, NG = CHUNK / G, WORDS = (NG * SB + 3) / 4;
    u32x4_t codes;
    uint32_t scale[WORDS], zero;

    // c: number of the chunk. Where the row ends inside it, what lies behind repeats its last codes and groups (their x is zero).
    __device__ __forceinline__ void load_codes(const Q4Args &a, const Rows<G, KIND> &r, int c) {
        uint32_t at = r.lane_codes;
        if (NG > 1 && a.K / G - c * NG < NG) at -= max(16 * (int)(threadIdx.x >> 4 & 3) - (a.K / 2 - c * (CHUNK / 2) - 16), 0);
        codes = *reinterpret_cast<const u32x4_t *>(r.codes + (int64_t)c * (CHUNK / 2) + at);
    }
    __device__ __forceinline__ void load(const Q4Args &a, const Rows<G, KIND> &r, int c) {
        load_codes(a, r, c);
        const int groups = a.K / G, left = groups - c * NG;
        const char *s = r.scale + (int64_t)c * NG * SB;
        const uint8_t *z = r.zero + (int64_t)c * NG;
        const uint32_t g = r.row * (uint32_t)groups;
        zero = 0x08080808u;
        if (NG == 1 || left >= NG) {                         // at once, from addresses aligned to elements
            if constexpr (NG * SB == 2) scale[0] = *reinterpret_cast<const uint16_t *>(s + g * SB);
            else __builtin_memcpy(scale, __builtin_assume_aligned(s + g * SB, SB), NG * SB);
            if (r.zero) {
                if constexpr (NG == 4) __builtin_memcpy(&zero, z + g, 4);
                else if constexpr (NG == 2) {
                    uint16_t v;
                    __builtin_memcpy(&v, z + g, 2);
                    zero = v;
                } else zero = z[g];
            }
        } else {
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const uint32_t i = g + min(j, left - 1);
                if constexpr (SB == 4) scale[j] = *reinterpret_cast<const uint32_t *>(s + i * SB);
                else scale[j / 2] = (j & 1 ? scale[j / 2] : 0u) | (uint32_t)*reinterpret_cast<const uint16_t *>(s + i * SB) << (16 * (j & 1));
            }
            if (r.zero) {
                zero = 0;
#pragma unroll
                for (int j = 0; j < NG; ++j) zero |= (uint32_t)z[g + min(j, left - 1)] << (8 * j);
            }
        }
    }
    __device__ __forceinline__ float scale_of(int j) const {
        if constexpr (KIND == Q4_F32) return __uint_as_float(scale[j]);
        const uint32_t h = scale[j / 2] >> (16 * (j & 1));
        return KIND == Q4_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h & 0xFFFFu);
    }
    // -(16 + zero point) as a pair of bf16
    __device__ __forceinline__ uint32_t offset_of(int j) const { return (zero >> (8 * j) & 15u) * 0x80008u + 0xC180C180u; }
};

// Scales and zero points of 32 groups of 16 rows: lane l has 8 (l / 16) .. + 7 of row l % 16. Read chunk by chunk, a few bytes of
// sixteen rows at a time, they would come out of the caches as whole lines again and again, since the codes that stream past them
// push them out of the L1.
template <int G, int KIND> struct Block {
    using C = Chunk<G, KIND>;
    static constexpr int SB = C::SB, NG = C::NG, GROUPS = 32, CHUNKS = GROUPS / NG;
    uint32_t scale[2 * SB], zero[2];

    // number b of a row's blocks; what lies behind the row's end is not used
    __device__ __forceinline__ void load(const Q4Args &a, const Rows<G, KIND> &r, int64_t first, int64_t total, int b) {
        const uint32_t at = r.row * (uint32_t)(a.K / G) + 8 * (threadIdx.x >> 4 & 3);
        const char *s = r.scale + (int64_t)b * GROUPS * SB;
        const uint8_t *z = r.zero + (int64_t)b * GROUPS;
        zero[0] = zero[1] = 0x08080808u;
        const int64_t left = total - first - (int64_t)b * GROUPS - at;       // groups from here to the end of the stack
        if (__ballot(left < 8) == 0) {
            __builtin_memcpy(scale, __builtin_assume_aligned(s + at * SB, SB), 8 * SB);
            if (r.zero) __builtin_memcpy(zero, z + at, 8);
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = j < left;
            if constexpr (SB == 4) scale[j] = in ? reinterpret_cast<const uint32_t *>(s)[at + j] : 0u;
            else scale[j / 2] = (j & 1 ? scale[j / 2] : 0u) | (in ? (uint32_t)reinterpret_cast<const uint16_t *>(s)[at + j] : 0u) << (16 * (j & 1));
            if (r.zero && in) zero[j / 4] = (zero[j / 4] & ~(0xFFu << 8 * (j & 3))) | (uint32_t)z[at + j] << (8 * (j & 3));
        }
    }
    // Those of chunk c to all lanes of its rows, u = c % 8 (compile-time).
    __device__ __forceinline__ void to_chunk(C &to, const Q4Args &a, int u, int c) const {
        const int from = 4 * ((c * NG % GROUPS / 8) * 16 + (threadIdx.x & 15));
        auto word = [&](uint32_t v) { return (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v); };
        constexpr int W = C::WORDS;
        if constexpr (NG * SB == 2) to.scale[0] = word(scale[u % 8 / 2]) >> (16 * (u & 1));
        else
#pragma unroll
            for (int j = 0; j < W; ++j) to.scale[j] = word(scale[u * W % (2 * SB) + j]);
        to.zero = a.zero ? word(zero[u * NG / 4 % 2]) >> (8 * (u * NG % 4)) : 0x08080808u;
        const int left = a.K / G - c * NG;
        if (NG > 1 && left < NG) {                           // nothing of the next row
#pragma unroll
            for (int j = 1; j < NG; ++j) {
                if (j < left) continue;
                if constexpr (SB == 4) to.scale[j] = 0;
                else to.scale[j / 2] &= j & 1 ? 0xFFFFu : 0u;
            }
        }
    }
};

__device__ __forceinline__ uint4 splat(uint32_t v) { return make_uint4(v, v, v, v); }

// One chunk's products of R blocks of 16 weight rows with NB blocks of 16 rows of x into acc; x(t, s) is block t's operand of
// columns 32 s .. + 31. (No branch stands between a matrix instruction and the reading of its result: behind a branch around a load
// the compiler has been seen to leave the shorter way too short a wait. Kernels that read their sums behind a loop have a branch
// there; tests/test_matrix_waits.py walks every way of the built code.)
template <int R, int NB, typename C, typename X>
__device__ __forceinline__ void chunk_products(const Unpack &unpack, const C (&p)[R], X x, f32x4_t (&acc)[R][NB]) {
    constexpr int STEPS = 4 / C::NG;                         // instructions per group
    uint32_t w[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int s = 0; s < 4; ++s) w[r][s] = p[r].codes[s];
        exchange(w[r]);
    }
#pragma unroll
    for (int j = 0; j < C::NG; ++j) {
        f32x4_t d[R][NB];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            uint4 y[NB];
#pragma unroll
            for (int t = 0; t < NB; ++t) y[t] = x(t, j * STEPS + s);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint4 off = splat(p[r].offset_of(j)), b = unpack(w[r][j * STEPS + s]);
#pragma unroll
                for (int t = 0; t < NB; ++t) d[r][t] = mfma16(y[t], off, s ? d[r][t] : f32x4_t{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int t = 0; t < NB; ++t) d[r][t] = mfma16(y[t], b, d[r][t]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float sc = p[r].scale_of(j);
#pragma unroll
            for (int t = 0; t < NB; ++t)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[r][t][v] = __fmaf_rn(sc, d[r][t][v], acc[r][t][v]);
        }
    }
}

__device__ __forceinline__ void store(const Q4Args &a, int64_t i, float v) {
    if (a.out_bf16) static_cast<__bf16 *>(a.out)[i] = (__bf16)v;
    else static_cast<float *>(a.out)[i] = v;
}

// ---------------------------------------------------------------------------
// Few weights in all: a workgroup has 16 weight rows (SwiGLU: 16 of gate and the same of up) and up to 16 positions of a group;
// its waves take the row's chunks in turn, FEW_AHEAD of them loaded at once, and their sums meet in LDS. 1 token, 4096 x 4096:
// 5.2 us, the launch and two rounds of dependent loads; 4096 x 8192 8.1.
// ---------------------------------------------------------------------------
constexpr int FEW_WAVES = 8, FEW_AHEAD = 2;

template <int G, int KIND, bool SWIGLU>
__global__ __launch_bounds__(64 * FEW_WAVES, 4) void k_few(Q4Args a, int most, int tiles_n) {
    constexpr int R = SWIGLU ? 2 : 1;
    __shared__ __attribute__((aligned(16))) f32x4_t part[FEW_WAVES][R][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i16 = lane & 15, q = lane >> 4;
    Tile t;
    int n0;
    if (!place(a.g, 16, 16, most, tiles_n, t, n0)) return;
    const int xr = t.begin + i16 < t.end ? in_row(a.g, t.begin + i16, a.x_rows) : -1, x_end = xr < 0 ? 0 : a.K - 8 * q;
    const uint16_t *x = a.x + (int64_t)max(xr, 0) * a.K + 8 * q;
    Rows<G, KIND> rows[R];
#pragma unroll
    for (int r = 0; r < R; ++r) rows[r].set(a, ((int64_t)t.group * R + r) * a.N + n0, min(n0 + i16, a.N - 1) - n0);
    const int chunks = (a.K + CHUNK - 1) / CHUNK;
    const Unpack unpack;
    f32x4_t acc[R][1];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r][0] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int c0 = wave; c0 < chunks; c0 += FEW_AHEAD * FEW_WAVES) {
        Chunk<G, KIND> p[FEW_AHEAD][R];
        uint4 v[FEW_AHEAD][4];
#pragma unroll
        for (int u = 0; u < FEW_AHEAD; ++u) {
            const int c = min(c0 + u * FEW_WAVES, chunks - 1);
#pragma unroll
            for (int r = 0; r < R; ++r) p[u][r].load(a, rows[r], c);
#pragma unroll
            for (int s = 0; s < 4; ++s) v[u][s] = load_or_zeros(x + c * CHUNK + 32 * s, c * CHUNK + 32 * s < x_end);
        }
#pragma unroll
        for (int u = 0; u < FEW_AHEAD; ++u) {
            if (c0 + u * FEW_WAVES >= chunks) break;
            chunk_products<R, 1>(unpack, p[u], [&](int, int s) { return reorder(v[u][s]); }, acc);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) part[wave][r][lane] = acc[r][0];
    __syncthreads();
    // lane l's four values are positions 4 (l / 16) .. + 3 of weight row l % 16
    const float *sums = reinterpret_cast<const float *>(part);
    const int e = threadIdx.x, n = e & 15, pos = e >> 4;
    if (pos >= 16 || t.begin + pos >= t.end || n0 + n >= a.N) return;
    const int row = out_row(a.g, t.begin + pos, a.out_rows);
    if (row < 0) return;
    float y[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        y[r] = 0.f;
#pragma unroll
        for (int w = 0; w < FEW_WAVES; ++w) y[r] += sums[((w * R + r) * 64 + n + 16 * (pos >> 2)) * 4 + (pos & 3)];
    }
    store(a, (int64_t)row * a.N + n0 + n, SWIGLU ? swiglu(y[0], y[R - 1]) : y[0]);
}

// ---------------------------------------------------------------------------
// Many: a wave has two blocks of 16 weight rows (SwiGLU: 16 of gate and the same of up) along all of K, a workgroup four waves,
// and up to 16 MAXB positions of a group, in one, two or four blocks of 16 (NB). Codes go straight to registers, AHEAD chunks ahead,
// scales and zero points a block of 32 groups ahead; the x of a chunk passes through LDS, put into the order of unpack() on its
// way, 16-byte piece i of row r at i ^ r: sixteen rows' reads of one piece column touch every bank once. With KS = 2 a workgroup has
// eight waves, four for each half of K. Tiles of 64 have registers for two waves to a SIMD, the smaller ones for three (two chunks
// ahead instead of four for it where there are two blocks; not with the scales of a block in fp32 and two blocks: 30 to 44 registers
// short). All products of four groups before their scales: no gain.
// ---------------------------------------------------------------------------
constexpr int MANY_WAVES = 4, MANY_ROWS = 32 * MANY_WAVES;

__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <int NB, int AHEAD, int KS, int G, int KIND, bool SWIGLU>
__device__ __forceinline__ void many(const Q4Args &a, const Tile &t, int n0, uint4 *lds) {
    using B = Block<G, KIND>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i16 = lane & 15, q = lane >> 4;
    const int w4 = wave % MANY_WAVES, part = wave / MANY_WAVES;
    uint4 (*tile)[16 * NB][16] = reinterpret_cast<uint4 (*)[16 * NB][16]>(lds + part * (2 * 16 * NB * 16));
    // the chunks of this group of waves: from c_begin on, `rounds` for every group, as far as there are any
    const int chunks = (a.K + CHUNK - 1) / CHUNK, rounds = KS == 1 ? chunks : (chunks + 8 * KS - 1) / (8 * KS) * 8;
    const int c_begin = part * rounds, c_end = min(c_begin + rounds, chunks);
    // this thread's part of x: rows thread / 16 + 16 b, piece thread % 16 of a chunk, of the 256 threads of its group
    const int xi = threadIdx.x & 15, xr = threadIdx.x >> 4 & 15;
    const uint16_t *x[NB];
    int x_end[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int p = t.begin + 16 * b + xr, row = p < t.end ? in_row(a.g, p, a.x_rows) : -1;
        x[b] = a.x + (int64_t)max(row, 0) * a.K + 8 * xi;
        x_end[b] = row < 0 ? 0 : min(a.K, c_end * CHUNK) - 8 * xi;
    }
    Rows<G, KIND> rows[2];
    int64_t first_group[2];
    const int64_t groups = (int64_t)a.g.n * a.N * (SWIGLU ? 2 : 1) * (a.K / G);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int first = min(n0 + w4 * (SWIGLU ? 16 : 32) + (SWIGLU ? 0 : 16 * r), a.N - 1);
        const int64_t row = ((int64_t)t.group * (SWIGLU ? 2 : 1) + (SWIGLU ? r : 0)) * a.N + first;
        rows[r].set(a, row, min(first + i16, a.N - 1) - first);
        first_group[r] = row * (a.K / G);
    }
    const Unpack unpack;
    Chunk<G, KIND> p[AHEAD][2];
    B now[2], next[2];
    uint4 v[2][NB];
    auto load_codes = [&](int u, int c) __attribute__((always_inline)) {     // of chunk c, behind the last one that again
#pragma unroll
        for (int r = 0; r < 2; ++r) p[u][r].load_codes(a, rows[r], min(c, chunks - 1));
    };
    auto load_block = [&](int b) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) next[r].load(a, rows[r], first_group[r], groups, b);
    };
    auto load_x = [&](int u, int c) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < NB; ++b) v[u][b] = load_or_zeros(x[b] + c * CHUNK, c * CHUNK < x_end[b]);
    };
    auto put_x = [&](int u) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < NB; ++b) tile[u][16 * b + xr][xi ^ xr] = reorder(v[u][b]);
    };
    f32x4_t acc[2][NB];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[r][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    load_x(0, c_begin);
    load_x(1, c_begin + 1);
    load_block(c_begin / B::CHUNKS);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) load_codes(u, c_begin + u);
    put_x(0);
    load_x(0, c_begin + 2);
    for (int c0 = c_begin; c0 < c_begin + rounds; c0 += 8) {
        if (c0 == c_begin || c0 % B::CHUNKS == 0) {
#pragma unroll
            for (int r = 0; r < 2; ++r) now[r] = next[r];
            load_block(c0 / B::CHUNKS + 1);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int c = c0 + u;
            if (KS == 1 && c >= chunks) break;
            lds_barrier();                                   // this chunk's x is there, and nobody reads the one before it
            put_x((u + 1) & 1);
            load_x((u + 1) & 1, c + 3);
            if (KS == 1 || c < chunks) {
#pragma unroll
                for (int r = 0; r < 2; ++r) now[r].to_chunk(p[u % AHEAD][r], a, u, c);
                chunk_products<2, NB>(unpack, p[u % AHEAD], [&](int b, int s) { return tile[u & 1][16 * b + i16][(4 * s + q) ^ i16]; }, acc);
            }
            load_codes(u % AHEAD, c + AHEAD);
        }
    }
    if constexpr (KS > 1) {                                  // the groups' sums join the first's, which goes on alone
        static_assert(KS == 2, "");
        f32x4_t *sums = reinterpret_cast<f32x4_t *>(lds);
        __syncthreads();
        if (part) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int b = 0; b < NB; ++b) sums[((r * NB + b) * MANY_WAVES + w4) * 64 + lane] = acc[r][b];
        }
        __syncthreads();
        if (part) return;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[r][b] += sums[((r * NB + b) * MANY_WAVES + w4) * 64 + lane];
    }
    // lane l's four values are positions 4 (l / 16) .. + 3 of weight row l % 16
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int pos = t.begin + 16 * b + 4 * q + j, row = pos < t.end ? out_row(a.g, pos, a.out_rows) : -1;
            if (row < 0) continue;
#pragma unroll
            for (int r = 0; r < (SWIGLU ? 1 : 2); ++r) {
                const int n = n0 + w4 * (SWIGLU ? 16 : 32) + 16 * r + i16;
                if (n < a.N) store(a, (int64_t)row * a.N + n, SWIGLU ? swiglu(acc[0][b][j], acc[1][b][j]) : acc[r][b][j]);
            }
        }
}

template <int MAXB, int KS, int G, int KIND, bool SWIGLU>
__global__ __launch_bounds__(64 * MANY_WAVES * KS, KS == 1 && (MAXB == 1 || (MAXB == 2 && KIND != Q4_F32)) ? 3 : 2) void k_many(Q4Args a, int most, int tiles_n) {
    __shared__ __attribute__((aligned(16))) uint4 lds[KS * 2 * 16 * MAXB * 16];
    Tile t;
    int n0;
    if (!place(a.g, 16 * MAXB, SWIGLU ? MANY_ROWS / 2 : MANY_ROWS, most, tiles_n, t, n0)) return;
    const int blocks = (t.end - t.begin + 15) / 16;
    if constexpr (MAXB == 1) many<1, 4, KS, G, KIND, SWIGLU>(a, t, n0, lds);
    else if (blocks <= 1) many<1, 4, KS, G, KIND, SWIGLU>(a, t, n0, lds);
    else if (MAXB == 2 || blocks == 2) many<2, MAXB == 2 ? 2 : 4, KS, G, KIND, SWIGLU>(a, t, n0, lds);
    else if constexpr (MAXB == 4) many<4, 2, KS, G, KIND, SWIGLU>(a, t, n0, lds);
}

template <int MAXB, int KS, int G, int KIND, bool SWIGLU> hipError_t launch_many(const Q4Args &a, hipStream_t st) {
    constexpr int threads = 64 * MANY_WAVES * KS;
    const int64_t tn = ceil_div(a.N, SWIGLU ? MANY_ROWS / 2 : MANY_ROWS), most = most_tiles(a.g, 16 * MAXB), blocks = (most * tn + 7) / 8 * 8;
    if (!grid_fits(blocks, threads)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_many<MAXB, KS, G, KIND, SWIGLU>), dim3((unsigned)blocks), dim3(threads), 0, st, a, (int)most, (int)tn);
    return hipGetLastError();
}

template <int G, int KIND, bool SWIGLU> hipError_t launch_few(const Q4Args &a, hipStream_t st) {
    const int64_t tn = ceil_div(a.N, 16), most = most_tiles(a.g, 16), blocks = (most * tn + 7) / 8 * 8;
    if (!grid_fits(blocks, 64 * FEW_WAVES)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_few<G, KIND, SWIGLU>), dim3((unsigned)blocks), dim3(64 * FEW_WAVES), 0, st, a, (int)most, (int)tn);
    return hipGetLastError();
}

template <int G, int KIND, bool SWIGLU> hipError_t launch_kind(const Q4Args &a, hipStream_t st) {
    switch (q4_choice(SWIGLU, a.g.n, a.g.rows, a.N, a.K, G)) {
        case Q4_FEW: return launch_few<G, KIND, SWIGLU>(a, st);
        case Q4_16_HALVES: return launch_many<1, 2, G, KIND, SWIGLU>(a, st);
        case Q4_16: return launch_many<1, 1, G, KIND, SWIGLU>(a, st);
        case Q4_32: return launch_many<2, 1, G, KIND, SWIGLU>(a, st);
        case Q4_64_HALVES: return launch_many<4, 2, G, KIND, SWIGLU>(a, st);
        case Q4_64: break;
    }
    return launch_many<4, 1, G, KIND, SWIGLU>(a, st);
}

template <int G, int KIND> hipError_t launch_act(const Q4Args &a, hipStream_t st) {
    return a.swiglu ? launch_kind<G, KIND, true>(a, st) : launch_kind<G, KIND, false>(a, st);
}

}  // namespace

namespace moe {

template <int G> hipError_t launch_q4_group(const Q4Args &a, hipStream_t st) {
    return a.scale_kind == Q4_F32 ? launch_act<G, Q4_F32>(a, st) : a.scale_kind == Q4_BF16 ? launch_act<G, Q4_BF16>(a, st)
                                                                                           : launch_act<G, Q4_F16>(a, st);
}

}  // namespace moe
