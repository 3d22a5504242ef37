// Products with 4-bit weights and group scales over rows grouped by expert (moe_q4_linear):
//
//   out[o][n] = sum over groups j of scale[n][j] * sum over k in j of (code[n][k] - zero[n][j]) x[r][k]
//
// on the bf16 matrix cores. A code c becomes the bf16 number 16 + c by two bit operations (c goes into the mantissa behind the
// exponent of 16), and a product of x with -(16 + zero), also exact in bf16, opens each group's sum:
//
//   sum (16 + c) x + sum -(16 + zero) x = sum (c - zero) x
//
// so that no weight is rounded; the group's sum takes its scale in fp32.
//
// The matrix instruction takes 16 weight rows, 16 rows of x and 32 columns: lane l has weight row (x row) l % 16 and columns
// 8 (l / 16) .. + 7. Codes are loaded 16 bytes (32 columns) to a lane, four lanes to a row; a 4 x 4 exchange of dwords among these
// four gives each instruction 32 consecutive columns, so that any group of 32 or more is whole.
#include "groups.h"

using namespace moe;

namespace {

constexpr int MANY_FROM = 256;
constexpr int CHUNK = 128;                                   // columns of a row that four lanes load at once

__device__ __forceinline__ f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

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

// Scales (of type KIND) and zero points of one row's groups in a chunk, as they are loaded. TAIL: K is no multiple of a chunk;
// groups behind the row's end repeat its last one (their products are zero).
template <int G, int KIND, bool TAIL> struct Params {
    static constexpr int SB = KIND == Q4_F32 ? 4 : 2, NG = CHUNK / G, WORDS = (NG * SB + 3) / 4;
    uint32_t scale[WORDS], zero;

    // i: the chunk's first group (index into scale and zero); left: groups from there to the row's end
    __device__ __forceinline__ void load(const Q4Args &a, int64_t i, int left) {
        const char *from = static_cast<const char *>(a.scale) + i * SB;
        zero = 0x08080808u;
        if constexpr (!TAIL) {                               // at once, from an address aligned to elements
            if constexpr (NG * SB == 2) {
                scale[0] = *reinterpret_cast<const uint16_t *>(from);
            } else {
                __builtin_memcpy(scale, __builtin_assume_aligned(from, SB), NG * SB);
            }
            if (a.zero) {
                if constexpr (NG == 4) __builtin_memcpy(&zero, a.zero + i, 4);
                else if constexpr (NG == 2) {
                    uint16_t z;
                    __builtin_memcpy(&z, a.zero + i, 2);
                    zero = z;
                } else zero = a.zero[i];
            }
        } else {
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const int at = min(j, left - 1);
                if constexpr (SB == 4) scale[j] = reinterpret_cast<const uint32_t *>(from)[at];
                else scale[j / 2] = (j & 1 ? scale[j / 2] : 0u) | (uint32_t)reinterpret_cast<const uint16_t *>(from)[at] << (16 * (j & 1));
            }
            if (a.zero) {
                zero = 0;
#pragma unroll
                for (int j = 0; j < NG; ++j) zero |= (uint32_t)a.zero[i + min(j, left - 1)] << (8 * j);
            }
        }
    }
    __device__ __forceinline__ float scale_of(int j) const {
        if constexpr (KIND == Q4_F32) return __uint_as_float(scale[j]);
        const uint32_t h = scale[j / 2] >> (16 * (j & 1));
        return KIND == Q4_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h & 0xFFFFu);
    }
    // -(16 + zero point) as a pair of bf16
    __device__ __forceinline__ uint32_t offset_of(int j) const {
        const uint32_t z = (zero >> (8 * j) & 15u) << 3;
        return 0xC180C180u | z | z << 16;
    }
};

__device__ __forceinline__ uint4 splat(uint32_t v) { return make_uint4(v, v, v, v); }

// One chunk's products of R blocks of 16 weight rows with NB blocks of 16 rows of x into acc; x(t, s) is block t's operand of
// columns 32 s .. + 31. (No branch may stand between a matrix instruction and the reading of its result: the compiler then loses
// the wait between the two on one of the ways.)
template <int R, int NB, typename P, typename X>
__device__ __forceinline__ void chunk_products(const Unpack &unpack, const u32x4_t (&codes)[R], const P (&p)[R], X x, f32x4_t (&acc)[R][NB]) {
    constexpr int STEPS = 4 / P::NG;                         // instructions per group
    uint32_t w[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int s = 0; s < 4; ++s) w[r][s] = codes[r][s];
        exchange(w[r]);
    }
#pragma unroll
    for (int j = 0; j < P::NG; ++j) {
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

__device__ const u32x4_t zeros[1] = {};

// 16 bytes at p, or of zeros.
typedef const __attribute__((address_space(1))) u32x4_t *global_u32x4;
__device__ __forceinline__ uint4 load_or_zeros(const uint16_t *p, bool in) {
    const uintptr_t at = in ? reinterpret_cast<uintptr_t>(p) : reinterpret_cast<uintptr_t>(zeros);
    return __builtin_bit_cast(uint4, *reinterpret_cast<global_u32x4>(at));
}

__device__ __forceinline__ void store(const Q4Args &a, int64_t i, float v) {
    if (a.out_bf16) static_cast<__bf16 *>(a.out)[i] = (__bf16)v;
    else static_cast<float *>(a.out)[i] = v;
}

// A workgroup's place: positions of a group, and rows of its matrix from n0 on. XCD-aware order: consecutive workgroups go to
// the eight XCDs in turn; each takes a run of tiles, in blocks of four tiles of positions that read the same weights.
__device__ __forceinline__ bool place(const Q4Args &a, int height, int rows, int tiles_n, Tile &t, int &n0) {
    const Tiles all = scan_tiles(a.g, height);
    const int total = all.total * tiles_n, per = (total + 7) / 8;
    const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= total) return false;
    const int block = id / (4 * tiles_n), in = id - block * 4 * tiles_n, tiles = min(4, all.total - 4 * block), tn = in / tiles;
    n0 = tn * rows;
    t = tile_at(a.g, all, height, 4 * block + in - tn * tiles);
    return true;
}

// ---------------------------------------------------------------------------
// Few weights in all: a workgroup has 16 R weight rows (SwiGLU: 16 of gate and the same of up) and up to 16 positions of a group;
// its waves take the row's chunks in turn, FEW_AHEAD of them loaded at once, and their sums meet in LDS.
// ---------------------------------------------------------------------------
constexpr int FEW_WAVES = 8, FEW_AHEAD = 2;

template <int R, int G, int KIND, bool TAIL, bool SWIGLU>
__global__ __launch_bounds__(64 * FEW_WAVES, 4) void k_few(Q4Args a, int tiles_n) {
    static_assert(!SWIGLU || R == 2, "");
    constexpr int ROWS = SWIGLU ? 16 : 16 * R;               // results per position
    __shared__ __attribute__((aligned(16))) f32x4_t part[FEW_WAVES][R][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i16 = lane & 15, q = lane >> 4;
    Tile t;
    int n0;
    if (!place(a, 16, ROWS, tiles_n, t, n0)) return;
    const int xr = t.begin + i16 < t.end ? in_row(a.g, t.begin + i16, a.x_rows) : -1, x_end = xr < 0 ? 0 : a.K;
    const uint16_t *x = a.x + (int64_t)max(xr, 0) * a.K + 8 * q;
    const uint8_t *codes[R];
    int64_t params[R];
    const int groups = a.K / G;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t row = (int64_t)t.group * a.N * (SWIGLU ? 2 : 1) +
                            (SWIGLU ? (int64_t)r * a.N + min(n0 + i16, a.N - 1) : min(n0 + 16 * r + i16, a.N - 1));
        codes[r] = a.codes + row * (a.K / 2);
        params[r] = row * groups;
    }
    const Unpack unpack;
    f32x4_t acc[R][1];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r][0] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int c0 = wave * CHUNK; c0 < a.K; c0 += FEW_AHEAD * FEW_WAVES * CHUNK) {
        u32x4_t w[FEW_AHEAD][R];
        Params<G, KIND, TAIL> p[FEW_AHEAD][R];
        uint4 v[FEW_AHEAD][4];
#pragma unroll
        for (int u = 0; u < FEW_AHEAD; ++u) {
            // a chunk behind the end reads the first one again, and its x is zeros
            const int c = c0 + u * FEW_WAVES * CHUNK, at = c < a.K ? c : 0, end = c < a.K ? x_end : 0;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int col = TAIL ? min(at + 32 * q, a.K - 32) : at + 32 * q;
                w[u][r] = *reinterpret_cast<const u32x4_t *>(codes[r] + col / 2);
                p[u][r].load(a, params[r] + at / G, groups - at / G);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
                v[u][s] = load_or_zeros(x + at + 32 * s, TAIL ? at + 32 * s + 8 * q < end : end > 0);
        }
#pragma unroll
        for (int u = 0; u < FEW_AHEAD; ++u) {
            if (c0 + u * FEW_WAVES * CHUNK >= a.K) break;
            chunk_products<R, 1>(unpack, w[u], p[u], [&](int, int s) { return reorder(v[u][s]); }, acc);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) part[wave][r][lane] = acc[r][0];
    __syncthreads();
    // lane l's four values are positions 4 (l / 16) .. + 3 of weight row l % 16
    const float *sums = reinterpret_cast<const float *>(part);
    for (int e = threadIdx.x; e < 16 * ROWS; e += 64 * FEW_WAVES) {
        const int n = e % ROWS, pos = e / ROWS;
        if (t.begin + pos >= t.end || n0 + n >= a.N) continue;
        const int row = out_row(a.g, t.begin + pos, a.out_rows);
        if (row < 0) continue;
        auto sum = [&](int r) {
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < FEW_WAVES; ++w) y += sums[((w * R + r) * 64 + (n & 15) + 16 * (pos >> 2)) * 4 + (pos & 3)];
            return y;
        };
        store(a, (int64_t)row * a.N + n0 + n, SWIGLU ? swiglu(sum(0), sum(R - 1)) : sum(n >> 4));
    }
}

// ---------------------------------------------------------------------------
// Many: a wave has two blocks of 16 weight rows (SwiGLU: 16 of gate and the same of up) along all of K, a workgroup four waves,
// and up to 64 positions of a group, in one, two or four blocks of 16. Codes and parameters go straight to registers, AHEAD chunks ahead; the x of a chunk
// passes through LDS, put into the order of unpack() on its way, 16-byte piece i of row r at i ^ r: sixteen rows' reads of one
// piece column touch every bank once.
// ---------------------------------------------------------------------------
constexpr int MANY_WAVES = 4, MANY_ROWS = 32 * MANY_WAVES, MANY_BLOCKS = 4;

__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <int NB, int G, int KIND, bool TAIL, bool SWIGLU>
__device__ __forceinline__ void many(const Q4Args &a, const Tile &t, int n0, uint4 (*tile)[16 * MANY_BLOCKS][16]) {
    constexpr int AHEAD = NB == 4 ? 2 : 4;                   // chunks of weights under way
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i16 = lane & 15, q = lane >> 4;
    const int groups = a.K / G, chunks = (a.K + CHUNK - 1) / CHUNK;
    // this thread's part of x: rows threadIdx.x / 16 + 16 b, piece threadIdx.x % 16 of a chunk
    const int xi = threadIdx.x & 15, xr = threadIdx.x >> 4;
    const uint16_t *x[NB];
    int x_end[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int p = t.begin + 16 * b + xr, row = p < t.end ? in_row(a.g, p, a.x_rows) : -1;
        x[b] = a.x + (int64_t)max(row, 0) * a.K + 8 * xi;
        x_end[b] = row < 0 ? 0 : a.K - 8 * xi;
    }
    const uint8_t *codes[2];
    int64_t params[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int n = n0 + wave * (SWIGLU ? 16 : 32) + (SWIGLU ? 0 : 16 * r) + i16;
        const int64_t row = ((int64_t)t.group * (SWIGLU ? 2 : 1) + (SWIGLU ? r : 0)) * a.N + min(n, a.N - 1);
        codes[r] = a.codes + row * (a.K / 2);
        params[r] = row * groups;
    }
    const Unpack unpack;
    u32x4_t w[AHEAD][2];
    Params<G, KIND, TAIL> p[AHEAD][2];
    uint4 v[2][NB];
    auto load_weights = [&](int u, int c) {                  // chunk c (behind the last: that one) into place u
        const int at = min(c, chunks - 1) * CHUNK;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int col = TAIL ? min(at + 32 * q, a.K - 32) : at + 32 * q;
            w[u][r] = *reinterpret_cast<const u32x4_t *>(codes[r] + col / 2);
            p[u][r].load(a, params[r] + at / G, groups - at / G);
        }
    };
    auto load_x = [&](int u, int c) {
#pragma unroll
        for (int b = 0; b < NB; ++b) v[u][b] = load_or_zeros(x[b] + c * CHUNK, c * CHUNK < x_end[b]);
    };
    auto put_x = [&](int u) {
#pragma unroll
        for (int b = 0; b < NB; ++b) tile[u][16 * b + xr][xi ^ xr] = reorder(v[u][b]);
    };
    f32x4_t acc[2][NB];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[r][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    load_x(0, 0);
    load_x(1, 1);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) load_weights(u, u);
    put_x(0);
    load_x(0, 2);
    for (int c0 = 0; c0 < chunks; c0 += AHEAD) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int c = c0 + u;
            if (c >= chunks) break;
            lds_barrier();                                   // this chunk's x is there, and nobody reads the one before it
            put_x((u + 1) & 1);
            load_x((u + 1) & 1, c + 3);
            chunk_products<2, NB>(unpack, w[u], p[u], [&](int b, int s) { return tile[u & 1][16 * b + i16][(4 * s + q) ^ i16]; }, acc);
            load_weights(u, c + AHEAD);
        }
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
                const int n = n0 + wave * (SWIGLU ? 16 : 32) + 16 * r + i16;
                if (n < a.N) store(a, (int64_t)row * a.N + n, SWIGLU ? swiglu(acc[0][b][j], acc[1][b][j]) : acc[r][b][j]);
            }
        }
}

template <int G, int KIND, bool TAIL, bool SWIGLU>
__global__ __launch_bounds__(64 * MANY_WAVES, 2) void k_many(Q4Args a, int tiles_n) {
    __shared__ __attribute__((aligned(16))) uint4 tile[2][16 * MANY_BLOCKS][16];
    Tile t;
    int n0;
    if (!place(a, 16 * MANY_BLOCKS, SWIGLU ? MANY_ROWS / 2 : MANY_ROWS, tiles_n, t, n0)) return;
    const int blocks = (t.end - t.begin + 15) / 16;
    if (blocks <= 1) many<1, G, KIND, TAIL, SWIGLU>(a, t, n0, tile);
    else if (blocks == 2) many<2, G, KIND, TAIL, SWIGLU>(a, t, n0, tile);
    else many<4, G, KIND, TAIL, SWIGLU>(a, t, n0, tile);
}

int64_t tiles(int N, int rows) { return (N + rows - 1) / rows; }

template <int G, int KIND, bool TAIL, bool SWIGLU> hipError_t launch_many(const Q4Args &a, hipStream_t st) {
    const int64_t tn = tiles(a.N, SWIGLU ? MANY_ROWS / 2 : MANY_ROWS), blocks = (most_tiles(a.g, 16 * MANY_BLOCKS) * tn + 7) / 8 * 8;
    if (!grid_fits(blocks, 64 * MANY_WAVES)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_many<G, KIND, TAIL, SWIGLU>), dim3((unsigned)blocks), dim3(64 * MANY_WAVES), 0, st, a, (int)tn);
    return hipGetLastError();
}

template <int R, int G, int KIND, bool TAIL, bool SWIGLU> hipError_t launch_few(const Q4Args &a, hipStream_t st) {
    const int64_t tn = tiles(a.N, SWIGLU ? 16 : 16 * R), blocks = (most_tiles(a.g, 16) * tn + 7) / 8 * 8;
    if (!grid_fits(blocks, 64 * FEW_WAVES)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_few<R, G, KIND, TAIL, SWIGLU>), dim3((unsigned)blocks), dim3(64 * FEW_WAVES), 0, st, a, (int)tn);
    return hipGetLastError();
}

template <int G, int KIND, bool TAIL, bool SWIGLU> hipError_t launch_kind(const Q4Args &a, hipStream_t st) {
    const int64_t used = a.g.n < a.g.rows ? a.g.n : a.g.rows;        // groups that can have rows
    if (tiles(a.N, SWIGLU ? MANY_ROWS / 2 : MANY_ROWS) * used >= MANY_FROM) return launch_many<G, KIND, TAIL, SWIGLU>(a, st);
    return launch_few<SWIGLU ? 2 : 1, G, KIND, TAIL, SWIGLU>(a, st);
}

template <int G, int KIND, bool TAIL> hipError_t launch_act(const Q4Args &a, hipStream_t st) {
    return a.swiglu ? launch_kind<G, KIND, TAIL, true>(a, st) : launch_kind<G, KIND, TAIL, false>(a, st);
}

template <int G, int KIND> hipError_t launch_tail(const Q4Args &a, hipStream_t st) {
    if constexpr (G < CHUNK) {
        if (a.K % CHUNK) return launch_act<G, KIND, true>(a, st);
    }
    return launch_act<G, KIND, false>(a, st);
}

template <int G> hipError_t launch_group(const Q4Args &a, hipStream_t st) {
    return a.scale_kind == Q4_F32 ? launch_tail<G, Q4_F32>(a, st) : a.scale_kind == Q4_BF16 ? launch_tail<G, Q4_BF16>(a, st)
                                                                                            : launch_tail<G, Q4_F16>(a, st);
}

}  // namespace

namespace moe {

hipError_t launch_q4(const Q4Args &a, hipStream_t st) {
    return a.group == 32 ? launch_group<32>(a, st) : a.group == 64 ? launch_group<64>(a, st) : launch_group<128>(a, st);
}

}  // namespace moe
