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

// Eight codes as 16 + code, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 unpack(uint32_t w) {
    constexpr uint32_t M = 0x00780078u, E = 0x41804180u;
    return make_uint4((w << 3 & M) | E, (w >> 1 & M) | E, (w >> 5 & M) | E, (w >> 9 & M) | E);
}

// Eight values of x in the same order.
__device__ __forceinline__ uint4 reorder(uint4 v) {
    return make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                      __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u));
}

// Scales and zero points of one row's groups in a chunk, as they are loaded.
template <int G> struct Params {
    static constexpr int NG = CHUNK / G;
    uint32_t scale[NG], zero;

    // c0: the chunk's first column; row: the row's first group (index into scale and zero)
    __device__ __forceinline__ void load(const Q4Args &a, int64_t row, int c0) {
        const int64_t i = row + c0 / G;
        zero = 0x08080808u;
        if (NG == 1 || c0 + CHUNK <= a.K) {                  // all of the chunk's groups, at addresses aligned to elements
            if (a.scale_kind == Q4_F32) {
                __builtin_memcpy(scale, static_cast<const float *>(a.scale) + i, 4 * NG);
            } else {
                uint16_t h[NG];
                __builtin_memcpy(h, static_cast<const uint16_t *>(a.scale) + i, 2 * NG);
#pragma unroll
                for (int j = 0; j < NG; ++j) scale[j] = h[j];
            }
            if (a.zero) {
                uint8_t z[NG];
                __builtin_memcpy(z, a.zero + i, NG);
#pragma unroll
                for (int j = 0; j < NG; ++j) zero = (j ? zero : 0u) | (uint32_t)z[j] << (8 * j);
            }
        } else {                                             // the row ends here
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const bool in = c0 + j * G < a.K;
                scale[j] = !in ? 0u : a.scale_kind == Q4_F32 ? static_cast<const uint32_t *>(a.scale)[i + j]
                                                             : (uint32_t)static_cast<const uint16_t *>(a.scale)[i + j];
                if (a.zero && in) zero = (zero & ~(0xFFu << (8 * j))) | (uint32_t)a.zero[i + j] << (8 * j);
            }
        }
    }
    __device__ __forceinline__ float scale_of(const Q4Args &a, int j) const {
        return a.scale_kind == Q4_F32 ? __uint_as_float(scale[j])
               : a.scale_kind == Q4_BF16 ? bf16_bits_to_f32(scale[j]) : f16_bits_to_f32(scale[j]);
    }
    // -(16 + zero point) as a pair of bf16
    __device__ __forceinline__ uint32_t offset_of(int j) const {
        return ((zero >> (8 * j) & 15u) << 3 | 0xC180u) * 0x10001u;
    }
};

__device__ __forceinline__ uint4 splat(uint32_t v) { return make_uint4(v, v, v, v); }

// One chunk's products of 16 weight rows with 16 rows of x into acc.
template <int G>
__device__ __forceinline__ void chunk_products(const Q4Args &a, uint32_t (&w)[4], const Params<G> &p, const uint4 (&x)[4], f32x4_t &acc) {
    exchange(w);
#pragma unroll
    for (int j = 0; j < CHUNK / G; ++j) {
        const uint4 off = splat(p.offset_of(j));
        f32x4_t d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = j * G / 32; s < (j + 1) * G / 32; ++s) {
            d = mfma16(x[s], off, d);
            d = mfma16(x[s], unpack(w[s]), d);
        }
        const float sc = p.scale_of(a, j);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] = __fmaf_rn(sc, d[v], acc[v]);
    }
}

__device__ __forceinline__ void store(const Q4Args &a, int64_t i, float v) {
    if (a.out_bf16) static_cast<__bf16 *>(a.out)[i] = (__bf16)v;
    else static_cast<float *>(a.out)[i] = v;
}

// ---------------------------------------------------------------------------
// Few rows of x: a workgroup has 16 R weight rows (SwiGLU: R halves of gate and up) and up to 16 positions of a group; its waves
// take the row's chunks in turn, FEW_AHEAD of them loaded at once, and their sums meet in LDS.
// ---------------------------------------------------------------------------
constexpr int FEW_WAVES = 8, FEW_AHEAD = 4;

template <int R, int G, bool SWIGLU>
__global__ __launch_bounds__(64 * FEW_WAVES) void k_few(Q4Args a, int tiles_n) {
    static_assert(!SWIGLU || R == 2, "");
    constexpr int ROWS = SWIGLU ? 16 : 16 * R;               // results per position
    __shared__ __attribute__((aligned(16))) f32x4_t part[FEW_WAVES][R][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i16 = lane & 15, q = lane >> 4;
    const Tiles all = scan_tiles(a.g, 16);
    const int total = all.total * tiles_n, per = (total + 7) / 8;
    const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
    const int block = id / (4 * tiles_n), in = id - block * 4 * tiles_n, height = min(4, all.total - 4 * block);
    const int tn = in / height, n0 = tn * ROWS;
    const Tile t = tile_at(a.g, all, 16, 4 * block + in - tn * height);
    const int xr = t.begin + i16 < t.end ? in_row(a.g, t.begin + i16, a.x_rows) : -1;
    const uint16_t *x = a.x + (int64_t)max(xr, 0) * a.K + 8 * q;
    const uint8_t *codes[R];
    int64_t params[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t row = (int64_t)t.group * a.N * (SWIGLU ? 2 : 1) +
                            (SWIGLU ? (int64_t)r * a.N + min(n0 + i16, a.N - 1) : min(n0 + 16 * r + i16, a.N - 1));
        codes[r] = a.codes + row * (a.K / 2) + 16 * q;
        params[r] = row * (a.K / G);
    }
    f32x4_t acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int c0 = wave * CHUNK; c0 < a.K; c0 += FEW_AHEAD * FEW_WAVES * CHUNK) {
        u32x4_t w[FEW_AHEAD][R];
        Params<G> p[FEW_AHEAD][R];
        uint4 v[FEW_AHEAD][4];
#pragma unroll
        for (int u = 0; u < FEW_AHEAD; ++u) {
            const int c = c0 + u * FEW_WAVES * CHUNK;
            if (c >= a.K) break;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                w[u][r] = u32x4_t{0, 0, 0, 0};
                if (c + 32 * q < a.K) w[u][r] = *reinterpret_cast<const u32x4_t *>(codes[r] + c / 2);
                p[u][r].load(a, params[r], c);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                v[u][s] = make_uint4(0, 0, 0, 0);
                if (xr >= 0 && c + 32 * s < a.K) v[u][s] = *reinterpret_cast<const uint4 *>(x + c + 32 * s);
            }
        }
#pragma unroll
        for (int u = 0; u < FEW_AHEAD; ++u) {
            if (c0 + u * FEW_WAVES * CHUNK >= a.K) break;
            uint4 y[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) y[s] = reorder(v[u][s]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                uint32_t c[4] = {w[u][r][0], w[u][r][1], w[u][r][2], w[u][r][3]};
                chunk_products<G>(a, c, p[u][r], y, acc[r]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) part[wave][r][lane] = acc[r];
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

template <int R, int G, bool SWIGLU> hipError_t launch_few(const Q4Args &a, hipStream_t st) {
    const int64_t tn = (a.N + (SWIGLU ? 16 : 16 * R) - 1) / (SWIGLU ? 16 : 16 * R), blocks = (most_tiles(a.g, 16) * tn + 7) / 8 * 8;
    if (!grid_fits(blocks, 64 * FEW_WAVES)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_few<R, G, SWIGLU>), dim3((unsigned)blocks), dim3(64 * FEW_WAVES), 0, st, a, (int)tn);
    return hipGetLastError();
}

template <int G> hipError_t launch_group(const Q4Args &a, hipStream_t st) {
    return a.swiglu ? launch_few<2, G, true>(a, st) : launch_few<1, G, false>(a, st);
}

}  // namespace

namespace moe {

hipError_t launch_q4(const Q4Args &a, hipStream_t st) {
    return a.group == 32 ? launch_group<32>(a, st) : a.group == 64 ? launch_group<64>(a, st) : launch_group<128>(a, st);
}

}  // namespace moe
