// Products over rows grouped by expert (moe_grouped_linear, moe_grouped_dgrad, moe_grouped_wgrad, moe_q4_linear):
//
//   forward           out[o][n] = sum_k x[r][k] W_g[n][k]
//   input's gradient  dx[i][k]  = sum_n dy[o][n] W_g[n][k]
//   weights' gradient dW_g[n][k] = sum over the positions of g of dy[o][n] x[r][k]
//
// One workgroup computes 64 x 64 results from fp32 tiles in LDS, 16 steps of the sum at a time.
#include "groups.h"

using namespace moe;

namespace {

constexpr int TILE = 64, STEP = 16;

__device__ __forceinline__ float at(const uint16_t *p, int64_t i) { return bf16_bits_to_f32(p[i]); }


__device__ __forceinline__ float q4_scale(const Q4Args &a, int64_t i) {
    if (a.scale_kind == Q4_F32) return static_cast<const float *>(a.scale)[i];
    const uint16_t v = static_cast<const uint16_t *>(a.scale)[i];
    return a.scale_kind == Q4_BF16 ? bf16_bits_to_f32(v) : f16_bits_to_f32(v);
}

// Weight row n, column k of matrix m.
__device__ __forceinline__ float q4_at(const Q4Args &a, int64_t row, int k) {
    const int64_t s = row * (a.K / a.group) + k / a.group;
    const int q = a.codes[row * (a.K / 2) + k / 2] >> (k & 1 ? 4 : 0) & 15, z = a.zero ? a.zero[s] & 15 : 8;
    return (float)(q - z) * q4_scale(a, s);
}

// R x C tile of products of load_a(row, k) and load_b(col, k), k < K; accumulates into acc[4][4].
template <typename A, typename B>
__device__ __forceinline__ void products(int K, A load_a, B load_b, float (&acc)[4][4]) {
    __shared__ float as[STEP][TILE], bs[STEP][TILE];
    const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
    for (int k0 = 0; k0 < K; k0 += STEP) {
        for (int e = threadIdx.x; e < STEP * TILE; e += 256) {
            const int r = e / STEP, k = e % STEP;
            as[k][r] = k0 + k < K ? load_a(r, k0 + k) : 0.f;
            bs[k][r] = k0 + k < K ? load_b(r, k0 + k) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < STEP; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(as[k][tr * 4 + i], bs[k][tc * 4 + j], acc[i][j]);
        __syncthreads();
    }
}

__device__ __forceinline__ void store(void *out, int bf16, int64_t i, float v) {
    if (bf16) static_cast<__bf16 *>(out)[i] = (__bf16)v;
    else static_cast<float *>(out)[i] = v;
}

template <int OP, bool SWIGLU> __global__ __launch_bounds__(256) void k_rows(GroupedArgs a) {
    Tile t;
    if (!find_tile(a.g, TILE, blockIdx.x, t)) return;
    const int K = OP == GROUPED_FWD ? a.n_in : a.n_out, N = OP == GROUPED_FWD ? a.n_out : a.n_in, n0 = blockIdx.y * TILE;
    const uint16_t *w = a.b + (int64_t)t.group * a.n_out * a.n_in * (SWIGLU ? 2 : 1);
    auto load_a = [&](int r, int k) {
        const int p = t.begin + r;
        if (p >= t.end) return 0.f;
        const int row = OP == GROUPED_FWD ? in_row(a.g, p, a.a_rows) : out_row(a.g, p, a.a_rows);
        return row < 0 ? 0.f : at(a.a, (int64_t)row * K + k);
    };
    float acc[2][4][4] = {};
    for (int h = 0; h < (SWIGLU ? 2 : 1); ++h)
        products(K, load_a, [&](int c, int k) {
            if (n0 + c >= N) return 0.f;
            return OP == GROUPED_FWD ? at(w, ((int64_t)h * N + n0 + c) * K + k) : at(w, (int64_t)k * N + n0 + c);
        }, acc[h]);
    const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
    for (int i = 0; i < 4; ++i) {
        const int p = t.begin + tr * 4 + i;
        if (p >= t.end) continue;
        const int row = OP == GROUPED_FWD ? out_row(a.g, p, a.out_rows) : in_slot(a.g, p, a.out_rows);
        if (row < 0) continue;
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tc * 4 + j;
            if (n < N) store(a.out, a.out_bf16, (int64_t)row * N + n, SWIGLU ? swiglu(acc[0][i][j], acc[1][i][j]) : acc[0][i][j]);
        }
    }
}

__global__ __launch_bounds__(256) void k_weights(GroupedArgs a) {
    const int g = blockIdx.x, n0 = blockIdx.z * TILE, k0 = blockIdx.y * TILE, b = group_edge(a.g, g), e = group_edge(a.g, g + 1);
    float acc[4][4] = {};
    products(max(e - b, 0), [&](int n, int p) {
        const int row = out_row(a.g, b + p, a.b_rows);
        return row < 0 || n0 + n >= a.n_out ? 0.f : at(a.b, (int64_t)row * a.n_out + n0 + n);
    }, [&](int k, int p) {
        const int row = in_row(a.g, b + p, a.a_rows);
        return row < 0 || k0 + k >= a.n_in ? 0.f : at(a.a, (int64_t)row * a.n_in + k0 + k);
    }, acc);
    const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tr * 4 + i, k = k0 + tc * 4 + j;
            if (n >= a.n_out || k >= a.n_in) continue;
            const int64_t o = ((int64_t)g * a.n_out + n) * a.n_in + k;
            float v = acc[i][j];
            if (a.accumulate) v += a.out_bf16 ? at(static_cast<const uint16_t *>(a.out), o) : static_cast<const float *>(a.out)[o];
            store(a.out, a.out_bf16, o, v);
        }
}

template <bool SWIGLU> __global__ __launch_bounds__(256) void k_q4(Q4Args a) {
    Tile t;
    if (!find_tile(a.g, TILE, blockIdx.x, t)) return;
    const int n0 = blockIdx.y * TILE;
    const int64_t w = (int64_t)t.group * a.N * (SWIGLU ? 2 : 1);
    auto load_a = [&](int r, int k) {
        const int p = t.begin + r, row = p < t.end ? in_row(a.g, p, a.x_rows) : -1;
        return row < 0 ? 0.f : at(a.x, (int64_t)row * a.K + k);
    };
    float acc[2][4][4] = {};
    for (int h = 0; h < (SWIGLU ? 2 : 1); ++h)
        products(a.K, load_a, [&](int c, int k) { return n0 + c < a.N ? q4_at(a, w + (int64_t)h * a.N + n0 + c, k) : 0.f; }, acc[h]);
    const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
    for (int i = 0; i < 4; ++i) {
        const int p = t.begin + tr * 4 + i, row = p < t.end ? out_row(a.g, p, a.out_rows) : -1;
        if (row < 0) continue;
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tc * 4 + j;
            if (n < a.N) store(a.out, a.out_bf16, (int64_t)row * a.N + n, SWIGLU ? swiglu(acc[0][i][j], acc[1][i][j]) : acc[0][i][j]);
        }
    }
}

// A grid whose threads and blocks a launch can count (2^32 threads, 2^16 blocks along y and z).
bool fits(int64_t x, int64_t y, int64_t z, int threads) {
    return x * threads < ((int64_t)1 << 32) && y < 65536 && z < 65536;
}

}  // namespace

namespace moe {

hipError_t launch_grouped(int op, const GroupedArgs &a, hipStream_t st) {
    const int64_t tn = (a.n_out + TILE - 1) / TILE, tk = (a.n_in + TILE - 1) / TILE, tr = most_tiles(a.g, TILE);
    if (!fits(tr, tn, tk, 256)) return hipErrorInvalidConfiguration;
    if (op == GROUPED_WGRAD) hipLaunchKernelGGL(k_weights, dim3(a.g.n, tk, tn), dim3(256), 0, st, a);
    else if (op == GROUPED_DGRAD) hipLaunchKernelGGL((k_rows<GROUPED_DGRAD, false>), dim3(tr, tk), dim3(256), 0, st, a);
    else if (a.swiglu) hipLaunchKernelGGL((k_rows<GROUPED_FWD, true>), dim3(tr, tn), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_rows<GROUPED_FWD, false>), dim3(tr, tn), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_q4(const Q4Args &a, hipStream_t st) {
    const int64_t tr = most_tiles(a.g, TILE), tn = (a.N + TILE - 1) / TILE;
    if (!fits(tr, tn, 1, 256)) return hipErrorInvalidConfiguration;
    if (a.swiglu) hipLaunchKernelGGL(k_q4<true>, dim3(tr, tn), dim3(256), 0, st, a);
    else hipLaunchKernelGGL(k_q4<false>, dim3(tr, tn), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace moe
