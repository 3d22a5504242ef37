// Residual addition and RMS norm, alone (moe_add_rms_norm) or closing the layer's combine (moe_combine_norm):
//
//   v = source row (x, or sum_j w_j o_j + shared, steered), v = round(v + residual) = residual_out
//   n = v / sqrt(sum v^2 / H + eps) * weight,  y = round(n)
//
// y is bf16, fp32, or e4m3: with one power-of-two scale per 32 columns (the block format that the scaled matrix
// instructions of gfx950 read) or one fp32 scale per row.  All sums are fp32, in an order fixed per launch shape.
//
// Bound: HBM traffic for many rows, one memory round trip and two barriers for few.  One workgroup holds one row in
// registers, so every input is read once: all loads of a row (source, residual, weight) are issued before the first
// reduction.  A copy of 2 GiB moves 4.97 TB/s on this chip; 11709 x 4096 with block scales takes 61.0 us (337 MB, 5.5 TB/s),
// 1469 x 4096 with row scales 14.8 (78 MB, 5.3 TB/s), 2048 combined rows of 8 x 4096 66.4 (344 MB, 5.2 TB/s); one row of 4096
// takes 2.4 us, one combined row 3.2, which is what a launch with one round trip to memory takes.
#include "common.h"
#include "internal.h"

using namespace moe;

namespace {

constexpr float E4M3_MAX = 448.f;

__device__ __forceinline__ float wg_sum(float d, float *part, int nw) {
    d = wave_sum(d);
    if (nw == 1) return d;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = d;
    __syncthreads();
    float tot = 0.f;
    for (int i = 0; i < nw; ++i) tot += part[i];
    return tot;
}

// v + its value in the lane that CTRL names
template <int CTRL> __device__ __forceinline__ double add_dpp_f64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)b, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(b >> 32), (int)(b >> 32), CTRL, 0xF, 0xF, false);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_f64(double v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), l) << 32 |
                                      (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l));
}

// 1 / sqrt(sum / H + eps) in two fp32 parts, from the threads' fp32 sums of squares.  The row's one factor moves all of its
// columns the same way, and where y is e4m3 an error in it decides blocks' scales and values that lie next to a rounding's
// border: so the sums meet in binary64, and the square root is taken there (the instruction's estimate and one Newton step).
// It costs no time: 11709 x 4096 61.2 us with and without, one row 6.3.
struct Factor { float hi, lo; };
__device__ __forceinline__ Factor row_factor(const NormArgs &a, float ss, double *part, int nw) {
    double d = add_dpp_f64<0xB1>((double)ss);               // quad swaps, then mirrors of 8 and 16 lanes
    d = add_dpp_f64<0x4E>(d);
    d = add_dpp_f64<0x141>(d);
    d = add_dpp_f64<0x140>(d);
    d = (lane_f64(d, 0) + lane_f64(d, 16)) + (lane_f64(d, 32) + lane_f64(d, 48));
    if (nw > 1) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = d;
        __syncthreads();
        d = 0.0;
        for (int i = 0; i < nw; ++i) d += part[i];
    }
    const double m = fma(d, a.inv_hidden, (double)a.eps), r0 = __builtin_amdgcn_rsq(m);
    const double r = m == HUGE_VAL ? 0.0 : fma(0.5 * r0, fma(-m * r0, r0, 1.0), r0);
    const float hi = (float)r;
    return {hi, (float)(r - (double)hi)};
}
// v * factor * w, off by little more than its one rounding
__device__ __forceinline__ float normed(float v, const Factor &r, float w) {
    const float hi = v * r.hi;
    const float lo = __fmaf_rn(v, r.lo, __fmaf_rn(v, r.hi, -hi));
    return __fmaf_rn(hi, w, lo * w);
}

__device__ __forceinline__ float wg_max(float d, float *part, int nw) {
    d = wave_max_f32(d);
    if (nw == 1) return d;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = d;
    __syncthreads();
    float m = 0.f;
    for (int i = 0; i < nw; ++i) m = fmaxf(m, part[i]);
    return m;
}

// Power-of-two block scale: the least e with amax <= 448 * 2^e (448 = 1.75 * 2^8), clamped to [-127, 127].  With
// amax = 1.f * 2^p that is p - 8, one more when the fraction is above 0.75; nothing saturates, so every value is off by
// at most half an e4m3 step.  A zero (or subnormal) block gets -127.
__device__ __forceinline__ int mx_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, -127), 127);
}
// 2^-e for e in [-127, 127] (2^-127 is subnormal)
__device__ __forceinline__ float exp2_neg(int e) {
    return __uint_as_float(e < 127 ? (uint32_t)(127 - e) << 23 : 0x400000u);
}
__device__ __forceinline__ float row_scale(float amax) { return fmaxf(amax, E4M3_MAX * 0x1p-126f) / E4M3_MAX; }

// v / s, s > 0: the product with 1 / s and the remainder's share (an infinite s, of a row that holds one: the product alone)
__device__ __forceinline__ float quotient(float v, float s, float inv) {
    const float q = v * inv;
    return s < HUGE_VALF ? __fmaf_rn(__fmaf_rn(-q, s, v), inv, q) : q;
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)a, (__bf16)b});
}
__device__ __forceinline__ float bf16_round(float a) { return (float)(__bf16)a; }
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// --- eight consecutive columns of one thread -------------------------------------------------------------------
struct Raw8 { uint4 lo, hi; };          // bf16: lo alone

template <bool BF16> __device__ __forceinline__ Raw8 load8(const void *p, int64_t i) {
    Raw8 r;
    if constexpr (BF16) {
        r.lo = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
    } else {
        const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i);
        r.lo = q[0];
        r.hi = q[1];
    }
    return r;
}
template <bool BF16> __device__ __forceinline__ void unpack8(const Raw8 &r, float (&f)[8]) {
    if constexpr (BF16) {
        const uint32_t w[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const uint32_t w[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
}
__device__ __forceinline__ void store8_f32(void *p, int64_t i, const float (&f)[8]) {
    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8_bf16(void *p, int64_t i, const float (&f)[8]) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
        make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}

enum { SRC_F32 = 0, SRC_BF16 = 1, SRC_COMBINE = 2 };     // what the row comes from
// One row per workgroup, C groups of eight columns per thread: group g = threadIdx.x + r * blockDim.x, so the four
// groups of a 32-column block lie in four adjacent lanes.  Needs H % 8 == 0 and 16-byte aligned rows.
template <int SRC, int RES, int C, int KC>
__global__ __launch_bounds__(1024) void k_norm_vec(NormArgs a) {
    __shared__ float part[2][16];
    __shared__ double part64[16];
    const int64_t t = blockIdx.x, row = t * a.H;
    const int nt = blockDim.x, nw = nt >> 6, ng = a.H >> 3;
    float v[C][8];
    Raw8 res[C], wt[C];
    bool on[C];
#pragma unroll
    for (int r = 0; r < C; ++r) on[r] = (int)threadIdx.x + r * nt < ng;
    if constexpr (SRC == SRC_COMBINE) {
        const int k = KC > 0 ? KC : a.k;
        const float *w = a.topk_w + t * k;
#pragma unroll
        for (int r = 0; r < C; ++r) {
            const int64_t c = 8 * ((int64_t)threadIdx.x + (int64_t)r * nt);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[r][i] = 0.f;
            if (!on[r]) continue;
            if constexpr (RES != RES_NONE) res[r] = load8<RES == RES_BF16>(a.residual, row + c);
            wt[r] = a.w_bf16 ? load8<true>(a.weight, c) : load8<false>(a.weight, c);
            if constexpr (KC > 0) {
                Raw8 o[KC], sh;
#pragma unroll
                for (int j = 0; j < KC; ++j) o[j] = load8<false>(a.slot_out, (t * KC + j) * a.H + c);
                if (a.shared_out) sh = load8<false>(a.shared_out, row + c);
#pragma unroll
                for (int j = 0; j < KC; ++j) {
                    float f[8];
                    unpack8<false>(o[j], f);
                    const float wj = w[j];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[r][i] = __fmaf_rn(wj, f[i], v[r][i]);
                }
                if (a.shared_out) {
                    float f[8];
                    unpack8<false>(sh, f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[r][i] += f[i];
                }
            } else {
                for (int j = 0; j < k; ++j) {
                    float f[8];
                    unpack8<false>(load8<false>(a.slot_out, (t * k + j) * a.H + c), f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[r][i] = __fmaf_rn(w[j], f[i], v[r][i]);
                }
                if (a.shared_out) {
                    float f[8];
                    unpack8<false>(load8<false>(a.shared_out, row + c), f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[r][i] += f[i];
                }
            }
        }
        if (a.steer_v) {
            float d = 0.f;
            float sv[C][8];
#pragma unroll
            for (int r = 0; r < C; ++r) {
                if (!on[r]) continue;
                unpack8<false>(load8<false>(a.steer_v, 8 * ((int64_t)threadIdx.x + (int64_t)r * nt)), sv[r]);
#pragma unroll
                for (int i = 0; i < 8; ++i) d = __fmaf_rn(sv[r][i], v[r][i], d);
            }
            const float sf = -a.steer_f * wg_sum(d, part[0], nw);
#pragma unroll
            for (int r = 0; r < C; ++r) {
                if (!on[r]) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[r][i] = __fmaf_rn(sf, sv[r][i], v[r][i]);
            }
        }
    } else {
        Raw8 x[C];
#pragma unroll
        for (int r = 0; r < C; ++r) {
            const int64_t c = 8 * ((int64_t)threadIdx.x + (int64_t)r * nt);
            if (!on[r]) continue;
            x[r] = load8<SRC == SRC_BF16>(a.x, row + c);
            if constexpr (RES != RES_NONE) res[r] = load8<RES == RES_BF16>(a.residual, row + c);
        }
#pragma unroll
        for (int r = 0; r < C; ++r) {
            if (!on[r]) continue;
            const int64_t c = 8 * ((int64_t)threadIdx.x + (int64_t)r * nt);
            wt[r] = a.w_bf16 ? load8<true>(a.weight, c) : load8<false>(a.weight, c);
        }
#pragma unroll
        for (int r = 0; r < C; ++r) {
            if (on[r]) {
                unpack8<SRC == SRC_BF16>(x[r], v[r]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[r][i] = 0.f;
            }
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        const int64_t c = 8 * ((int64_t)threadIdx.x + (int64_t)r * nt);
        if constexpr (RES != RES_NONE) {
            if (on[r]) {
                float f[8];
                unpack8<RES == RES_BF16>(res[r], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[r][i] += f[i];
                    if constexpr (RES == RES_BF16) v[r][i] = bf16_round(v[r][i]);   // the norm is of what is stored
                }
                if constexpr (RES == RES_BF16) store8_bf16(a.residual_out, row + c, v[r]);
                else store8_f32(a.residual_out, row + c, v[r]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __fmaf_rn(v[r][i], v[r][i], ss);
    }
    const Factor rinv = row_factor(a, ss, part64, nw);
    float amax = 0.f;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        float f[8] = {};
        if (on[r]) {
            if (a.w_bf16) unpack8<true>(wt[r], f);
            else unpack8<false>(wt[r], f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[r][i] = on[r] ? normed(v[r][i], rinv, f[i]) : 0.f;
            amax = fmaxf(amax, fabsf(v[r][i]));
        }
    }
    float inv = 1.f;
    if (a.y_kind == NORM_ROW8) {
        const float s = row_scale(wg_max(amax, part[1], nw));
        if (threadIdx.x == 0) static_cast<float *>(a.y_scale)[t] = s;
        const float rs = 1.0f / s;
#pragma unroll
        for (int r = 0; r < C; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[r][i] = quotient(v[r][i], s, rs);
    }
#pragma unroll
    for (int r = 0; r < C; ++r) {
        const int g = (int)threadIdx.x + r * nt;
        const int64_t c = 8 * (int64_t)g;
        if (a.y_kind == NORM_BF16) {
            if (on[r]) store8_bf16(a.y, row + c, v[r]);
        } else if (a.y_kind == NORM_F32) {
            if (on[r]) store8_f32(a.y, row + c, v[r]);
        } else {
            if (a.y_kind == NORM_MX8) {
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[r][i]));
                m = fmax_dpp<0xB1>(m);                     // the block's other three lanes: quad swaps 1 and 2
                m = fmax_dpp<0x4E>(m);
                const int e = mx_exponent(m);
                if (on[r] && (g & 3) == 0)
                    static_cast<uint8_t *>(a.y_scale)[t * ((a.H + 31) / 32) + (g >> 2)] = (uint8_t)(e + 127);
                inv = exp2_neg(e);
            }
            if (on[r]) {
                const float (&f)[8] = v[r];
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.y) + row + c) =
                    make_uint2(e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                               e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
            }
        }
    }
}

__device__ __forceinline__ float load1(const void *p, int64_t i, bool bf16) {
    return bf16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

// Any row length up to EL * blockDim.x and any alignment: column c = threadIdx.x + i * blockDim.x, one element per
// load, so a 32-column block lies in one half of a wave.  Columns behind the row's end load its last one and count as
// zero: without branches around them all of a row's loads are in flight at once (515 x 2055 bf16: 9.8 us, 16.4 with branches;
// 8.5 MB in elements of 2 bytes per lane, bound by their number and two barriers).
template <int EL, int MAX_THREADS>
__global__ __launch_bounds__(MAX_THREADS) void k_norm_any(NormArgs a, int src) {
    __shared__ float part[2][16];
    __shared__ double part64[16];
    const int64_t t = blockIdx.x, row = t * a.H;
    const int nt = blockDim.x, nw = nt >> 6;
    float v[EL], res[EL], wt[EL];
    int at[EL];
#pragma unroll
    for (int i = 0; i < EL; ++i) at[i] = min((int)threadIdx.x + i * nt, a.H - 1);
    if (src == SRC_COMBINE) {
#pragma unroll
        for (int i = 0; i < EL; ++i) v[i] = 0.f;
        for (int j = 0; j < a.k; ++j) {
            const float *o = a.slot_out + (t * a.k + j) * a.H, w = a.topk_w[t * a.k + j];
            float x[EL];
#pragma unroll
            for (int i = 0; i < EL; ++i) x[i] = o[at[i]];
#pragma unroll
            for (int i = 0; i < EL; ++i) v[i] = __fmaf_rn(w, x[i], v[i]);
        }
        if (a.shared_out) {
            float x[EL];
#pragma unroll
            for (int i = 0; i < EL; ++i) x[i] = a.shared_out[row + at[i]];
#pragma unroll
            for (int i = 0; i < EL; ++i) v[i] += x[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < EL; ++i) v[i] = load1(a.x, row + at[i], src == SRC_BF16);
    }
    if (a.res_kind != RES_NONE) {
#pragma unroll
        for (int i = 0; i < EL; ++i) res[i] = load1(a.residual, row + at[i], a.res_kind == RES_BF16);
    }
#pragma unroll
    for (int i = 0; i < EL; ++i) wt[i] = load1(a.weight, at[i], a.w_bf16);
    if (src == SRC_COMBINE && a.steer_v) {
        float d = 0.f, sv[EL];
#pragma unroll
        for (int i = 0; i < EL; ++i) sv[i] = a.steer_v[at[i]];
#pragma unroll
        for (int i = 0; i < EL; ++i) d = (int)threadIdx.x + i * nt < a.H ? __fmaf_rn(sv[i], v[i], d) : d;
        const float sf = -a.steer_f * wg_sum(d, part[0], nw);
#pragma unroll
        for (int i = 0; i < EL; ++i) v[i] = __fmaf_rn(sf, sv[i], v[i]);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < EL; ++i) {
        const int c = (int)threadIdx.x + i * nt;
        if (a.res_kind != RES_NONE) v[i] += res[i];
        if (a.res_kind == RES_BF16) v[i] = bf16_round(v[i]);
        if (c >= a.H) v[i] = 0.f;
        ss = __fmaf_rn(v[i], v[i], ss);
        if (c < a.H && a.res_kind == RES_F32) static_cast<float *>(a.residual_out)[row + c] = v[i];
        if (c < a.H && a.res_kind == RES_BF16) static_cast<__bf16 *>(a.residual_out)[row + c] = (__bf16)v[i];
    }
    const Factor rinv = row_factor(a, ss, part64, nw);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < EL; ++i) {
        v[i] = normed(v[i], rinv, wt[i]);
        amax = fmaxf(amax, fabsf(v[i]));
    }
    float inv = 1.f;
    if (a.y_kind == NORM_ROW8) {
        const float s = row_scale(wg_max(amax, part[1], nw));
        if (threadIdx.x == 0) static_cast<float *>(a.y_scale)[t] = s;
        const float rs = 1.0f / s;
#pragma unroll
        for (int i = 0; i < EL; ++i) v[i] = quotient(v[i], s, rs);
    }
#pragma unroll
    for (int i = 0; i < EL; ++i) {
        const int c = (int)threadIdx.x + i * nt;
        if (a.y_kind == NORM_MX8) {
            float m = fabsf(v[i]);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
            const int e = mx_exponent(m);
            if (c < a.H && (c & 31) == 0)
                static_cast<uint8_t *>(a.y_scale)[t * ((a.H + 31) / 32) + (c >> 5)] = (uint8_t)(e + 127);
            inv = exp2_neg(e);
        }
        if (c >= a.H) continue;
        if (a.y_kind == NORM_BF16) static_cast<__bf16 *>(a.y)[row + c] = (__bf16)v[i];
        else if (a.y_kind == NORM_F32) static_cast<float *>(a.y)[row + c] = v[i];
        else static_cast<uint8_t *>(a.y)[row + c] = (uint8_t)(e4m3x4(v[i] * inv, 0.f, 0.f, 0.f) & 0xFFu);
    }
}

template <int SRC, int RES, int KC>
hipError_t launch_vec(const NormArgs &a, int c, int nt, hipStream_t st) {
    const dim3 grd((unsigned)a.T), blk((unsigned)nt);
    if (c == 1) hipLaunchKernelGGL((k_norm_vec<SRC, RES, 1, KC>), grd, blk, 0, st, a);
    else if (c == 2) hipLaunchKernelGGL((k_norm_vec<SRC, RES, 2, KC>), grd, blk, 0, st, a);
    else hipLaunchKernelGGL((k_norm_vec<SRC, RES, 4, KC>), grd, blk, 0, st, a);
    return hipGetLastError();
}

template <int SRC, int KC>
hipError_t launch_res(const NormArgs &a, int c, int nt, hipStream_t st) {
    if (a.res_kind == RES_NONE) return launch_vec<SRC, RES_NONE, KC>(a, c, nt, st);
    if (a.res_kind == RES_F32) return launch_vec<SRC, RES_F32, KC>(a, c, nt, st);
    return launch_vec<SRC, RES_BF16, KC>(a, c, nt, st);
}

bool aligned16(const void *p) { return ((uintptr_t)p % 16) == 0; }

}  // namespace

namespace moe {

hipError_t launch_norm(const NormArgs &a, hipStream_t st) {
    const int src = a.slot_out ? SRC_COMBINE : a.x_bf16 ? SRC_BF16 : SRC_F32;
    const bool vec = a.H % 8 == 0 && aligned16(a.x) && aligned16(a.residual) && aligned16(a.residual_out) &&
                     aligned16(a.weight) && aligned16(a.y) && aligned16(a.slot_out) && aligned16(a.shared_out) &&
                     aligned16(a.steer_v);
    if (!vec) {
        const int nt = a.H <= 256 ? 64 : a.H <= 8192 ? 256 : 1024;
        const dim3 grd((unsigned)a.T), blk((unsigned)nt);
        if (a.H <= 4 * nt) hipLaunchKernelGGL((k_norm_any<4, 256>), grd, blk, 0, st, a, src);
        else if (a.H <= 4096) hipLaunchKernelGGL((k_norm_any<16, 256>), grd, blk, 0, st, a, src);
        else if (a.H <= 8192) hipLaunchKernelGGL((k_norm_any<32, 256>), grd, blk, 0, st, a, src);
        else if (a.H <= 16384) hipLaunchKernelGGL((k_norm_any<16, 1024>), grd, blk, 0, st, a, src);
        else hipLaunchKernelGGL((k_norm_any<32, 1024>), grd, blk, 0, st, a, src);
        return hipGetLastError();
    }
    const int ng = a.H / 8;
    const int c = ng <= 1024 ? 1 : ng <= 2048 ? 2 : 4;
    const int nt = ((ng + c - 1) / c + 63) / 64 * 64;
    if (src == SRC_F32) return launch_res<SRC_F32, 0>(a, c, nt, st);
    if (src == SRC_BF16) return launch_res<SRC_BF16, 0>(a, c, nt, st);
    if (a.k == 8) return launch_res<SRC_COMBINE, 8>(a, c, nt, st);
    return launch_res<SRC_COMBINE, 0>(a, c, nt, st);
}

}  // namespace moe
