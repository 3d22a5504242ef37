// Residual addition and RMS norm, alone (moe_add_rms_norm) or closing the layer's combine (moe_combine_norm):
//
//   v = source row (x, or sum_j w_j o_j + shared, steered), v = round(v + residual) = residual_out
//   n = v / sqrt(sum v^2 / H + eps) * weight,  y = round(n)
//
// y is bf16, fp32, or e4m3: with one power-of-two scale per 32 columns (the block format that the scaled matrix
// instructions of gfx950 read) or one fp32 scale per row.  All sums are in binary64, in an order fixed per launch shape.
//
// Bound: HBM traffic for many rows, one memory round trip and two barriers for few.  One workgroup holds one row in
// registers, so every input is read once: all loads of a row (source, residual, weight) are issued before the first
// reduction.  A copy of 2 GiB moves 4.85 to 4.97 TB/s on this chip; 11709 x 4096 with block scales takes 61.5 us (337 MB, 5.5
// TB/s), 1469 x 4096 with row scales 15.6 (78 MB, 5.0 TB/s), 2048 combined rows of 8 x 4096 66.4 (344 MB, 5.2 TB/s); one row of
// 4096 takes 2.4 us, one combined row 3.4, which is what a launch with one round trip to memory takes (kernels alone, medians).
// Short rows leave most of a workgroup's lanes without columns (whole calls: 16384 x 128 bf16 8.3 us, 2.0 TB/s), and rows of
// more than 16384 columns spill registers (512 x 32768 bf16 38 us, 3.5 TB/s; 512 x 16384 16.1, 4.2).
#include <type_traits>

#include "common.h"
#include "internal.h"

using namespace moe;

namespace {

// The waves' exchanges through LDS; a barrier that does not wait for the residual's stores.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// v of the lane that CTRL names
template <int CTRL> __device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)b, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(b >> 32), (int)(b >> 32), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_f64(double v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), l) << 32 |
                                      (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l));
}

// Sum, or largest value that is no NaN (of values >= 0), over the workgroup
template <bool MAX> __device__ __forceinline__ double join(double x, double y) { return MAX ? fmax(x, y) : x + y; }
template <bool MAX> __device__ __forceinline__ double wg_join(double d, double *part, int nw) {
    d = join<MAX>(d, dpp_f64<0xB1>(d));                     // quad swaps, then mirrors of 8 and 16 lanes
    d = join<MAX>(d, dpp_f64<0x4E>(d));
    d = join<MAX>(d, dpp_f64<0x141>(d));
    d = join<MAX>(d, dpp_f64<0x140>(d));
    d = join<MAX>(join<MAX>(lane_f64(d, 0), lane_f64(d, 16)), join<MAX>(lane_f64(d, 32), lane_f64(d, 48)));
    if (nw == 1) return d;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = d;
    lds_barrier();
    d = 0.0;
    for (int i = 0; i < nw; ++i) d = join<MAX>(d, part[i]);
    return d;
}
__device__ __forceinline__ double wg_sum(double d, double *part, int nw) { return wg_join<false>(d, part, nw); }

// 1 / sqrt(sum / H + eps) in two fp32 parts, from the threads' binary64 sums of squares. The row's one factor moves all of its
// columns the same way, and where y is e4m3 an error in it decides blocks' scales and values that lie next to a rounding's
// border; and fp32 holds the squares of half of its own exponents only. The square root is taken in binary64 too (the
// instruction's estimate and one Newton step). Whole calls with fp32 squares per thread and with binary64 ones: 11709 x 4096
// 60.6 and 61.1 us, 1469 x 4096 15.0 and 15.1, one row the same. Combined rows in binary64 cost nothing (2048 x 8 x 4096 66.2
// and 66.3 us), a row's scale and the quotients by it little (1469 x 4096 14.7 and 15.1). What is left is n's one rounding to
// fp32.
struct Factor { float hi, lo; double r; int exp; };
__device__ __forceinline__ Factor row_factor(const NormArgs &a, double ss, double *part, int nw) {
    const double m = fma(wg_sum(ss, part, nw), a.inv_hidden, (double)a.eps), r0 = __builtin_amdgcn_rsq(m);
    const double r = m == HUGE_VAL ? 0.0 : fma(0.5 * r0, fma(-m * r0, r0, 1.0), r0);
    // Beside values near the ends of fp32 the factor is beyond it, or its low part is: then the values are multiplied by 2^exp
    // first, exactly, and the factor is near 1
    const bool far = r > 0x1p60 ? r < HUGE_VAL : r < 0x1p-60 && r > 0.0;
    const int e = __builtin_amdgcn_readfirstlane(far ? ilogb(r) : 0);        // the same for the whole row
    const double q = ldexp(r, -e);
    const float hi = (float)q;
    return {hi, (float)(q - (double)hi), r, e};
}
// v * factor * w, off by little more than its one rounding; v has been brought to the factor's 2^-exp
__device__ __forceinline__ float normed(float v, const Factor &r, float w) {
    const float hi = v * r.hi;
    const float lo = __fmaf_rn(v, r.lo, __fmaf_rn(v, r.hi, -hi));
    return __fmaf_rn(hi, w, lo * w);
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
// A row's scale from its largest |n|.  Rows with one are normed, scaled and only then rounded: n / s in binary64.
__device__ __forceinline__ double row_scale(double amax) { return fmax(amax, 448 * 0x1p-126) / 448; }

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

// 16 and 8 bytes at addresses that are aligned (AL) or whole elements only: one load or store either way. (Vector types of the
// compiler's own: a class like uint4 keeps its alignment in a packed struct.)
struct __attribute__((packed)) Any16 { u32x4_t v; };
struct __attribute__((packed)) Any8 { u32x2_t v; };
static_assert(alignof(Any16) == 1 && alignof(Any8) == 1, "");
template <bool AL> __device__ __forceinline__ uint4 get16(const void *p) {
    if constexpr (AL) return *static_cast<const uint4 *>(p);
    else return __builtin_bit_cast(uint4, static_cast<const Any16 *>(p)->v);
}
template <bool AL> __device__ __forceinline__ void put16(void *p, uint4 v) {
    if constexpr (AL) *static_cast<uint4 *>(p) = v;
    else static_cast<Any16 *>(p)->v = __builtin_bit_cast(u32x4_t, v);
}

template <bool BF16, bool AL> __device__ __forceinline__ Raw8 load8(const void *p, int64_t i) {
    Raw8 r;
    if constexpr (BF16) {
        r.lo = get16<AL>(static_cast<const uint16_t *>(p) + i);
    } else {
        r.lo = get16<AL>(static_cast<const float *>(p) + i);
        r.hi = get16<AL>(static_cast<const float *>(p) + i + 4);
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
// The first `n` of eight columns are stored: all of them, or (AL false, a row's last group) fewer.
template <bool AL> __device__ __forceinline__ void store8_f32(void *p, int64_t i, const float (&f)[8], int n) {
    float *q = static_cast<float *>(p) + i;
    if (AL || n == 8) {
        put16<AL>(q, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
        put16<AL>(q + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) q[e] = f[e];
}
template <bool AL> __device__ __forceinline__ void store8_bf16(void *p, int64_t i, const float (&f)[8], int n) {
    uint16_t *q = static_cast<uint16_t *>(p) + i;
    if (AL || n == 8) {
        put16<AL>(q, make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])));
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) q[e] = (uint16_t)(bf16_pair(f[e], 0.f) & 0xFFFFu);
}
template <bool AL> __device__ __forceinline__ void store8_e4m3(void *p, int64_t i, const float (&f)[8], float k, int n) {
    uint8_t *q = static_cast<uint8_t *>(p) + i;
    const uint2 v = make_uint2(e4m3x4(f[0] * k, f[1] * k, f[2] * k, f[3] * k), e4m3x4(f[4] * k, f[5] * k, f[6] * k, f[7] * k));
    if constexpr (AL) {
        *reinterpret_cast<uint2 *>(q) = v;
    } else if (n == 8) {
        reinterpret_cast<Any8 *>(q)->v = __builtin_bit_cast(u32x2_t, v);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) q[e] = (uint8_t)((e < 4 ? v.x : v.y) >> (8 * (e & 3)));
    }
}
// f[i] = f[i + s], 0 <= s <= 7, zeros from the end on
template <typename V> __device__ __forceinline__ void shift8(V (&f)[8], int s) {
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (s & o) == 0 ? f[i] : i + o < 8 ? f[i + o] : V(0);
}

// v = x + residual is an fp32 value, whatever it is rounded to next (the compiler would round binary64 to bf16 at once)
__device__ __forceinline__ float to_f32(double v) {
    float f = (float)v;
    asm("" : "+v"(f));
    return f;
}
__device__ __forceinline__ float to_f32(float v) { return v; }

enum { SRC_F32 = 0, SRC_BF16 = 1, SRC_COMBINE = 2 };     // what the row comes from
// One row per workgroup, C groups of eight columns per thread: group g = threadIdx.x + r * blockDim.x, so the four
// groups of a 32-column block lie in four adjacent lanes.  AL: H % 8 == 0 and 16-byte aligned rows.  Else a row's last group
// loads its last eight columns (H >= 8) and moves its own to the front, and addresses are aligned to elements only: one load
// for eight columns all the same.  515 x 2055 bf16, whole call: 5.4 us, with one column per lane and load 9.9.
template <int SRC, int RES, int C, int KC, bool AL>
__global__ __launch_bounds__(1024) void k_norm_vec(NormArgs a) {
    __shared__ double part64[3][16];
    const int64_t t = blockIdx.x, row = t * a.H;
    const int nt = blockDim.x, nw = nt >> 6;
    // combined rows are summed in binary64 and rounded once, with the residual
    typename std::conditional<SRC == SRC_COMBINE, double, float>::type s[C][8];
    float v[C][8];
    Raw8 res[C], wt[C];
    bool on[C];
    int n[C];                                                // columns of the group
    int64_t at[C];                                           // its first column as loaded
#pragma unroll
    for (int r = 0; r < C; ++r) {
        const int c = 8 * ((int)threadIdx.x + r * nt);
        on[r] = c < a.H;
        n[r] = AL ? 8 : min(8, a.H - c);
        at[r] = AL ? c : min(c, a.H - 8);
    }
    auto own = [&](auto &f, int r) __attribute__((always_inline)) {
        if (!AL && __ballot(on[r] && n[r] < 8)) shift8(f, on[r] ? 8 - n[r] : 0);
    };
    if constexpr (SRC == SRC_COMBINE) {
        constexpr int KB = KC > 0 ? KC : 4;                  // rows whose loads go out together
        const int k = KC > 0 ? KC : a.k;
        const float *w = a.topk_w + t * k;
#pragma unroll
        for (int r = 0; r < C; ++r) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s[r][i] = 0.0;
            if (!on[r]) continue;
            if constexpr (RES != RES_NONE) res[r] = load8<RES == RES_BF16, AL>(a.residual, row + at[r]);
            wt[r] = a.w_bf16 ? load8<true, AL>(a.weight, at[r]) : load8<false, AL>(a.weight, at[r]);
            Raw8 sh;
            if (a.shared_out) sh = load8<false, AL>(a.shared_out, row + at[r]);
            for (int j0 = 0; j0 < k; j0 += KB) {
                Raw8 o[KB];
#pragma unroll
                for (int j = 0; j < KB; ++j)
                    o[j] = load8<false, AL>(a.slot_out, (t * k + (KC > 0 ? j : min(j0 + j, k - 1))) * a.H + at[r]);
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    if (KC == 0 && j0 + j >= k) break;
                    float f[8];
                    unpack8<false>(o[j], f);
                    const double wj = (double)w[j0 + j];
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[r][i] = fma(wj, (double)f[i], s[r][i]);
                }
            }
            if (a.shared_out) {
                float f[8];
                unpack8<false>(sh, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[r][i] += (double)f[i];
            }
        }
#pragma unroll
        for (int r = 0; r < C; ++r) own(s[r], r);
        if (a.steer_v) {
            double d = 0.0;
            float sv[C][8];
#pragma unroll
            for (int r = 0; r < C; ++r) {
                if (on[r]) {
                    unpack8<false>(load8<false, AL>(a.steer_v, at[r]), sv[r]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) sv[r][i] = 0.f;
                }
            }
#pragma unroll
            for (int r = 0; r < C; ++r) {
                own(sv[r], r);
#pragma unroll
                for (int i = 0; i < 8; ++i) d = fma((double)sv[r][i], s[r][i], d);
            }
            const double sf = -(double)a.steer_f * wg_sum(d, part64[1], nw);
#pragma unroll
            for (int r = 0; r < C; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i) s[r][i] = fma(sf, (double)sv[r][i], s[r][i]);
        }
    } else {
        Raw8 x[C];
#pragma unroll
        for (int r = 0; r < C; ++r) {
            if (!on[r]) continue;
            x[r] = load8<SRC == SRC_BF16, AL>(a.x, row + at[r]);
            if constexpr (RES != RES_NONE) res[r] = load8<RES == RES_BF16, AL>(a.residual, row + at[r]);
        }
#pragma unroll
        for (int r = 0; r < C; ++r)
            if (on[r]) wt[r] = a.w_bf16 ? load8<true, AL>(a.weight, at[r]) : load8<false, AL>(a.weight, at[r]);
#pragma unroll
        for (int r = 0; r < C; ++r) {
            if (on[r]) {
                unpack8<SRC == SRC_BF16>(x[r], s[r]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) s[r][i] = 0.f;
            }
            own(s[r], r);
        }
    }
    double ss = 0.0;                                         // a square of fp32 is exact in binary64, however small or large
#pragma unroll
    for (int r = 0; r < C; ++r) {
        const int64_t c = 8 * ((int64_t)threadIdx.x + (int64_t)r * nt);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[r][i] = (float)s[r][i];
        if constexpr (RES != RES_NONE) {
            float f[8] = {};
            if (on[r]) unpack8<RES == RES_BF16>(res[r], f);
            own(f, r);
            if (on[r]) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[r][i] = to_f32(s[r][i] + f[i]);
                    if constexpr (RES == RES_BF16) v[r][i] = bf16_round(v[r][i]);   // the norm is of what is stored
                }
                if constexpr (RES == RES_BF16) store8_bf16<AL>(a.residual_out, row + c, v[r], n[r]);
                else store8_f32<AL>(a.residual_out, row + c, v[r], n[r]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            ss = fma((double)v[r][i], (double)v[r][i], ss);
            asm("" : "+v"(v[r][i]));                         // from here on v is fp32 again: its binary64 form is not kept
        }
    }
    const Factor rinv = row_factor(a, ss, part64[0], nw);
    auto weights = [&](float (&f)[8], int r) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.f;
        if (on[r]) {
            if (a.w_bf16) unpack8<true>(wt[r], f);
            else unpack8<false>(wt[r], f);
        }
        own(f, r);
    };
    float inv = 1.f;
    if (a.y_kind == NORM_ROW8) {
        double amax = 0.0;                                   // of v * weight, which binary64 holds exactly
#pragma unroll
        for (int r = 0; r < C; ++r) {
            float f[8];
            weights(f, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmax(amax, on[r] ? fabs((double)v[r][i] * (double)f[i]) : 0.0);
        }
        const double s = row_scale(wg_join<true>(amax, part64[2], nw) * rinv.r), k = rinv.r / s;
        if (threadIdx.x == 0) static_cast<float *>(a.y_scale)[t] = (float)s;
#pragma unroll
        for (int r = 0; r < C; ++r) {
            float f[8];
            weights(f, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[r][i] = on[r] ? (float)((double)v[r][i] * (double)f[i] * k) : 0.f;
        }
    } else {
        if (rinv.exp) {
#pragma unroll
            for (int r = 0; r < C; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[r][i] = ldexpf(v[r][i], rinv.exp);
        }
#pragma unroll
        for (int r = 0; r < C; ++r) {
            float f[8];
            weights(f, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[r][i] = on[r] ? normed(v[r][i], rinv, f[i]) : 0.f;
        }
    }
#pragma unroll
    for (int r = 0; r < C; ++r) {
        const int g = (int)threadIdx.x + r * nt;
        const int64_t c = 8 * (int64_t)g;
        if (a.y_kind == NORM_BF16) {
            if (on[r]) store8_bf16<AL>(a.y, row + c, v[r], n[r]);
        } else if (a.y_kind == NORM_F32) {
            if (on[r]) store8_f32<AL>(a.y, row + c, v[r], n[r]);
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
            if (on[r]) store8_e4m3<AL>(a.y, row + c, v[r], inv, n[r]);
        }
    }
}

__device__ __forceinline__ float load1(const void *p, int64_t i, bool bf16) {
    return bf16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

// Rows of fewer than eight columns: one wave per row, one column per lane.
__global__ __launch_bounds__(64) void k_norm_short(NormArgs a, int src) {
    const int64_t t = blockIdx.x, row = t * a.H;
    const int c = threadIdx.x;
    const bool on = c < a.H;
    float w = 0.f;
    double s = 0.0;
    if (on) {
        if (src == SRC_COMBINE) {
            for (int j = 0; j < a.k; ++j) s = fma((double)a.topk_w[t * a.k + j], (double)a.slot_out[(t * a.k + j) * a.H + c], s);
            if (a.shared_out) s += (double)a.shared_out[row + c];
        } else {
            s = (double)load1(a.x, row + c, src == SRC_BF16);
        }
        w = load1(a.weight, c, a.w_bf16);
    }
    if (src == SRC_COMBINE && a.steer_v) {
        const double sv = on ? (double)a.steer_v[c] : 0.0;
        s = fma(-(double)a.steer_f * wg_sum(sv * s, nullptr, 1), sv, s);
    }
    float v = (float)s;
    if (on && a.res_kind != RES_NONE) {
        v = to_f32(s + (double)load1(a.residual, row + c, a.res_kind == RES_BF16));
        if (a.res_kind == RES_BF16) v = bf16_round(v);
        if (a.res_kind == RES_BF16) static_cast<__bf16 *>(a.residual_out)[row + c] = (__bf16)v;
        else static_cast<float *>(a.residual_out)[row + c] = v;
    }
    const Factor rinv = row_factor(a, on ? (double)v * (double)v : 0.0, nullptr, 1);
    const double n = on ? (double)v * rinv.r * (double)w : 0.0;
    v = on ? normed(ldexpf(v, rinv.exp), rinv, w) : 0.f;
    if (a.y_kind == NORM_ROW8) {
        const double scale = row_scale(wg_join<true>(fabs(n), nullptr, 1));
        if (c == 0) static_cast<float *>(a.y_scale)[t] = (float)scale;
        v = (float)(n / scale);
    } else if (a.y_kind == NORM_MX8) {
        const int e = mx_exponent(wave_max_f32(fabsf(v)));
        if (c == 0) static_cast<uint8_t *>(a.y_scale)[t] = (uint8_t)(e + 127);
        v *= exp2_neg(e);
    }
    if (!on) return;
    if (a.y_kind == NORM_BF16) static_cast<__bf16 *>(a.y)[row + c] = (__bf16)v;
    else if (a.y_kind == NORM_F32) static_cast<float *>(a.y)[row + c] = v;
    else static_cast<uint8_t *>(a.y)[row + c] = (uint8_t)(e4m3x4(v, 0.f, 0.f, 0.f) & 0xFFu);
}

template <int SRC, int RES, int KC, bool AL>
hipError_t launch_vec(const NormArgs &a, int c, int nt, hipStream_t st) {
    const dim3 grd((unsigned)a.T), blk((unsigned)nt);
    if (c == 1) hipLaunchKernelGGL((k_norm_vec<SRC, RES, 1, KC, AL>), grd, blk, 0, st, a);
    else if (c == 2) hipLaunchKernelGGL((k_norm_vec<SRC, RES, 2, KC, AL>), grd, blk, 0, st, a);
    else hipLaunchKernelGGL((k_norm_vec<SRC, RES, 4, KC, AL>), grd, blk, 0, st, a);
    return hipGetLastError();
}

template <int SRC, int KC, bool AL>
hipError_t launch_res(const NormArgs &a, int c, int nt, hipStream_t st) {
    if (a.res_kind == RES_NONE) return launch_vec<SRC, RES_NONE, KC, AL>(a, c, nt, st);
    if (a.res_kind == RES_F32) return launch_vec<SRC, RES_F32, KC, AL>(a, c, nt, st);
    return launch_vec<SRC, RES_BF16, KC, AL>(a, c, nt, st);
}

template <bool AL>
hipError_t launch_rows(const NormArgs &a, int src, hipStream_t st) {
    const int ng = (a.H + 7) / 8;
    const int c = ng <= 1024 ? 1 : ng <= 2048 ? 2 : 4;
    const int nt = ((ng + c - 1) / c + 63) / 64 * 64;
    if (src == SRC_F32) return launch_res<SRC_F32, 0, AL>(a, c, nt, st);
    if (src == SRC_BF16) return launch_res<SRC_BF16, 0, AL>(a, c, nt, st);
    if constexpr (AL) {
        if (a.k == 8) return launch_res<SRC_COMBINE, 8, AL>(a, c, nt, st);
    }
    return launch_res<SRC_COMBINE, 0, AL>(a, c, nt, st);
}

bool aligned16(const void *p) { return ((uintptr_t)p % 16) == 0; }

}  // namespace

namespace moe {

hipError_t launch_norm(const NormArgs &a, hipStream_t st) {
    const int src = a.slot_out ? SRC_COMBINE : a.x_bf16 ? SRC_BF16 : SRC_F32;
    const bool vec = a.H % 8 == 0 && aligned16(a.x) && aligned16(a.residual) && aligned16(a.residual_out) &&
                     aligned16(a.weight) && aligned16(a.y) && aligned16(a.slot_out) && aligned16(a.shared_out) &&
                     aligned16(a.steer_v);
    if (a.H < 8) {
        hipLaunchKernelGGL(k_norm_short, dim3((unsigned)a.T), dim3(64), 0, st, a, src);
        return hipGetLastError();
    }
    return vec ? launch_rows<true>(a, src, st) : launch_rows<false>(a, src, st);
}

}  // namespace moe
