// The shared expert as a call of its own, with low-rank adapters of many requests (moe_shared_ffn):
//
//   g = Wg x + c_a Bg_a (Ag_a x),  u likewise,  h = silu(g) * u,  out = Wd h + c_a Bd_a (Ad_a h)
//
// with a = token_adapter[t] (no adapter terms where it is outside 0 .. n_adapters - 1).  All products run on the bf16
// matrix cores with fp32 sums.  Launches: [split] [plan] [down-rank] gate/up [down-rank] down --
//
//   split      fp32 activations as two bf16 planes hi + lo = bf16(x), bf16(x - hi): 16 significant bits
//   plan       (many tokens) the tokens ordered by adapter, and work items of up to 64 tokens of one adapter
//   down-rank  s[t][r] = A_a[r] . x[t] for each token's own adapter, fp32, summed over a few K splits by the reader
//   gate/up    weight rows x tokens; the adapters' B_a s in the epilogue; SwiGLU; h as one bf16 plane (bf16 result)
//              or two (fp32 result, whose error then stays near 2^-17)
//   down       the same product with Wd and h
//
// An adapter's term is formed in accumulators of its own and added to the rows of its own tokens only, so nothing of
// one request's adapter (not even a NaN) reaches another request.
#include "common.h"
#include "internal.h"

using namespace moe;

namespace {

typedef __attribute__((address_space(3))) void *las_ptr;

__device__ uint4 zero_chunk;             // 16 zero bytes that tiles read past the end of a row

__device__ __forceinline__ f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}
__device__ __forceinline__ f32x16_t mfma32(uint4 a, uint4 b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

__device__ __forceinline__ uint4 load16(const uint16_t *p) { return *reinterpret_cast<const uint4 *>(p); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)a, (__bf16)b});
}
__device__ __forceinline__ float bf16_rest(float a) { return a - (float)(__bf16)a; }

// The first `n` of eight bf16 values, the others zero.
__device__ __forceinline__ uint4 keep_first(uint4 v, int n) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 2 * i + 1 < n ? w[i] : 2 * i < n ? w[i] & 0xFFFFu : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ int rank_of(const SharedArgs &a, int ad) {
    return a.rank ? min(max(a.rank[ad], 0), a.R) : a.R;
}

// Adapter of row `pos` (sorted position with a plan, else token), -1 for none.
__device__ __forceinline__ int adapter_at(const SharedArgs &a, int pos) {
    if (!a.n || pos >= a.T) return -1;
    const int id = a.sorted ? a.plan_ad[pos] : a.token_adapter[pos];
    return (unsigned)id < (unsigned)a.n ? id : -1;
}

// Eight columns j8*8.. of the down-rank result of row `pos` (projection `proj` of `np`), scaled, as bf16 hi and lo.
__device__ __forceinline__ void low_rank8(const SharedArgs &a, const float *s, int np, int pos, int proj, int j8,
                                          float scale, int rank, uint4 &hi, uint4 &lo) {
    float v[8] = {};
    for (int k = 0; k < a.ks; ++k) {
        const float4 *p = reinterpret_cast<const float4 *>(s + (((int64_t)k * a.T + pos) * np + proj) * a.R + 8 * j8);
        const float4 x = p[0], y = p[1];
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 8 * j8 + i < rank ? v[i] * scale : 0.f;
    hi = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = bf16_rest(v[i]);
    lo = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// ---------------------------------------------------------------------------
// fp32 activations -> bf16 planes [2][T][H]
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_split(const float *__restrict__ x, uint16_t *__restrict__ planes, int64_t n) {
    const int64_t i = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (i >= n) return;
    const float4 v = *reinterpret_cast<const float4 *>(x + i);
    *reinterpret_cast<uint2 *>(planes + i) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    *reinterpret_cast<uint2 *>(planes + n + i) =
        make_uint2(pack_bf16(bf16_rest(v.x), bf16_rest(v.y)), pack_bf16(bf16_rest(v.z), bf16_rest(v.w)));
}

// ---------------------------------------------------------------------------
// plan: tokens ordered by adapter (those without one last), and items of up to ITEM_TOKENS tokens of one adapter.
// One workgroup.  Within an adapter the order is that of LDS atomics and may differ between calls: a row's place in
// a tile changes no bit of its result.
// ---------------------------------------------------------------------------
constexpr int PLAN_THREADS = 1024;

__global__ __launch_bounds__(PLAN_THREADS) void k_plan(SharedArgs a) {
    __shared__ int count[MAX_ADAPTERS + 1], wsum[2][PLAN_THREADS / 64];
    const int n = a.n, tid = threadIdx.x;
    for (int i = tid; i <= n; i += PLAN_THREADS) count[i] = 0;
    __syncthreads();
    for (int t = tid; t < a.T; t += PLAN_THREADS) {
        const int id = a.token_adapter[t];
        atomicAdd(&count[(unsigned)id < (unsigned)n ? id : n], 1);
    }
    __syncthreads();
    constexpr int PER = MAX_ADAPTERS / PLAN_THREADS + 1;             // consecutive bins per thread
    int c[PER], tok = 0, it = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int b = tid * PER + j;
        c[j] = b <= n ? count[b] : 0;
        tok += c[j];
        if (b < n) it += (c[j] + ITEM_TOKENS - 1) / ITEM_TOKENS;
    }
    int ptok = tok, pit = it;                                        // inclusive scans over the wave, then the waves
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(ptok, o, 64), y = __shfl_up(pit, o, 64);
        if ((tid & 63) >= o) { ptok += x; pit += y; }
    }
    if ((tid & 63) == 63) { wsum[0][tid >> 6] = ptok; wsum[1][tid >> 6] = pit; }
    __syncthreads();
    int btok = ptok - tok, bit = pit - it;
    for (int w = 0; w < (tid >> 6); ++w) { btok += wsum[0][w]; bit += wsum[1][w]; }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int b = tid * PER + j;
        if (b > n) break;
        count[b] = btok;                                             // becomes the bin's cursor
        if (b < n)
            for (int s = 0; s < c[j]; s += ITEM_TOKENS)
                a.items[bit++] = make_int4(b, btok + s, min(ITEM_TOKENS, c[j] - s), 0);
        btok += c[j];
    }
    if (tid == PLAN_THREADS - 1) *a.n_items = bit;
    __syncthreads();
    for (int t = tid; t < a.T; t += PLAN_THREADS) {
        const int id = a.token_adapter[t], b = (unsigned)id < (unsigned)n ? id : n;
        const int pos = atomicAdd(&count[b], 1);
        a.perm[pos] = t;
        a.plan_ad[pos] = b < n ? b : -1;
    }
}

// ---------------------------------------------------------------------------
// down-rank: s[ks][pos][proj][r] = sum over this K split of A_a[r] . x[pos] for the NP projections that read x.
// blockIdx.x = item (sorted: of the plan; else the blockIdx.x-th distinct adapter among at most 64 tokens),
// blockIdx.y = K split; the four waves split K further and their sums meet in LDS.
// ---------------------------------------------------------------------------
constexpr int LR_FRAGS = 8;              // 16-row fragments of [NP][R] per pass

template <int P, bool SORTED>
__global__ __launch_bounds__(256) void k_low_rank(SharedArgs a, LowRank L) {
    __shared__ float red[4][LR_FRAGS * 256];
    __shared__ int rows[64], meta[2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, q = lane >> 4;
    int ad, cnt;
    if constexpr (SORTED) {
        if ((int)blockIdx.x >= *a.n_items) return;
        const int4 it = a.items[blockIdx.x];
        ad = it.x;
        cnt = it.z;
        if ((int)threadIdx.x < cnt) rows[threadIdx.x] = it.y + threadIdx.x;
        __syncthreads();
    } else {
        if (wave == 0) {
            const int id = adapter_at(a, lane);
            unsigned long long left = __ballot(id >= 0);
            int found = -1, num = 0;
            for (int d = 0; left; ++d) {
                const int first = __ffsll(left) - 1;
                const int cur = __shfl(id, first, 64);
                const unsigned long long same = __ballot(id == cur);
                if (d == (int)blockIdx.x) {
                    found = cur;
                    num = __popcll(same);
                    if (id == cur) rows[__popcll(same & ((1ull << lane) - 1))] = lane;
                    break;
                }
                left &= ~same;
            }
            if (lane == 0) { meta[0] = found; meta[1] = num; }
        }
        __syncthreads();
        ad = meta[0];
        cnt = meta[1];
        if (ad < 0) return;
    }
    const int K = L.K, R = a.R, nrows = L.np * R, rank = rank_of(a, ad);
    const int steps = (K + 31) / 32, parts = a.ks * 4, part = blockIdx.y * 4 + wave;
    const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
    for (int t0 = 0; t0 < cnt; t0 += 16) {
        const int pos = rows[min(t0 + i16, cnt - 1)];
        const int64_t xrow = SORTED && L.gather ? a.perm[pos] : pos;
        for (int f0 = 0; f0 * 16 < nrows; f0 += LR_FRAGS) {
            f32x4_t acc[LR_FRAGS];
            const uint16_t *arow[LR_FRAGS];
#pragma unroll
            for (int f = 0; f < LR_FRAGS; ++f) {
                acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                const int rr = (f0 + f) * 16 + i16, proj = rr / R, r = rr - proj * R;
                arow[f] = rr < nrows && r < rank && L.a[proj] ? L.a[proj] + ((int64_t)ad * R + r) * K : nullptr;
            }
            for (int s = s0; s < s1; ++s) {
                const int k = s * 32 + q * 8;
                uint4 b[P];
#pragma unroll
                for (int p = 0; p < P; ++p)
                    b[p] = k < K ? load16(L.x + ((int64_t)p * a.T + xrow) * K + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int f = 0; f < LR_FRAGS; ++f) {
                    if ((f0 + f) * 16 >= nrows) break;
                    const uint4 w = arow[f] && k < K ? load16(arow[f] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int p = 0; p < P; ++p) acc[f] = mfma16(w, b[p], acc[f]);
                }
            }
#pragma unroll
            for (int f = 0; f < LR_FRAGS; ++f)
                *reinterpret_cast<f32x4_t *>(&red[wave][f * 256 + i16 * 16 + 4 * q]) = acc[f];   // [token][row]
            __syncthreads();
            for (int e = threadIdx.x; e < LR_FRAGS * 256; e += 256) {
                const int f = e >> 8, tok = (e >> 4) & 15, rr = (f0 + f) * 16 + (e & 15);
                if (t0 + tok < cnt && rr < nrows)
                    L.s[((int64_t)blockIdx.y * a.T + rows[t0 + tok]) * nrows + rr] =
                        (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------------------
// Few tokens: one workgroup streams 16 weight rows (gate/up: 8 gate rows and the same 8 of up) once, straight into
// the matrix instruction's operand registers; its eight waves split K and their sums meet in LDS.
// ---------------------------------------------------------------------------
template <bool GU, int P, int TF>
__global__ __launch_bounds__(512) void k_few(SharedArgs a, Product g) {
    __shared__ float red[8][TF][16][17];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, q = lane >> 4;
    const int K = g.K, r0 = blockIdx.x * (GU ? 8 : 16);
    const int wr = GU ? r0 + (i16 & 7) : r0 + i16;
    const uint16_t *wrow = (GU && i16 >= 8 ? g.w[1] : g.w[0]) + (int64_t)min(wr, g.N - 1) * K;
    const int steps = (K + 31) / 32;
    const int s0 = steps * wave / 8, s1 = steps * (wave + 1) / 8;
    f32x4_t acc[TF];
    const uint16_t *xrow[TF];
#pragma unroll
    for (int f = 0; f < TF; ++f) {
        acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        xrow[f] = g.x + (int64_t)min(f * 16 + i16, a.T - 1) * K;
    }
    const int64_t plane = (int64_t)a.T * K;
    constexpr int U = TF == 1 ? 8 : 4;
    for (int s = s0; s < s1; s += U) {
        uint4 w[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int k = (s + j) * 32 + q * 8;
            w[j] = s + j < s1 && k < K ? load16(wrow + k) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int k = (s + j) * 32 + q * 8;
            const bool in = s + j < s1 && k < K;
#pragma unroll
            for (int f = 0; f < TF; ++f)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    acc[f] = mfma16(w[j], in ? load16(xrow[f] + p * plane + k) : make_uint4(0, 0, 0, 0), acc[f]);
        }
    }
    if (a.n) {
        // adapter a is added by wave a % 8: a token's sum has the same order whatever else is in the batch
        const int c8 = a.R / 8, chunks = GU ? 2 * c8 : c8;
#pragma unroll
        for (int f = 0; f < TF; ++f) {
            const int pos = f * 16 + i16, id = adapter_at(a, pos);
            unsigned long long left = __ballot(id >= 0 && (id & 7) == wave);
            while (left) {
                const int ad = __shfl(id, __ffsll(left) - 1, 64);
                left &= ~__ballot(id == ad);
                const float scale = a.scale ? a.scale[ad] : 1.f;
                const int rank = rank_of(a, ad);
                f32x4_t d = {0.f, 0.f, 0.f, 0.f};
                for (int c0 = 0; c0 < chunks; c0 += 4) {
                    const int c = c0 + q, proj = c / c8, j8 = c - proj * c8;
                    uint4 w = make_uint4(0, 0, 0, 0), hi = w, lo = w;
                    if (c < chunks && 8 * j8 < rank && g.b[proj]) {
                        if ((!GU || (i16 >> 3) == proj) && wr < g.N)
                            w = keep_first(load16(g.b[proj] + ((int64_t)ad * g.N + wr) * a.R + 8 * j8), rank - 8 * j8);
                        if (id == ad) low_rank8(a, g.s, GU ? 2 : 1, pos, proj, j8, scale, rank, hi, lo);
                    }
                    d = mfma16(w, hi, d);
                    d = mfma16(w, lo, d);
                }
                if (id == ad) acc[f] += d;
            }
        }
    }
#pragma unroll
    for (int f = 0; f < TF; ++f)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[wave][f][i16][4 * q + v] = acc[f][v];       // [token][row]
    __syncthreads();
    constexpr int NR = GU ? 8 : 16;
    for (int e = threadIdx.x; e < TF * 16 * NR; e += 512) {
        const int r = e % NR, tok = e / NR, f = tok >> 4, c = tok & 15;
        if (tok >= a.T || r0 + r >= g.N) continue;
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) y += red[w][f][c][r];
        const int64_t o = (int64_t)tok * g.N + r0 + r;
        if constexpr (GU) {
            float up = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) up += red[w][f][c][r + 8];
            const float h = silu_mul(y, up);
            g.h[o] = __builtin_bit_cast(uint16_t, (__bf16)h);
            if (g.hp == 2) g.h[(int64_t)a.T * g.N + o] = __builtin_bit_cast(uint16_t, (__bf16)bf16_rest(h));
        } else {
            if (g.out_bf16) static_cast<__bf16 *>(g.out)[o] = (__bf16)y;
            else static_cast<float *>(g.out)[o] = y;
        }
    }
}

// ---------------------------------------------------------------------------
// Many tokens: a workgroup of four waves computes 128 weight rows (gate/up: 64 of each) x BT tokens, each wave 64 x BT/2
// of them; both operands pass through LDS in 64-wide K stages, three of them, filled by direct-to-LDS loads.
// LDS rows are 128 bytes; 16-byte chunk c of row r lies at position c ^ (r & 7), so eight rows' reads of one chunk
// column touch all banks once.
//
// The loads are written as assembly: the compiler would otherwise wait for all of them before any LDS read.  They
// have no register outputs; wait_stage() counts them (the kernel has no other vector memory access between the first
// issue and the last stage) and orders the workgroup.
// ---------------------------------------------------------------------------
template <int N> __device__ __forceinline__ void wait_stage() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 64 lanes' 16 bytes at their `src` -> 1 KiB of LDS at byte address `dst` (wave-uniform), in lane order.  The
// destination goes through m0, which is put back: the compiler may count on its value.
__device__ __forceinline__ void load_to_lds(const void *src, uint32_t dst) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off\n\t"
                 "s_mov_b32 m0, %0"
                 : "=&s"(m0) : "v"(src), "s"(dst) : "memory");
}

constexpr int BW = 128, BK = 64, STAGES = 3;

template <bool GU, int P, int BT>
__global__ __launch_bounds__(256) void k_many(SharedArgs a, Product g, int tiles_w, int tiles_t) {
    constexpr int WT = 2;                                    // waves along the tokens, and along the weight rows
    constexpr int FW = BW / 2 / 32, FT = BT / WT / 32;       // 32 x 32 fragments per wave
    constexpr int ROWS = BW + BT, LOADS = ROWS / 8 / 4;      // direct-to-LDS loads (8 rows each) per wave and stage
    __shared__ __attribute__((aligned(1024))) uint4 tile[STAGES][ROWS * 8];
    const int lane = threadIdx.x & 63, i32 = lane & 31, hh = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int K = g.K;
    // XCD-aware order: consecutive workgroups go to the eight XCDs in turn; each XCD takes a run of tiles with the
    // token tile fastest, so the workgroups that read the same weight rows share an L2
    const int total = tiles_w * tiles_t, per = (total + 7) / 8;
    const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
    const int tw = id / tiles_t, tt = id - tw * tiles_t;
    const int w0 = tw * (GU ? BW / 2 : BW), t0 = tt * BT;

    // this lane's global rows: load i of this wave fills tile rows 8 * (wave * LOADS + i) .. + 7
    const uint16_t *src[LOADS];
    const int chunk = (lane & 7) ^ (lane >> 3);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = 8 * (wave * LOADS + i) + (lane >> 3);
        if (r < BW) {
            // gate/up: rows come in 32-row groups gate, up, gate, up so that a wave holds both of the same rows
            const int m = GU ? (r >> 5) & 1 : 0, wr = GU ? w0 + (r >> 6) * 32 + (r & 31) : w0 + r;
            src[i] = g.w[m] + (int64_t)min(wr, g.N - 1) * K;
        } else {
            const int pos = min(t0 + r - BW, a.T - 1);
            src[i] = g.x + (int64_t)(g.gather && a.sorted ? a.perm[pos] : pos) * K;
        }
        src[i] += 8 * chunk;
    }
    const int nsteps = (K + BK - 1) / BK * P;
    const int64_t plane = (int64_t)a.T * K;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(las_ptr)tile + wave * LOADS * 1024u;
    const uint16_t *zeros = reinterpret_cast<const uint16_t *>(&zero_chunk);
    asm("" : "+v"(zeros));                                   // kept in registers: a select below, not a branch
    // Loads of the next stage to issue: its K offset and plane.  Past the end of the last row, and in stages behind the last,
    // they read zeros, so that every stage has the same number of loads in flight.
    int ik = 0, ip = 0;
    bool in = 8 * chunk < K;
    uint32_t idst = lds0;
    auto issue = [&](int i) {                                // i: load of this wave (compile-time)
        const uint16_t *q = src[i] + ik;
        if (P > 1 && (wave * LOADS + i) * 8 >= BW) q += ip ? plane : 0;
        load_to_lds(in ? q : zeros, idst + i * 1024u);
    };
    auto next_stage = [&]() {
        ik += BK;
        if (P > 1 && ip == 0 && ik >= K) { ik = 0; ip = 1; }
        in = ik + 8 * chunk < K;
        idst = idst == lds0 + (STAGES - 1) * ROWS * 128u ? lds0 : idst + ROWS * 128u;
    };
    f32x16_t acc[FW][FT];
#pragma unroll
    for (int i = 0; i < FW; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int rw = (wave / WT) * FW * 32, rt = BW + (wave % WT) * FT * 32;
    uint4 fw[2][FW], ft[2][FT];
    auto read = [&](const uint4 *t, int kk, int b) {
        const int c = (2 * kk + hh) ^ (i32 & 7);
#pragma unroll
        for (int i = 0; i < FW; ++i) fw[b][i] = t[(rw + i * 32 + i32) * 8 + c];
#pragma unroll
        for (int j = 0; j < FT; ++j) ft[b][j] = t[(rt + j * 32 + i32) * 8 + c];
    };
    // the products of one 16-wide slice, with a quarter of a stage's loads issued among them
    auto products = [&](int b, int quarter) {
        constexpr int M = FW * FT;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            acc[m % FW][m / FW] = mfma32(fw[b][m % FW], ft[b][m / FW], acc[m % FW][m / FW]);
            const int l0 = quarter * LOADS / 4, n = (quarter + 1) * LOADS / 4 - l0;
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                if (i >= l0 + m * n / M && i < l0 + (m + 1) * n / M) issue(i);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Stages 0 and 1 and the first quarter of stage 2 are loaded ahead.  Fragments of the next slice are read while the
    // matrix cores work on the present one.  Before a stage's last slice: wait for the next stage (the one after it stays
    // in flight) and for the workgroup; from then on nobody reads the present stage's buffer, and it takes the loads of
    // the stage three further on.
#pragma unroll
    for (int i = 0; i < LOADS; ++i) issue(i);
    next_stage();
#pragma unroll
    for (int i = 0; i < LOADS; ++i) issue(i);
    next_stage();
#pragma unroll
    for (int i = 0; i < LOADS / 4; ++i) issue(i);
    wait_stage<LOADS + LOADS / 4>();
    int rb = 0;
    read(tile[0], 0, 0);
    for (int s = 0; s < nsteps; ++s) {
        const uint4 *t = tile[rb];
#pragma unroll
        for (int kk = 0; kk < 3; ++kk) {
            read(t, kk + 1, (kk + 1) & 1);
            products(kk & 1, kk + 1);
        }
        next_stage();
        rb = rb == STAGES - 1 ? 0 : rb + 1;
        wait_stage<LOADS>();
        read(tile[rb], 0, 0);                                // behind the last stage: zeros, not used
        products(1, 0);
    }
    wait_stage<0>();
    // D: lane holds token i32 of a fragment, weight rows 8 * (v / 4) + 4 * hh + v % 4
    const int np = GU ? 2 : 1;
#pragma unroll
    for (int j = 0; j < FT; ++j) {
        const int pos = t0 + (rt - BW) + j * 32 + i32;
        if (a.n) {
            const int id = adapter_at(a, pos);
            unsigned long long left = __ballot(id >= 0);
            while (left) {
                const int ad = __shfl(id, __ffsll(left) - 1, 64);
                left &= ~__ballot(id == ad);
                const float scale = a.scale ? a.scale[ad] : 1.f;
                const int rank = rank_of(a, ad);
                f32x16_t d[FW];
#pragma unroll
                for (int i = 0; i < FW; ++i)
#pragma unroll
                    for (int v = 0; v < 16; ++v) d[i][v] = 0.f;
                for (int c0 = 0; 8 * c0 < rank; c0 += 2) {
                    const int j8 = c0 + hh;
                    const bool in = 8 * j8 < rank;
                    uint4 hi[2], lo[2];
#pragma unroll
                    for (int p = 0; p < np; ++p) {
                        hi[p] = lo[p] = make_uint4(0, 0, 0, 0);
                        if (in && id == ad && g.b[p])
                            low_rank8(a, g.s, np, pos, p, j8, scale, rank, hi[p], lo[p]);
                    }
#pragma unroll
                    for (int i = 0; i < FW; ++i) {
                        const int m = GU ? i & 1 : 0;
                        const int wr = GU ? w0 + (rw >> 6) * 32 + i32 : w0 + rw + i * 32 + i32;
                        uint4 w = make_uint4(0, 0, 0, 0);
                        if (in && wr < g.N && g.b[m])
                            w = keep_first(load16(g.b[m] + ((int64_t)ad * g.N + wr) * a.R + 8 * j8), rank - 8 * j8);
                        d[i] = mfma32(w, hi[m], d[i]);
                        d[i] = mfma32(w, lo[m], d[i]);
                    }
                }
                if (id == ad) {
#pragma unroll
                    for (int i = 0; i < FW; ++i) acc[i][j] += d[i];
                }
            }
        }
        if (pos >= a.T) continue;
        if constexpr (GU) {
            const int64_t row = (int64_t)pos * g.N;
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4) {
                const int wr = w0 + (rw >> 6) * 32 + 8 * v4 + 4 * hh;
                if (wr >= g.N) continue;
                float h[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) h[v] = silu_mul(acc[0][j][4 * v4 + v], acc[1][j][4 * v4 + v]);
                *reinterpret_cast<uint2 *>(g.h + row + wr) = make_uint2(pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]));
                if (g.hp == 2)
                    *reinterpret_cast<uint2 *>(g.h + (int64_t)a.T * g.N + row + wr) =
                        make_uint2(pack_bf16(bf16_rest(h[0]), bf16_rest(h[1])),
                                   pack_bf16(bf16_rest(h[2]), bf16_rest(h[3])));
            }
        } else {
            const int64_t row = (int64_t)(a.sorted ? a.perm[pos] : pos) * g.N;
#pragma unroll
            for (int i = 0; i < FW; ++i)
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    const int wr = w0 + rw + i * 32 + 8 * v4 + 4 * hh;
                    if (wr >= g.N) continue;
                    const f32x16_t &y = acc[i][j];
                    if (g.out_bf16)
                        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(g.out) + row + wr) =
                            make_uint2(pack_bf16(y[4 * v4], y[4 * v4 + 1]), pack_bf16(y[4 * v4 + 2], y[4 * v4 + 3]));
                    else
                        *reinterpret_cast<float4 *>(static_cast<float *>(g.out) + row + wr) =
                            make_float4(y[4 * v4], y[4 * v4 + 1], y[4 * v4 + 2], y[4 * v4 + 3]);
                }
        }
    }
}

template <bool GU, int P>
hipError_t launch_product(const SharedArgs &a, const Product &g, hipStream_t st) {
    const int T = a.T;
    if (T <= FEW_TOKENS) {
        const dim3 grd((unsigned)((g.N + (GU ? 7 : 15)) / (GU ? 8 : 16))), blk(512);
        if (T <= 16) hipLaunchKernelGGL((k_few<GU, P, 1>), grd, blk, 0, st, a, g);
        else if (T <= 32) hipLaunchKernelGGL((k_few<GU, P, 2>), grd, blk, 0, st, a, g);
        else hipLaunchKernelGGL((k_few<GU, P, 4>), grd, blk, 0, st, a, g);
        return hipGetLastError();
    }
    const int rows = GU ? BW / 2 : BW, tw = (g.N + rows - 1) / rows;
    const dim3 blk(256);
    auto tiles = [&](int bt) { return tw * ((T + bt - 1) / bt); };
    const int bt = tiles(256) >= 256 ? 256 : tiles(128) >= 256 ? 128 : 64;
    const dim3 grd((unsigned)((tiles(bt) + 7) / 8 * 8));
    const int tt = (T + bt - 1) / bt;
    if (bt == 256) hipLaunchKernelGGL((k_many<GU, P, 256>), grd, blk, 0, st, a, g, tw, tt);
    else if (bt == 128) hipLaunchKernelGGL((k_many<GU, P, 128>), grd, blk, 0, st, a, g, tw, tt);
    else hipLaunchKernelGGL((k_many<GU, P, 64>), grd, blk, 0, st, a, g, tw, tt);
    return hipGetLastError();
}

template <int P>
hipError_t launch_low_rank(const SharedArgs &a, const LowRank &L, hipStream_t st) {
    const int nd = a.T < a.n ? a.T : a.n;
    if (a.sorted) {
        const dim3 grd((unsigned)(a.T / ITEM_TOKENS + nd), (unsigned)a.ks);
        hipLaunchKernelGGL((k_low_rank<P, true>), grd, dim3(256), 0, st, a, L);
    } else {
        hipLaunchKernelGGL((k_low_rank<P, false>), dim3((unsigned)nd, (unsigned)a.ks), dim3(256), 0, st, a, L);
    }
    return hipGetLastError();
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

// Workspace layout, from the shapes and types alone.
struct Layout {
    size_t x, perm, ad, items, n_items, s, h, total;
};
Layout layout(int T, int H, int Is, int n, int R, int ks, bool x_f32, int hp) {
    Layout l;
    size_t o = 0;
    auto take = [&](size_t b) { const size_t at = o; o += up256(b); return at; };
    const bool sorted = n > 0 && T > FEW_TOKENS;
    const size_t nd = (size_t)(T < n ? T : n);
    l.x = take(x_f32 ? (size_t)T * H * 4 : 0);
    l.perm = take(sorted ? (size_t)T * 4 : 0);
    l.ad = take(sorted ? (size_t)T * 4 : 0);
    l.items = take(sorted ? ((size_t)T / ITEM_TOKENS + nd) * 16 : 0);
    l.n_items = take(sorted ? 4 : 0);
    l.s = take(n > 0 ? (size_t)ks * T * 2 * R * 4 : 0);      // gate/up's, then down's
    l.h = take((size_t)T * Is * 2 * hp);
    l.total = o;
    return l;
}

// K splits of the down-rank products: enough workgroups for the 256 CUs, at most 8 partial sums for the reader.
int low_rank_splits(int T, int n) {
    if (!n) return 0;
    const int nd = T < n ? T : n, items = T > FEW_TOKENS ? T / ITEM_TOKENS + nd : nd;
    int ks = 1;
    while (ks < 8 && ks * items < 256) ks *= 2;
    return ks;
}

}  // namespace

namespace moe {

size_t shared_workspace(int T, int H, int Is, int n, int R) {
    // the largest over the activation and result types, so that one buffer serves every call of these sizes
    return layout(T, H, Is, n, R, low_rank_splits(T, n), true, 2).total;
}

hipError_t launch_shared(SharedArgs a, void *ws, hipStream_t st) {
    char *base = static_cast<char *>(ws);
    const int hp = a.out_bf16 ? 1 : 2;
    a.ks = low_rank_splits(a.T, a.n);
    a.sorted = a.n > 0 && a.T > FEW_TOKENS;
    const Layout l = layout(a.T, a.H, a.Is, a.n, a.R, a.ks, !a.x_bf16, hp);
    const uint16_t *x = static_cast<const uint16_t *>(a.x);
    hipError_t e;
    if (!a.x_bf16) {
        uint16_t *planes = reinterpret_cast<uint16_t *>(base + l.x);
        const int64_t n = (int64_t)a.T * a.H;
        hipLaunchKernelGGL(k_split, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, st,
                           static_cast<const float *>(a.x), planes, n);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        x = planes;
    }
    if (a.sorted) {
        a.perm = reinterpret_cast<int32_t *>(base + l.perm);
        a.plan_ad = reinterpret_cast<int32_t *>(base + l.ad);
        a.items = reinterpret_cast<int4 *>(base + l.items);
        a.n_items = reinterpret_cast<int32_t *>(base + l.n_items);
        hipLaunchKernelGGL(k_plan, dim3(1), dim3(PLAN_THREADS), 0, st, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    float *s = reinterpret_cast<float *>(base + l.s);
    uint16_t *h = reinterpret_cast<uint16_t *>(base + l.h);
    LowRank lx = {x, a.H, 2, 1, {a.gate_a, a.up_a}, s}, lh = {h, a.Is, 1, 0, {a.down_a, nullptr}, s};
    Product gu = {}, dn = {};
    gu.x = x; gu.K = a.H; gu.N = a.Is; gu.gather = 1;
    gu.w[0] = a.gate; gu.w[1] = a.up; gu.b[0] = a.gate_b; gu.b[1] = a.up_b; gu.s = s; gu.h = h; gu.hp = hp;
    dn.x = h; dn.K = a.Is; dn.N = a.H; dn.gather = 0;
    dn.w[0] = a.down; dn.b[0] = a.down_b; dn.s = s; dn.out = a.out; dn.out_bf16 = a.out_bf16;
    SharedArgs ag = a, ad = a;                              // a half without adapters runs as if there were none
    if (!a.gate_a && !a.up_a) ag.n = 0;
    if (!a.down_a) ad.n = 0;
    if (ag.n && (e = a.x_bf16 ? launch_low_rank<1>(ag, lx, st) : launch_low_rank<2>(ag, lx, st)) != hipSuccess) return e;
    if ((e = a.x_bf16 ? launch_product<true, 1>(ag, gu, st) : launch_product<true, 2>(ag, gu, st)) != hipSuccess) return e;
    if (ad.n && (e = hp == 1 ? launch_low_rank<1>(ad, lh, st) : launch_low_rank<2>(ad, lh, st)) != hipSuccess) return e;
    return hp == 1 ? launch_product<false, 1>(ad, dn, st) : launch_product<false, 2>(ad, dn, st);
}

}  // namespace moe
