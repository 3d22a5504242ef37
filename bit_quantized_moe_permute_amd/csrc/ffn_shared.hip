// The shared expert as a call of its own, with low-rank adapters of many requests (moe_shared_ffn):
//
//   g = Wg x + c_a Bg_a (Ag_a x),  u likewise,  h = silu(g) * u,  out = Wd h + c_a Bd_a (Ad_a h)
//
// with a = token_adapter[t] (no adapter terms where it is outside 0 .. n_adapters - 1).  All products run on the bf16
// matrix cores with fp32 sums.  What is not bf16 by itself -- fp32 activations, the low-rank results, and h -- is carried as bf16
// parts and multiplied part by part: three (24 bits) where the result is fp32, two (16 bits) where it is bf16.
// Launches: [plan] [down-rank] gate/up [down-rank] down --
//
//   plan       (many tokens) the tokens ordered by adapter, and work items of up to 64 tokens of one adapter
//   down-rank  s[t][r] = c_a (A_a[r] . x[t]) for each token's own adapter
//   gate/up    weight rows x tokens; the adapters' B_a s in the epilogue; SwiGLU; h
//   down       the same product with Wd and h
//
// An adapter's term is formed in accumulators of its own and added to the rows of its own tokens only, so nothing of
// one request's adapter (not even a NaN) reaches another request.
//
// Bound: the weights' bytes for few tokens, the matrix cores and the tiles' way into LDS for many.  hidden 4096, inter 2048,
// kernels alone, medians (a copy reaches 4.85 to 4.97 TB/s on this chip, a 2048 x 4096 x 4096 library product takes 62 us):
//   1 token, rank 16:     inputs 3.8 us, gate/up 10.6 (33.6 MB, 3.2 TB/s), down 9.3 (16.9 MB, 1.8 TB/s)
//   24 requests, rank 64: inputs 7.3, gate/up 15.2, inputs 4.8, down 11.8 (together 100 MB in 39.1 us, 2.6 TB/s)
//   512 tokens, rank 16, fp32 out: plan 4.8, down-rank 6.6 + 6.0, gate/up 29 to 38 from run to run (0.45 to 0.6 PFLOP/s),
//                         down-rank 6.8 + 6.2, down 29 (three planes: 0.9 PFLOP/s)
//   2048 tokens, rank 32, bf16 out: plan 6.2, down-rank 11 + 6.6, gate/up 81 to 87 (0.8 PFLOP/s), down-rank 9.4 + 6.4, down 81
//                         to 87 (two planes: 0.8)
//   the same, fp32 out:   down-rank 13 + 6.1, down 135 (three planes: 0.8), the others as before
#include <algorithm>

#include "common.h"
#include "internal.h"

using namespace moe;

namespace {

typedef __attribute__((address_space(3))) void *las_ptr;

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

// Part p of 3 of a value: three bf16 parts, each the rounded rest of those before, hold all 24 bits of an fp32 value.
__device__ __forceinline__ float bf16_part(float v, int p) { return p == 0 ? v : p == 1 ? bf16_rest(v) : bf16_rest(bf16_rest(v)); }
__device__ __forceinline__ uint4 pack_part(const float (&v)[8], int p) {
    return make_uint4(pack_bf16(bf16_part(v[0], p), bf16_part(v[1], p)), pack_bf16(bf16_part(v[2], p), bf16_part(v[3], p)),
                      pack_bf16(bf16_part(v[4], p), bf16_part(v[5], p)), pack_bf16(bf16_part(v[6], p), bf16_part(v[7], p)));
}
__device__ __forceinline__ uint2 pack_part(const float (&v)[4], int p) {
    return make_uint2(pack_bf16(bf16_part(v[0], p), bf16_part(v[1], p)), pack_bf16(bf16_part(v[2], p), bf16_part(v[3], p)));
}
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// c + sum of eight products of bf16 values, fp32
__device__ __forceinline__ float dot8(uint4 a, uint4 b, float c) {
    c = dot2_bf16(__builtin_bit_cast(bf16x2_t, a.x), __builtin_bit_cast(bf16x2_t, b.x), c);
    c = dot2_bf16(__builtin_bit_cast(bf16x2_t, a.y), __builtin_bit_cast(bf16x2_t, b.y), c);
    c = dot2_bf16(__builtin_bit_cast(bf16x2_t, a.z), __builtin_bit_cast(bf16x2_t, b.z), c);
    return dot2_bf16(__builtin_bit_cast(bf16x2_t, a.w), __builtin_bit_cast(bf16x2_t, b.w), c);
}

// Eight products of bf16 and fp32 values into two sums
__device__ __forceinline__ void dot8_f32(uint4 a, uint4 lo, uint4 hi, float (&c)[2]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w}, x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[0] = __fmaf_rn(__uint_as_float(w[i] << 16), __uint_as_float(x[2 * i]), c[0]);
        c[1] = __fmaf_rn(__uint_as_float(w[i] & 0xFFFF0000u), __uint_as_float(x[2 * i + 1]), c[1]);
    }
}

// The first `n` of eight bf16 values, the others zero.
__device__ __forceinline__ uint4 keep_first(uint4 v, int n) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 2 * i + 1 < n ? w[i] : 2 * i < n ? w[i] & 0xFFFFu : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int N> __device__ __forceinline__ void wait_stage() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 64 lanes' 16 bytes at base + off -> 1 KiB of LDS at byte address `dst` (wave-uniform), in lane order.  The destination
// goes through m0, which is put back: the compiler may count on its value.
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32 |
           (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
}
__device__ __forceinline__ void load_to_lds(uint64_t base, uint32_t off, uint32_t dst) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0) : "v"(off), "s"(base), "s"(dst) : "memory");
}

// A value at a wave-uniform place, through the scalar cache: its wait is apart from that for the vector loads in flight.
template <typename T> __device__ __forceinline__ T uniform_at(const T *p, int64_t i) {
    return reinterpret_cast<const __attribute__((address_space(4))) T *>(reinterpret_cast<uintptr_t>(p))[i];
}

__device__ __forceinline__ int rank_of(const SharedArgs &a, int ad) {
    return a.rank ? min(max(uniform_at(a.rank, ad), 0), a.R) : a.R;
}

// Adapter of row `pos` (sorted position with a plan, else token), -1 for none.
__device__ __forceinline__ int adapter_at(const SharedArgs &a, int pos) {
    if (!a.n || pos >= a.T) return -1;
    const int id = a.sorted ? a.plan_ad[pos] : a.token_adapter[pos];
    return (unsigned)id < (unsigned)a.n ? id : -1;
}

// Row `pos` of the low-rank results of projection `proj` of `np`: [3 parts][R] bf16, scaled, zero from the adapter's rank on.
__device__ __forceinline__ const uint16_t *low_rank_row(const SharedArgs &a, const uint16_t *s, int np, int pos, int proj) {
    return s + ((int64_t)pos * np + proj) * 3 * a.R;
}

// ---------------------------------------------------------------------------
// plan (many tokens): tokens ordered by adapter (those without one last), and items of up to ITEM_TOKENS tokens of one adapter.
// One workgroup; the launch's others bring fp32 activations into xp bf16 planes [xp][T][H].  Within an adapter the order is that
// of LDS atomics and may differ between calls: a row's place in a tile changes no bit of its result.  Bound by its chain of
// loads, LDS atomics and barriers: 4.8 us for 512 tokens, 5.8 for 2048, of which a launch alone is about 3.
// ---------------------------------------------------------------------------
constexpr int PLAN_THREADS = 1024;

__global__ __launch_bounds__(PLAN_THREADS) void k_plan(SharedArgs a, uint16_t *planes, int xp, int plans) {
    if ((int)blockIdx.x >= plans) {
        const int64_t i = 4 * ((int64_t)(blockIdx.x - plans) * PLAN_THREADS + threadIdx.x), m = (int64_t)a.T * a.H;
        if (i >= m) return;
        const float4 x = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.x) + i);
        const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int p = 0; p < 3; ++p)
            if (p < xp) *reinterpret_cast<uint2 *>(planes + p * m + i) = pack_part(v, p);
        return;
    }
    __shared__ int count[MAX_ADAPTERS + 1], begin[MAX_ADAPTERS + 2], item0[MAX_ADAPTERS + 1], wsum[2][PLAN_THREADS / 64];
    const int n = a.n, tid = threadIdx.x;
    for (int i = tid; i <= n; i += PLAN_THREADS) count[i] = 0;
    constexpr int HELD = 4;                                          // tokens per thread whose bin stays in a register
    int bin[HELD];
    auto bin_of = [&](int t) {
        const int id = t < a.T ? a.token_adapter[t] : -1;
        return (unsigned)id < (unsigned)n ? id : n;
    };
#pragma unroll
    for (int j = 0; j < HELD; ++j) bin[j] = bin_of(tid + j * PLAN_THREADS);
    __syncthreads();
    // a wave whose tokens all have one bin (runs of one request) adds once
    auto add = [&](int t, int b) -> int {
        const unsigned long long in = __ballot(t < a.T);
        if (in == 0) return 0;
        const int b0 = __builtin_amdgcn_readfirstlane(b);
        if (__ballot(t < a.T && b != b0) == 0) {
            int base = 0;
            if ((tid & 63) == 0) base = atomicAdd(&count[b0], __popcll(in));
            return __builtin_amdgcn_readfirstlane(base) + (tid & 63);
        }
        return t < a.T ? atomicAdd(&count[b], 1) : 0;
    };
#pragma unroll
    for (int j = 0; j < HELD; ++j) add(tid + j * PLAN_THREADS, bin[j]);
    for (int t = tid + HELD * PLAN_THREADS; t - tid < a.T; t += PLAN_THREADS) add(t, bin_of(t));
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
        count[b] = begin[b] = btok;                                  // the bin's cursor, its first position, its first item
        item0[b] = bit;
        btok += c[j];
        if (b < n) bit += (c[j] + ITEM_TOKENS - 1) / ITEM_TOKENS;
        if (b == n) begin[n + 1] = btok;
    }
    if (tid == PLAN_THREADS - 1) *a.n_items = bit;
    __syncthreads();
    auto place = [&](int t, int b) {
        const int pos = add(t, b);
        if (t >= a.T) return;
        a.perm[pos] = t;
        a.plan_ad[pos] = b < n ? b : -1;
        const int i = pos - begin[b];                                // every ITEM_TOKENS-th position opens an item
        if (b < n && i % ITEM_TOKENS == 0)
            a.items[item0[b] + i / ITEM_TOKENS] = make_int4(b, pos, min(ITEM_TOKENS, begin[b + 1] - pos), 0);
    };
#pragma unroll
    for (int j = 0; j < HELD; ++j) place(tid + j * PLAN_THREADS, bin[j]);
    for (int t = tid + HELD * PLAN_THREADS; t - tid < a.T; t += PLAN_THREADS) place(t, bin_of(t));
}

// ---------------------------------------------------------------------------
// Few tokens: what a product reads of its activations.
//
// Tokens go in groups of up to 64.  Packed activations [group][P][TF][steps][64 lanes][8]: the matrix instruction's operand of
// 16 tokens and 32 of K in lane order, so that a wave reads 1 KiB in a row.  Lane l holds token l % 16 and k = 8 (l / 16) .. + 7;
// steps of 32 up to a multiple of 2048, zeros behind the end of K.
// Read from rows instead, the 64 lanes' 16-byte pieces would lie in 64 places, and a wave's load would take four times as
// long (64 requests, 4096 x 2048: gate/up 43 us reading rows, 22 with packed operands; down 33 and 17).
//
// Low-rank results s[t][proj][3 parts][r] = scale_a (A_a[r] . x[t]), one wave per (token, row): no wait but that for the token's
// adapter index and that for the row, and no exchange but the wave's own sum.
// ---------------------------------------------------------------------------
// TF: fragments of 16 tokens, rounded up to what the kernels are built for; those behind the last token hold anything.
__host__ __device__ __forceinline__ int few_frags(int T) { return T <= 16 ? 1 : T <= 32 ? 2 : 4; }

__host__ __device__ __forceinline__ int few_groups(int T) { return (T + FEW_TOKENS - 1) / FEW_TOKENS; }
constexpr int FEW_ROUND = 2048;
__host__ __device__ __forceinline__ int few_steps(int K) { return (K + FEW_ROUND - 1) / FEW_ROUND * (FEW_ROUND / 32); }

// PL: bf16 planes that fp32 activations are packed as; 1: they are bf16.
template <bool F32, int PL>
__global__ __launch_bounds__(256) void k_few_inputs(SharedArgs a, LowRank L, uint16_t *packed, int pack_blocks) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int K = L.K, steps = few_steps(K);
    if ((int)blockIdx.x < pack_blocks) {
        const int i = blockIdx.x * 4 + wave, tf = few_frags(a.T), frag = i / steps, step = i - frag * steps;
        const int grp = frag / tf, f = frag - grp * tf;
        if (frag * 16 >= a.T) return;
        const int t = frag * 16 + (lane & 15), k = step * 32 + 8 * (lane >> 4);
        uint4 *o = reinterpret_cast<uint4 *>(packed) + ((int64_t)(grp * PL * tf + f) * steps + step) * 64 + lane;
        const bool in = t < a.T && k < K;
        if constexpr (F32) {
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f), w = u;
            if (in) {
                const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(L.xv) + (int64_t)t * K + k);
                u = src[0];
                w = src[1];
            }
            const float v[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
            for (int p = 0; p < PL; ++p) o[(int64_t)p * tf * steps * 64] = pack_part(v, p);
        } else {
            o[0] = in ? load16(static_cast<const uint16_t *>(L.xv) + (int64_t)t * K + k) : make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const int nrows = L.np * a.R, id = (blockIdx.x - pack_blocks) * 4 + wave;
    if (id >= a.T * nrows) return;
    const int t = id / nrows, rr = id - t * nrows, proj = rr / a.R, r = rr - proj * a.R;
    const int token_ad = uniform_at(a.token_adapter, t), ad = (unsigned)token_ad < (unsigned)a.n ? token_ad : -1;
    const uint16_t *A = proj ? L.a[1] : L.a[0];
    if (ad < 0 || !A) return;                                // not read either
    A += ((int64_t)ad * a.R + r) * K;
    const int64_t row = (int64_t)t * K;
    constexpr int U = F32 ? 4 : 8, V = F32 ? 2 : 1;
    float acc[2] = {0.f, 0.f};
    for (int k0 = 0; k0 < K; k0 += U * 512) {
        uint4 w[U], v[V][U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int k = k0 + j * 512 + lane * 8;
            const bool in = k < K;
            w[j] = in ? load16(A + k) : make_uint4(0, 0, 0, 0);
            if constexpr (F32) {
                const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const float *>(L.xv) + row + k);
                v[0][j] = in ? x[0] : make_uint4(0, 0, 0, 0);
                v[1][j] = in ? x[1] : make_uint4(0, 0, 0, 0);
            } else {
                v[0][j] = in ? load16(static_cast<const uint16_t *>(L.xv) + row + k) : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if constexpr (F32) dot8_f32(w[j], v[0][j], v[1][j], acc);
            else acc[0] = dot8(w[j], v[0][j], acc[0]);
        }
    }
    float y = wave_sum(acc[0] + acc[1]);
    y = r < rank_of(a, ad) ? y * (a.scale ? uniform_at(a.scale, ad) : 1.f) : 0.f;
    uint16_t *o = L.s + ((int64_t)t * L.np + proj) * 3 * a.R + r;
    if (lane < 3) o[lane * a.R] = bf16_bits(bf16_part(y, lane));
}

// ---------------------------------------------------------------------------
// Few tokens, a product: one workgroup streams 16 weight rows (gate/up: 8 gate rows and the same 8 of up) once. Its waves split
// K: in each round of 2048 a wave takes 256 of every row, through LDS of its own that direct-to-LDS loads fill with 512-byte
// pieces of rows. The first two rounds are issued together (128 KiB per workgroup, what a copy's rate times the memory's
// latency asks of a compute unit; 16 rows, so that 4096 x 2048 makes 256 workgroups). From then on the second buffer hides
// little: a round's activations are loaded behind the next round's weights, and one wait stands for both. Chunk c of row r lies
// at position c ^ r, so that sixteen rows' reads of one chunk column touch every bank once. The waves' sums meet in LDS. An
// adapter's term is formed per token in fp32, wave w taking tokens w, w + NW, ...; its loads go out with the weights'.
// ---------------------------------------------------------------------------
constexpr int FEW_WAVES = 8;

__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// AD: the adapters' low-rank results are read (AD_READ), or (AD_HERE, down, few values) formed by every workgroup from the rows
// of h. Their loads go out behind those of the first two rounds of weights and come back behind them, so that their products
// follow the stream rather than run beside it. That reads A out of the caches in every workgroup, where a launch between the
// two products costs 4 us. fp32 result, a launch against here, whole calls: 16 values of 512 16.4 and 14.2 us, of 2048 (1
// token, rank 16, hidden 4096) 24.4 and 22.8, of 4096 38.6 and 37.2; 32 values of 512 16.3 and 15.0, of 2048 24.6 and 24.5; 8
// of 8192 107.1 and 108.4.
enum { AD_NONE = 0, AD_READ = 1, AD_HERE = 2 };
constexpr int HERE_VALUES = 32, HERE_TERMS = 1 << 16;        // for AD_HERE at most: tokens * max_rank, and times inter

template <bool GU, int P, int TF, int AD>
__global__ __launch_bounds__(64 * FEW_WAVES) void k_few(SharedArgs a, Product g) {
    constexpr int NW = FEW_WAVES, SLICE = FEW_ROUND / NW;         // K of a wave per round
    constexpr int LINE = SLICE / 8, LOADS = 16 * LINE / 64;              // chunks of a row's piece; loads of 64 chunks
    constexpr int TW = TF * 16 / NW, NP = GU ? 2 : 1;                    // tokens per wave (adapters' terms)
    __shared__ __attribute__((aligned(1024))) uint4 ring[2][NW][16 * LINE];
    __shared__ float low[TF * 16][16];
    __shared__ float here[AD == AD_HERE ? HERE_VALUES : 1];
    f32x4_t (*red)[TF][64] = reinterpret_cast<f32x4_t (*)[TF][64]>(ring);         // after the last product
    static_assert(sizeof(f32x4_t) * NW * TF * 64 <= sizeof(ring), "");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i16 = lane & 15, q = lane >> 4;
    const int K = g.K, r0 = blockIdx.x * (GU ? 8 : 16), hsteps = few_steps(g.N);
    const int t0 = blockIdx.y * FEW_TOKENS;                              // this workgroup's tokens
    uint16_t *const h = g.h + (int64_t)blockIdx.y * g.hp * TF * hsteps * 512;
    if (GU && r0 >= g.N) {                                               // packed rows end in zeros
        for (int e = threadIdx.x; e < g.hp * TF * 16; e += 64 * NW) {
            const int f = e >> 4, c = e & 15;                            // f: plane and fragment
            reinterpret_cast<uint4 *>(h)[((int64_t)f * hsteps + r0 / 32) * 64 + r0 % 32 / 8 * 16 + c] = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    // Load j fills 64 / LINE rows' pieces: lane's row j * 64 / LINE + lane / LINE, chunk c = lane % LINE ^ row.
    constexpr int RPL = 64 / LINE;                                       // rows per load
    const uint64_t w0 = uniform64((uint64_t)(uintptr_t)(g.w[0] + (int64_t)r0 * K));
    const uint64_t w1 = GU ? uniform64((uint64_t)(uintptr_t)(g.w[1] + (int64_t)r0 * K)) : w0;
    const int row0 = lane / LINE, c0 = (lane % LINE) ^ row0;
    const uint32_t stride = 2u * (uint32_t)K, lds0 = (uint32_t)(uintptr_t)(las_ptr)ring + wave * (16u * LINE * 16u);
    const int rows = GU ? 8 : min(16, g.N - r0);
    auto issue = [&](int r, int b) __attribute__((always_inline)) {
        const int k = r * FEW_ROUND + wave * SLICE;
        if (k >= K) return;
        const bool whole = k + SLICE <= K;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const int jr = GU ? j % (LOADS / 2) * RPL : j * RPL;         // first row of the load in its matrix
            const int c = c0 ^ (j * RPL);
            // rows behind the last repeat it (their sums are not stored)
            uint32_t o = (uint32_t)(GU ? jr + row0 : min(jr + row0, rows - 1)) * stride + 2u * (uint32_t)k;
            // a chunk behind the row's end repeats the piece's first (its products meet zero activations)
            o += whole || k + 8 * c < K ? 16u * c : 0u;
            load_to_lds(GU && j >= LOADS / 2 ? w1 : w0, o, lds0 + b * (uint32_t)(sizeof(ring) / 2) + j * 1024u);
        }
    };
    // An adapter's term for token f * NW + wave: lane (row lr = lane / 4, lane % 4) takes rank values 8 (lane % 4) .. + 7 of each
    // 32, so that four lanes in a row read 64 bytes of one row of B.
    const int lr = lane >> 2, half = GU ? lr >> 3 : 0, wr = GU ? r0 + (lr & 7) : r0 + lr, r4 = 8 * (lane & 3);
    const uint16_t *const gb = half ? g.b[1] : g.b[0];
    const bool has = wr < g.N && gb;
    constexpr int FB = TF < 4 ? TW : 2;                                  // tokens at once (the registers of 64 tokens' first
    constexpr bool AHEAD = FB == TW;                                     // loads would be too many)
    int ad[TW], rank[TW];
    uint4 bw[TW], sv[TW][3];
    auto load_low = [&](int f0, int c) __attribute__((always_inline)) {
#pragma unroll
        for (int f = f0; f < f0 + FB; ++f) {
            bw[f] = sv[f][0] = sv[f][1] = sv[f][2] = make_uint4(0, 0, 0, 0);
            if (ad[f] < 0 || 32 * c >= rank[f]) continue;                // uniform
            if (has && 32 * c + r4 < rank[f]) {
                bw[f] = load16(gb + ((int64_t)ad[f] * g.N + wr) * a.R + 32 * c + r4);
                if constexpr (AD == AD_READ) {
                    const uint16_t *p = low_rank_row(a, g.s, NP, t0 + f * NW + wave, half) + 32 * c + r4;
#pragma unroll
                    for (int i = 0; i < 3; ++i) sv[f][i] = load16(p + i * a.R);
                }
            }
        }
    };
    f32x4_t acc[TF];
#pragma unroll
    for (int f = 0; f < TF; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    constexpr int SPW = SLICE / 32;                                      // steps of a wave per round
    constexpr int XB = TF * P <= 2 ? SPW : TF * P <= 4 ? SPW / 2 : TF * P <= 8 ? SPW / 4 : SPW / 8;   // steps whose activations are
                                                                         // loaded together
    const int rounds = (K + FEW_ROUND - 1) / FEW_ROUND, steps = few_steps(K);
    const uint4 *xw = reinterpret_cast<const uint4 *>(g.x) + (int64_t)blockIdx.y * P * TF * steps * 64 + wave * (SPW * 64) + lane;
    uint4 x[XB][TF][P];
    auto load_x = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
        for (int f = 0; f < TF; ++f)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const uint4 *src = xw + (int64_t)(p * TF + f) * steps * 64 + i0 * 64;
#pragma unroll
                for (int i = 0; i < XB; ++i) x[i][f][p] = src[i * 64];
            }
    };
    issue(0, 0);
    if (rounds > 1) issue(1, 1);
    if constexpr (AD == AD_HERE) {
        // here[t][r] = scale (A[r] . h[t]), two rows of A (of one token: R is even) per wave at a time
        for (int e = 2 * wave; e < a.T * a.R; e += 2 * NW) {
            const int t = e / a.R, r = e - t * a.R, id = uniform_at(a.token_adapter, t);
            const int rows_a = (unsigned)id < (unsigned)a.n ? rank_of(a, id) - r : 0;
            float y[2][2] = {};
            if (rows_a > 0) {
                const uint16_t *A = g.a + ((int64_t)id * a.R + r) * K;
                const float *hr = g.hrow + (int64_t)t * K;
                for (int k0 = lane * 8; k0 < K; k0 += 4 * 512) {
                    uint4 av[4][2], hv[4][2];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = k0 + i * 512 < K ? k0 + i * 512 : lane * 8;
                        const uint4 *h4 = reinterpret_cast<const uint4 *>(hr + k);
                        hv[i][0] = h4[0];
                        hv[i][1] = h4[1];
                        av[i][0] = load16(A + k);
                        av[i][1] = load16(A + K + k);                    // behind the rank: of no use
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (k0 + i * 512 < K) {
                            dot8_f32(av[i][0], hv[i][0], hv[i][1], y[0]);
                            dot8_f32(av[i][1], hv[i][0], hv[i][1], y[1]);
                        }
                }
            }
            const float scale = rows_a > 0 && a.scale ? uniform_at(a.scale, id) : 1.f;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float sum = wave_sum(y[v][0] + y[v][1]) * scale;
                if (lane == 0) here[e + v] = v < rows_a ? sum : 0.f;
            }
        }
    }
    for (int r = 0; r < rounds; ++r, xw += FEW_ROUND / 32 * 64) {
        const int b = r & 1;
        if (r == 0) {
            if constexpr (AD != AD_NONE) {
#pragma unroll
                for (int f = 0; f < TW; ++f) {
                    const int t = t0 + f * NW + wave, id = t < a.T ? uniform_at(a.token_adapter, t) : -1;
                    ad[f] = (unsigned)id < (unsigned)a.n ? id : -1;
                    rank[f] = ad[f] < 0 ? 0 : rank_of(a, ad[f]);
                }
                if (AD == AD_READ && AHEAD) load_low(0, 0);
            }
        }
        if (r * FEW_ROUND + wave * SLICE >= K) break;                    // no slice in this round or a later one
        const uint4 *const slice = ring[b][wave] + i16 * LINE;
#pragma unroll
        for (int i0 = 0; i0 < SPW; i0 += XB) {
            load_x(i0);
            if (i0 == 0) wait_loads();
#pragma unroll
            for (int i = 0; i < XB; ++i) {
                const uint4 w = slice[(4 * (i0 + i) + q) ^ i16];
#pragma unroll
                for (int f = 0; f < TF; ++f)
#pragma unroll
                    for (int p = 0; p < P; ++p) acc[f] = mfma16(w, x[i][f][p], acc[f]);
            }
        }
        if (r + 2 < rounds) {
            wait_reads();                                                // the slice is read
            issue(r + 2, b);
        }
    }
    if constexpr (AD == AD_HERE) __syncthreads();
    if constexpr (AD != AD_NONE) {
        float d[TW] = {};
#pragma unroll
        for (int f0 = 0; f0 < TW; f0 += FB)
            for (int c = 0; 32 * c < a.R; ++c) {
                if (AD == AD_HERE || c || !AHEAD) load_low(f0, c);
#pragma unroll
                for (int f = f0; f < f0 + FB; ++f) {
                    if (32 * c >= rank[f]) continue;
                    const uint4 w = rank[f] - 32 * c >= 32 ? bw[f] : keep_first(bw[f], rank[f] - 32 * c - r4);
                    if constexpr (AD == AD_HERE) {
                        const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
                        const float *sv = here + (f * NW + wave) * a.R + 32 * c + r4;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (32 * c + r4 + i < rank[f])
                                d[f] = __fmaf_rn(__uint_as_float(i & 1 ? wv[i / 2] & 0xFFFF0000u : wv[i / 2] << 16), sv[i], d[f]);
                    } else {
                        d[f] = dot8(w, sv[f][2], dot8(w, sv[f][1], dot8(w, sv[f][0], d[f])));
                    }
                }
            }
#pragma unroll
        for (int f = 0; f < TW; ++f) {
            d[f] += __shfl_xor(d[f], 1, 64);
            d[f] += __shfl_xor(d[f], 2, 64);
            if ((lane & 3) == 0) low[f * NW + wave][lr] = d[f];
        }
    }
    wait_loads();                                            // a wave without steps has none; the ring is free after the barrier
    __syncthreads();
#pragma unroll
    for (int f = 0; f < TF; ++f) red[wave][f][lane] = acc[f];            // lane: token i16, rows 4 q .. + 3
    __syncthreads();
    constexpr int NR = GU ? 8 : 16;
    for (int e = threadIdx.x; e < TF * 16 * NR; e += 64 * NW) {
        const int r = e % NR, tok = e / NR, f = tok >> 4, c = tok & 15;
        const int t = t0 + tok;
        if (t >= a.T) continue;
        float y = AD != AD_NONE ? low[tok][r] : 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) y += red[w][f][(r >> 2) * 16 + c][r & 3];
        if constexpr (GU) {
            float up = AD != AD_NONE ? low[tok][r + 8] : 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) up += red[w][f][(r >> 2) * 16 + 32 + c][r & 3];
            const int i = r0 + r;
            const float hv = silu_mul(y, up);
            const int64_t o = (((int64_t)f * hsteps + i / 32) * 64 + (i % 32 / 8) * 16 + c) * 8 + i % 8;
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                if (p >= g.hp) break;
                const uint16_t part = bf16_bits(bf16_part(hv, p));
                h[p * ((int64_t)TF * hsteps * 512) + o] = part;
            }
            if (g.hrow) g.hrow[(int64_t)t * g.N + i] = hv;                       // for the down-rank products
        } else {
            if (r0 + r >= g.N) continue;
            const int64_t o = (int64_t)t * g.N + r0 + r;
            if (g.out_bf16) static_cast<__bf16 *>(g.out)[o] = (__bf16)y;
            else static_cast<float *>(g.out)[o] = y;
        }
    }
}

// ---------------------------------------------------------------------------
// Many tokens: a workgroup computes BW weight rows (gate/up: half of each) x BT tokens (P planes of them, which meet the same
// weights), each wave 64 x BT/2 of them; both operands pass through LDS in 64-wide K stages, three of them (more gave nothing:
// 512 tokens the same with four or six), filled by direct-to-LDS loads. The matrix cores are busy half of the time at 2048
// tokens, with no LDS bank conflict: a 16-wide slice of 128 x 256 (or of 128 x 128 in two planes) takes 256 cycles of matrix
// instructions, and LDS 288 for the 24 KiB that its waves read and the 12 that arrive. Waves of 128 x 128 would read a third
// less, but leave half of the compute units without a tile there; twice the waves with half the tokens each ran the same (161
// and 162 us the whole call).
// LDS rows are 128 bytes, half of the 64 banks; 16-byte chunk c of row r lies at position c ^ (r / 2 % 8), so sixteen rows'
// reads of one chunk column touch every bank once.
//
// The loads are written as assembly: the compiler would otherwise wait for all of them before any LDS read.  They
// have no register outputs; wait_stage() counts them and orders the workgroup.  The kernel has no other vector memory access
// between the first issue and the last stage but for two registers that gate/up's tile of 128 x 256 spills (12 bytes of scratch);
// one more in flight would only make the counted wait a stricter one.
// ---------------------------------------------------------------------------
constexpr int BK = 64, STAGES = 3;
constexpr int many_split(int BT) { return BT == 64 ? 2 : 1; }
constexpr int many_threads(int BW, int BT) { return 64 * (BW / 64) * 2 * many_split(BT); }
enum { MODE_GATE_UP = 0, MODE_DOWN = 1, MODE_LOW_RANK = 2 };

// Down-rank (MODE_LOW_RANK): a tile's tokens are an item of the plan, its weight rows those of that adapter's A matrices, and
// blockIdx.y is a part of K; the sums of the parts are added by k_low_rank_sum.
// The tiles of 64 tokens have two groups of waves, each working two of a stage's four 16-wide slices: with one wave per SIMD
// and a few products per slice, the waits for LDS would stand open.
// TAIL: K is no multiple of 64, so a row's last step is not a whole one.
template <int MODE, int P, int BW, int BT, bool TAIL>
__global__ __launch_bounds__(many_threads(BW, BT)) void k_many(SharedArgs a, Product g, int tiles_w, int tiles_t) {
    constexpr bool GU = MODE == MODE_GATE_UP, LOW = MODE == MODE_LOW_RANK;
    constexpr int WT = 2;                                    // waves along the tokens, and along the weight rows
    constexpr int FW = 2, FT = BT / WT / 32;                 // 32 x 32 fragments per wave
    constexpr int GW = BW / 64 * WT;                         // waves of a group, which computes the tile from
    constexpr int KSP = many_split(BT), NS = 4 / KSP;        // NS of a stage's four slices; groups
    constexpr int ROWS = BW + P * BT, LOADS = ROWS / 8 / (GW * KSP);         // direct-to-LDS loads (8 rows each) per wave and stage
    __shared__ __attribute__((aligned(1024))) uint4 tile[STAGES][ROWS * 8];
    const int lane = threadIdx.x & 63, i32 = lane & 31, hh = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w4 = wave % GW, kk0 = wave / GW * NS;
    const int K = g.K;
    // XCD-aware order: consecutive workgroups go to the eight XCDs in turn; each XCD takes a run of tiles with the
    // token tile fastest, so the workgroups that read the same weight rows share an L2
    const int total = tiles_w * tiles_t, per = (total + 7) / 8;
    const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
    const int tw = id / tiles_t, tt = id - tw * tiles_t;
    const int w0 = tw * (GU ? BW / 2 : BW);
    int t0 = tt * BT, last = a.T - 1, ad0 = 0;               // first and last row of the tile's tokens
    if constexpr (LOW) {
        if (tt >= *a.n_items) return;
        const int4 it = a.items[tt];
        ad0 = it.x;
        t0 = it.y;
        last = it.y + it.z - 1;
    }

    // Load i of this wave fills rows 8 * (wave * LOADS + i) .. + 7 of the tile from one operand (`base`); `off`: byte offset of
    // this lane's row and chunk from there (n_tokens * K < 2^30 and the limits of K keep them below 2^32).
    // Rows behind the last repeat it; their results are not stored.
    const int tail = K % BK / 8;                             // chunks in a row's last step (TAIL)
    uint64_t base[LOADS];
    uint32_t off[LOADS], back[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r8 = 8 * (wave * LOADS + i), r = r8 + (lane >> 3), c = (lane & 7) ^ (r >> 1 & 7);
        const uint16_t *from = g.x;
        int row;
        if (LOW && r8 < BW) {
            // the adapter's rows [projection][R], eight of them in one projection; in a projection without adapters any
            // (its results are not read)
            const int rr = min(w0 + r8, g.N - 8), proj = rr / a.R;
            row = rr - proj * a.R + (lane >> 3);
            from = (proj ? (g.w[1] ? g.w[1] : g.w[0]) : (g.w[0] ? g.w[0] : g.w[1])) + (int64_t)ad0 * a.R * K;
        } else if (r8 < BW) {
            // gate/up: rows come in 32-row groups gate, up, gate, up so that a wave holds both of the same rows
            row = min(GU ? (r >> 6) * 32 + (r & 31) : r, g.N - 1 - w0);
            from = (GU && (r8 >> 5 & 1) ? g.w[1] : g.w[0]) + (int64_t)w0 * K;
        } else {
            const int p = (r8 - BW) / BT, pos = min(t0 + r - BW - p * BT, last);
            row = g.gather && a.sorted ? a.perm[pos] : pos;
            from = g.x + (int64_t)p * a.T * K;
        }
        base[i] = uniform64((uint64_t)(uintptr_t)from);
        off[i] = 2u * ((uint32_t)row * (uint32_t)K + 8u * c);
        back[i] = TAIL && c >= tail ? 16u * c : 0u;
    }
    const int ksteps = (K + BK - 1) / BK;
    // steps of this workgroup: all, or (down-rank) those of its part of K
    const int sb = LOW ? ksteps * (int)blockIdx.y / (int)gridDim.y : 0;
    const int se = LOW ? ksteps * ((int)blockIdx.y + 1) / (int)gridDim.y : ksteps;
    const int nsteps = se - sb;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(las_ptr)tile + wave * LOADS * 1024u;
    // Loads of the next stage to issue: its step, and its byte offset in a row.  A chunk behind the row's end repeats the step's
    // first one (its products meet zero weights), and stages behind the last repeat that: every stage has the same number of
    // loads in flight.
    int istep = sb;
    uint32_t ioff = 2 * BK * sb, idst = lds0;
    auto issue = [&](int i) {                                // i: load of this wave (compile-time)
        uint32_t o = off[i] + ioff;
        if (TAIL && istep == ksteps - 1) o -= back[i];
        load_to_lds(base[i], o, idst + i * 1024u);
    };
    auto next_stage = [&]() {
        if (istep + 1 < se) { ++istep; ioff += 2 * BK; }
        idst = idst == lds0 + (STAGES - 1) * ROWS * 128u ? lds0 : idst + ROWS * 128u;
    };
    f32x16_t acc[FW][FT];
#pragma unroll
    for (int i = 0; i < FW; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int rw = (w4 / WT) * FW * 32, rt = BW + (w4 % WT) * FT * 32;
    int idj[FT];                                             // adapters of this lane's tokens (loaded ahead of the stages)
#pragma unroll
    for (int j = 0; j < FT; ++j) idj[j] = LOW ? -1 : adapter_at(a, t0 + (rt - BW) + j * 32 + i32);
    uint4 fw[2][FW], ft[2][P * FT];
    auto read_one = [&](const uint4 *t, int kk, int b, int n) {      // fragment n of the slice: weights first
        const int c = (2 * kk + hh) ^ (i32 >> 1 & 7);
        if (n < FW) fw[b][n] = t[(rw + n * 32 + i32) * 8 + c];
        else ft[b][n - FW] = t[(rt + (n - FW) / FT * BT + (n - FW) % FT * 32 + i32) * 8 + c];
    };
    // The products of one 16-wide slice (buffer b).  Between them go the reads of the next slice and part `part` of NS of a
    // stage's loads, so that the matrix cores have work while these are issued.
    auto slice = [&](int b, const uint4 *nt, int nkk, int part) {
        constexpr int M = P * FW * FT, NR = FW + P * FT;
        const int l0 = part * LOADS / NS, nl = (part + 1) * LOADS / NS - l0;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            acc[m % FW][m / FW % FT] = mfma32(fw[b][m % FW], ft[b][m / FW], acc[m % FW][m / FW % FT]);
#pragma unroll
            for (int n = 0; n < NR; ++n)
                if (n >= m * 2 * NR / M && n < (m + 1) * 2 * NR / M) read_one(nt, nkk, b ^ 1, n);      // in the first half
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                if (i >= l0 + m * nl / M && i < l0 + (m + 1) * nl / M) issue(i);                     // towards the end
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Stages 0 and 1 and the first part of stage 2 are loaded ahead.  Before a stage's last slice: wait for the next stage
    // (the one after it stays in flight) and for the workgroup; from then on nobody reads the present stage's buffer, and
    // it takes the loads of the stage three further on.
#pragma unroll
    for (int i = 0; i < LOADS; ++i) issue(i);
    next_stage();
#pragma unroll
    for (int i = 0; i < LOADS; ++i) issue(i);
    next_stage();
#pragma unroll
    for (int i = 0; i < LOADS / NS; ++i) issue(i);
    // Weights behind the row's end count as zeros: in the last step's stage they are overwritten in LDS once it is there.
    auto clear_tail = [&](int step, uint4 *t) {
        if (!TAIL || step != ksteps - 1) return;
        for (int e = threadIdx.x; e < BW * 8; e += 64 * GW * KSP)
            if (((e & 7) ^ (e >> 4 & 7)) >= tail) t[e] = make_uint4(0, 0, 0, 0);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    wait_stage<LOADS + LOADS / NS>();
    clear_tail(sb, tile[0]);
    int rb = 0, step = sb;
#pragma unroll
    for (int n = 0; n < FW + P * FT; ++n) read_one(tile[0], kk0, 0, n);
    for (int s = 0; s < nsteps; ++s) {
        const uint4 *t = tile[rb];
#pragma unroll
        for (int k = 0; k < NS - 1; ++k) slice(k & 1, t, kk0 + k + 1, k + 1);
        next_stage();
        rb = rb == STAGES - 1 ? 0 : rb + 1;
        wait_stage<LOADS>();
        clear_tail(++step, tile[rb]);
        slice(1, tile[rb], kk0, 0);                          // behind the last stage: a read of old values, not used
    }
    wait_stage<0>();
    if constexpr (KSP == 2) {                                // the second group's sums join the first's, which goes on alone
        f32x4_t *part = reinterpret_cast<f32x4_t *>(tile) + w4 * (FW * FT * 4 * 64) + lane;
        static_assert(GW * FW * FT * 4 * 64 * sizeof(f32x4_t) <= sizeof(tile), "");
        __syncthreads();
#pragma unroll
        for (int i = 0; i < FW * FT * 4; ++i) {
            f32x16_t &y = acc[i / 4 / FT][i / 4 % FT];
            const int v = i % 4 * 4;
            if (wave >= GW) part[i * 64] = f32x4_t{y[v], y[v + 1], y[v + 2], y[v + 3]};
        }
        __syncthreads();
        if (wave >= GW) return;
#pragma unroll
        for (int i = 0; i < FW * FT * 4; ++i) {
            f32x16_t &y = acc[i / 4 / FT][i / 4 % FT];
            const int v = i % 4 * 4;
            const f32x4_t x = part[i * 64];
            y[v] += x.x; y[v + 1] += x.y; y[v + 2] += x.z; y[v + 3] += x.w;
        }
    }
    // D: lane holds token i32 of a fragment, weight rows 8 * (v / 4) + 4 * hh + v % 4
    if constexpr (LOW) {
        // the whole K: s, scaled and split; else fp32 sums of this part of K: [part][pos][projection][R]
        const float scale = !g.part && a.scale ? uniform_at(a.scale, ad0) : 1.f;
        const int rank = g.part ? 0 : rank_of(a, ad0);
#pragma unroll
        for (int j = 0; j < FT; ++j) {
            const int pos = t0 + (rt - BW) + j * 32 + i32;
            if (pos > last) continue;
            if (!g.part) {
#pragma unroll
                for (int i = 0; i < FW; ++i)
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4) {
                        const int rr = w0 + rw + i * 32 + 8 * v4 + 4 * hh, proj = rr / a.R, r = rr - proj * a.R;
                        if (rr >= g.N) continue;
                        float y[4];
#pragma unroll
                        for (int v = 0; v < 4; ++v) y[v] = r + v < rank ? acc[i][j][4 * v4 + v] * scale : 0.f;
                        uint16_t *o = g.h + ((int64_t)pos * (g.N / a.R) + proj) * 3 * a.R + r;
#pragma unroll
                        for (int p = 0; p < 3; ++p) *reinterpret_cast<uint2 *>(o + p * a.R) = pack_part(y, p);
                    }
                continue;
            }
            float *o = g.part + ((int64_t)blockIdx.y * a.T + pos) * g.N;
#pragma unroll
            for (int i = 0; i < FW; ++i)
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    const int rr = w0 + rw + i * 32 + 8 * v4 + 4 * hh;
                    const f32x16_t &y = acc[i][j];
                    if (rr < g.N)
                        *reinterpret_cast<float4 *>(o + rr) = make_float4(y[4 * v4], y[4 * v4 + 1], y[4 * v4 + 2], y[4 * v4 + 3]);
                }
        }
        return;
    } else if (a.n) {
        // Up to NA adapters of 64 of this wave's tokens at a time, whose loads go out together (gate/up of 2048 tokens, rank
        // 16, side by side: 70 us, 77 with one adapter after the other and its rank before its loads; without adapters it is 3
        // us less than with them, 5 to 7 less at rank 32). Rank values go 16 at a time, each once with each part of the tokens'
        // low-rank results (two of which, 16 bits, beside a bf16 result). An adapter's products are formed for all of the
        // tokens, in sums of their own, and added to those of its own tokens.
        constexpr int NP = GU ? 2 : 1, JG = FT < 2 ? FT : 2, SP = !GU && P < 3 ? 2 : 3, NA = 4;
#pragma unroll
        for (int jg = 0; jg < FT; jg += JG) {
            unsigned long long left[JG];
#pragma unroll
            for (int j = 0; j < JG; ++j) left[j] = __ballot(idj[jg + j] >= 0);
            while (left[0] | left[JG - 1]) {
                int ad[NA], rank[NA], top = 0;
#pragma unroll
                for (int q = 0; q < NA; ++q) {
                    ad[q] = -1;
                    rank[q] = 0;
                    if (!(left[0] | left[JG - 1])) continue;
                    ad[q] = left[0] ? __builtin_amdgcn_readlane(idj[jg], __ffsll(left[0]) - 1)
                                    : __builtin_amdgcn_readlane(idj[jg + JG - 1], __ffsll(left[JG - 1]) - 1);
#pragma unroll
                    for (int j = 0; j < JG; ++j) left[j] &= ~__ballot(idj[jg + j] == ad[q]);
                    rank[q] = rank_of(a, ad[q]);
                }
                int c0 = 0;
                do {
                    const int j8 = c0 + hh;
                    const bool in = 8 * j8 < a.R;
                    uint4 w[NA][FW], u[JG][NP][SP];
#pragma unroll
                    for (int j = 0; j < JG; ++j)
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
#pragma unroll
                            for (int h = 0; h < SP; ++h) u[j][p][h] = make_uint4(0, 0, 0, 0);
                            if (in && idj[jg + j] >= 0 && g.b[p]) {
                                const uint16_t *s = low_rank_row(a, g.s, NP, t0 + (rt - BW) + (jg + j) * 32 + i32, p) + 8 * j8;
#pragma unroll
                                for (int h = 0; h < SP; ++h) u[j][p][h] = load16(s + h * a.R);
                            }
                        }
#pragma unroll
                    for (int q = 0; q < NA; ++q)
#pragma unroll
                        for (int i = 0; i < FW; ++i) {
                            const int m = GU ? i & 1 : 0;
                            const int wr = GU ? w0 + (rw >> 6) * 32 + i32 : w0 + rw + i * 32 + i32;
                            w[q][i] = make_uint4(0, 0, 0, 0);
                            if (in && ad[q] >= 0 && wr < g.N && g.b[m])
                                w[q][i] = load16(g.b[m] + ((int64_t)ad[q] * g.N + wr) * a.R + 8 * j8);
                        }
#pragma unroll
                    for (int q = 0; q < NA; ++q) {
                        if (8 * c0 >= rank[q]) continue;
                        top = max(top, rank[q]);
                        f32x16_t d[FW][JG];
#pragma unroll
                        for (int i = 0; i < FW; ++i) {
                            const uint4 wq = keep_first(w[q][i], rank[q] - 8 * j8);
#pragma unroll
                            for (int j = 0; j < JG; ++j) {
#pragma unroll
                                for (int v = 0; v < 16; ++v) d[i][j][v] = 0.f;
#pragma unroll
                                for (int h = 0; h < SP; ++h) d[i][j] = mfma32(wq, u[j][GU ? i & 1 : 0][h], d[i][j]);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < JG; ++j)
                            if (idj[jg + j] == ad[q]) {
#pragma unroll
                                for (int i = 0; i < FW; ++i) acc[i][jg + j] += d[i][j];
                            }
                    }
                    c0 += 2;
                } while (8 * c0 < top);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < FT; ++j) {
        const int pos = t0 + (rt - BW) + j * 32 + i32;
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
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    if (p < g.hp) *reinterpret_cast<uint2 *>(g.h + (int64_t)p * a.T * g.N + row + wr) = pack_part(h, p);
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

constexpr int MAX_PARTS = 8;

// s[pos][proj][3 parts][r] = scale_a * (sum of the parts of K, in order); 0 from the adapter's rank on.
__global__ __launch_bounds__(256) void k_low_rank_sum(SharedArgs a, const float *part, int parts, int np, uint16_t *s) {
    const int per = np * a.R / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)a.T * per) return;
    const int pos = (int)(i / per), rr = 4 * (int)(i - (int64_t)pos * per), proj = rr / a.R, r = rr - proj * a.R;
    const int ad = a.plan_ad[pos];
    f32x4_t v = {0.f, 0.f, 0.f, 0.f}, x[MAX_PARTS];
#pragma unroll
    for (int k = 0; k < MAX_PARTS; ++k) {
        x[k] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (k < parts) x[k] = *reinterpret_cast<const f32x4_t *>(part + ((int64_t)k * a.T + pos) * np * a.R + rr);
    }
#pragma unroll
    for (int k = 0; k < MAX_PARTS; ++k) v += x[k];
    if (ad < 0) return;                                      // of no adapter: neither written before nor read after
    const float c = a.scale ? a.scale[ad] : 1.f;
    const int rank = rank_of(a, ad) - r;
    v.x = 0 < rank ? v.x * c : 0.f;
    v.y = 1 < rank ? v.y * c : 0.f;
    v.z = 2 < rank ? v.z * c : 0.f;
    v.w = 3 < rank ? v.w * c : 0.f;
    const float y[4] = {v.x, v.y, v.z, v.w};
    uint16_t *o = s + ((int64_t)pos * np + proj) * 3 * a.R + r;
#pragma unroll
    for (int p = 0; p < 3; ++p) *reinterpret_cast<uint2 *>(o + p * a.R) = pack_part(y, p);
}

template <bool GU, int P, int AD>
hipError_t launch_few(const SharedArgs &a, const Product &g, hipStream_t st) {
    // gate/up: whole rounds of the packed h, whose last rows may be zeros
    const int tf = few_frags(a.T);
    const dim3 grd((unsigned)(GU ? few_steps(g.N) * 4 : (g.N + 15) / 16), (unsigned)few_groups(a.T)), blk(64 * FEW_WAVES);
    if (tf == 1) hipLaunchKernelGGL((k_few<GU, P, 1, AD>), grd, blk, 0, st, a, g);
    if constexpr (AD != AD_HERE) {
        if (tf == 2) hipLaunchKernelGGL((k_few<GU, P, 2, AD>), grd, blk, 0, st, a, g);
        else if (tf == 4) hipLaunchKernelGGL((k_few<GU, P, 4, AD>), grd, blk, 0, st, a, g);
    }
    return hipGetLastError();
}

bool low_rank_here(const SharedArgs &a) {
    return a.T <= HERE_VALUES && a.T * a.R <= HERE_VALUES && a.T * a.R * a.Is <= HERE_TERMS;
}

template <bool GU, int P>
hipError_t few_planes(const SharedArgs &a, const Product &g, hipStream_t st) {
    if (!a.n) return launch_few<GU, P, AD_NONE>(a, g, st);
    if constexpr (!GU) {
        if (low_rank_here(a)) return launch_few<GU, P, AD_HERE>(a, g, st);
    }
    return launch_few<GU, P, AD_READ>(a, g, st);
}

template <bool GU>
hipError_t few(const SharedArgs &a, const Product &g, int planes, hipStream_t st) {
    if constexpr (GU) {
        if (planes == 1) return few_planes<GU, 1>(a, g, st);
    }
    return planes == 2 ? few_planes<GU, 2>(a, g, st) : few_planes<GU, 3>(a, g, st);
}

// Packs the activations (packed) and forms the low-rank results (a.n), one launch for both.
hipError_t few_inputs(const SharedArgs &a, const LowRank &L, bool f32, int planes, uint16_t *packed, hipStream_t st) {
    const int pack = packed ? ((a.T + 15) / 16 * few_steps(L.K) + 3) / 4 : 0;
    const int low = a.n ? (a.T * L.np * a.R + 3) / 4 : 0;
    if (!pack && !low) return hipSuccess;
    const dim3 grd((unsigned)(pack + low)), blk(256);
    if (!f32) hipLaunchKernelGGL((k_few_inputs<false, 1>), grd, blk, 0, st, a, L, packed, pack);
    else if (planes == 2) hipLaunchKernelGGL((k_few_inputs<true, 2>), grd, blk, 0, st, a, L, packed, pack);
    else hipLaunchKernelGGL((k_few_inputs<true, 3>), grd, blk, 0, st, a, L, packed, pack);
    return hipGetLastError();
}

template <int MODE, int P, bool TAIL>
hipError_t launch_many(const SharedArgs &a, const Product &g, int bw, int bt, int tw, int tt, int parts, hipStream_t st) {
    const dim3 grd((unsigned)((tw * tt + 7) / 8 * 8), (unsigned)parts), blk((unsigned)many_threads(bw, bt));
    if constexpr (MODE != MODE_LOW_RANK && P == 1) {
        if (bt == 256) hipLaunchKernelGGL((k_many<MODE, P, 128, 256, TAIL>), grd, blk, 0, st, a, g, tw, tt);
    }
    if constexpr (MODE != MODE_LOW_RANK && P < 3) {
        if (bt == 128) hipLaunchKernelGGL((k_many<MODE, P, 128, 128, TAIL>), grd, blk, 0, st, a, g, tw, tt);
    }
    if (bt == 64 && bw == 128) hipLaunchKernelGGL((k_many<MODE, P, 128, 64, TAIL>), grd, blk, 0, st, a, g, tw, tt);
    else if (bt == 64) hipLaunchKernelGGL((k_many<MODE, P, 64, 64, TAIL>), grd, blk, 0, st, a, g, tw, tt);
    return hipGetLastError();
}

template <int MODE>
hipError_t many_tiles(const SharedArgs &a, const Product &g, int planes, int bw, int bt, int tt, int parts, hipStream_t st) {
    const int rows = MODE == MODE_GATE_UP ? bw / 2 : bw, tw = (g.N + rows - 1) / rows;
    if constexpr (MODE != MODE_DOWN) {
        if (planes == 1)
            return g.K % BK ? launch_many<MODE, 1, true>(a, g, bw, bt, tw, tt, parts, st)
                            : launch_many<MODE, 1, false>(a, g, bw, bt, tw, tt, parts, st);
    }
    if (planes == 2)
        return g.K % BK ? launch_many<MODE, 2, true>(a, g, bw, bt, tw, tt, parts, st)
                        : launch_many<MODE, 2, false>(a, g, bw, bt, tw, tt, parts, st);
    return g.K % BK ? launch_many<MODE, 3, true>(a, g, bw, bt, tw, tt, parts, st)
                    : launch_many<MODE, 3, false>(a, g, bw, bt, tw, tt, parts, st);
}

template <int MODE>
hipError_t many(const SharedArgs &a, const Product &g, int planes, hipStream_t st) {
    const int rows = MODE == MODE_GATE_UP ? 64 : 128, tw = (g.N + rows - 1) / rows;
    auto tiles = [&](int bt) { return tw * ((a.T + bt - 1) / bt); };
    // two planes of 256 tokens or three of 128 would not fit three times into LDS
    const int bt = planes < 2 && tiles(256) >= 256 ? 256 : planes < 3 && tiles(128) >= 256 ? 128 : 64;
    // half tiles where whole ones are for half of the compute units at most (whole call, whole tiles against half ones: 333
    // tokens 1000 x 520 61.2 and 58.0 us, 300 tokens 2048 x 512 51.4 and 48.5, 400 tokens 1024 x 1024 49.4 and 46.7)
    const int bw = bt == 64 && tiles(64) <= 128 ? 64 : 128;
    return many_tiles<MODE>(a, g, planes, bw, bt, (a.T + bt - 1) / bt, 1, st);
}

int plan_items(int T, int n) { return T / ITEM_TOKENS + (T < n ? T : n); }     // at most

// Parts of K of the down-rank products: one for short rows (no sum to launch; 400 tokens 1024 x 512 of rank 16, whole calls, two
// launches each against one: 42.2 and 40.3 us; of three planes and 16 steps, 333 tokens 1000 x 520: 52.9 and 55.5), else enough
// workgroups for the 256 CUs, each with some steps.
int low_rank_rows(int N) { return N <= 64 ? 64 : 128; }
int low_rank_parts(int T, int n, int R, int np, int K, int planes) {
    const int bw = low_rank_rows(np * R), tiles = plan_items(T, n) * ((np * R + bw - 1) / bw), steps = (K + BK - 1) / BK;
    int parts = 1;
    if (steps <= 16 && steps * planes <= 24) return 1;
    while (parts < MAX_PARTS && parts * tiles < 256 && steps >= 8 * parts) parts *= 2;
    return parts;
}

hipError_t many_low_rank(const SharedArgs &a, const LowRank &L, int planes, hipStream_t st) {
    Product g = {};
    g.x = static_cast<const uint16_t *>(L.xv); g.K = L.K; g.N = L.np * a.R; g.gather = L.gather;
    g.w[0] = L.a[0]; g.w[1] = L.a[1]; g.h = L.s;
    const int parts = low_rank_parts(a.T, a.n, a.R, L.np, L.K, planes);
    if (parts > 1) g.part = L.part;
    hipError_t e = many_tiles<MODE_LOW_RANK>(a, g, planes, low_rank_rows(g.N), 64, plan_items(a.T, a.n), parts, st);
    if (e != hipSuccess || parts == 1) return e;
    const int64_t quads = (int64_t)a.T * g.N / 4;
    hipLaunchKernelGGL(k_low_rank_sum, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, st, a, L.part, parts, L.np, L.s);
    return hipGetLastError();
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

// Whether the weights stream past groups of up to 64 tokens (once from memory, then from the caches), or tiles of both operands
// pass through LDS, which costs up to five more launches for the plan and the down-rank parts.  Streamed against tiles,
// hidden x inter, 16 adapters of rank up to 16 in runs, fp32 out:
//   2 groups: 100 tokens 1024 x 1024 30.3 and 47.8 us, 128 tokens 4096 x 2048 75 and 68 (bf16 out 68 and 65; an adapter of
//     rank 64 for each of 100 tokens, bf16 out: 103 and 211);
//   4 groups: 256 tokens 512 x 512 33.2 and 37.4, 1024 x 1024 (bf16 out) 38.8 and 43.8, 200 tokens 2048 x 1024 56.0 and 51.1,
//     256 tokens 4096 x 512 73.8 and 54.5;
//   6 groups: 333 tokens 1000 x 520 (fp32 x) 69.4 and 51.7.
bool few_path(int T, int H, int Is) {
    const int64_t reads = (int64_t)few_groups(T) * H * Is;
    return T <= FEW_TOKENS || (T <= 2 * FEW_TOKENS && reads <= 1 << 24) || (T <= 4 * FEW_TOKENS && reads <= 1 << 22);
}

// Workspace layout, from the shapes and types alone.
struct Layout {
    size_t x, perm, ad, items, n_items, s, part, h, hrow, total;
};
Layout layout(int T, int H, int Is, int n, int R, int xp, int hp) {
    Layout l = {};
    size_t o = 0;
    auto take = [&](size_t b) { const size_t at = o; o += (b + 255) / 256 * 256; return at; };
    const bool small = few_path(T, H, Is);
    const size_t tf = (size_t)few_groups(T) * few_frags(T);
    auto packed = [&](int K, int p) { return (size_t)p * tf * few_steps(K) * 1024; };
    l.s = take(n > 0 ? (size_t)T * 2 * 3 * R * 2 : 0);       // gate/up's, then down's
    if (small) {
        l.x = take(packed(H, xp));
        l.h = take(packed(Is, hp));
        l.hrow = take(n > 0 ? (size_t)T * Is * 4 : 0);
    } else {
        l.x = take(xp > 1 ? (size_t)T * H * xp * 2 : 0);
        l.h = take((size_t)T * Is * 2 * hp);
        if (n > 0) {
            l.perm = take((size_t)T * 4);
            l.ad = take((size_t)T * 4);
            l.items = take((size_t)plan_items(T, n) * 16);
            l.n_items = take(4);
            // parts * T of the down-rank products of T or fewer tokens: MAX_PARTS parts at most, and more than one (a single part
            // writes its results at once) only where parts / 2 times more than T / ITEM_TOKENS items are below 256 workgroups
            l.part = take(std::min<size_t>((size_t)MAX_PARTS * T, 2 * 256 * ITEM_TOKENS) * 2 * R * 4);
        }
    }
    l.total = o;
    return l;
}

}  // namespace

namespace moe {

size_t shared_workspace(int T, int H, int Is, int n, int R) {
    // the largest over the activation and result types and over fewer tokens (whose streamed path pads its operands), so that
    // one buffer serves every call of these sizes
    size_t most = layout(T, H, Is, n, R, 3, 3).total;
    for (int t = FEW_TOKENS; t <= 4 * FEW_TOKENS; t += FEW_TOKENS)
        if (t < T && few_path(t, H, Is)) most = std::max(most, layout(t, H, Is, n, R, 3, 3).total);
    return most;
}

hipError_t launch_shared(SharedArgs a, void *ws, hipStream_t st) {
    char *base = static_cast<char *>(ws);
    // bf16 parts of x and h.  Beside a bf16 result 16 bits are enough: what they leave is 2^-8 of its own rounding.  One part
    // of h would not be, though it halves the down product: its rounding is as large as the result's (2048 tokens of 4096 x
    // 2048, error against binary64 2.35e-3 with one part, 1.66e-3 with two, which is that of one rounding).
    const bool small = few_path(a.T, a.H, a.Is);
    const int xp = a.x_bf16 ? 1 : a.out_bf16 ? 2 : 3, hp = a.out_bf16 ? 2 : 3;
    const Layout l = layout(a.T, a.H, a.Is, a.n, a.R, xp, hp);
    auto u16 = [&](size_t at) { return reinterpret_cast<uint16_t *>(base + at); };
    uint16_t *s = u16(l.s), *h = u16(l.h);
    float *part = reinterpret_cast<float *>(base + l.part);
    a.sorted = a.n > 0 && !small;
    SharedArgs ag = a, ad = a;                              // a half without adapters runs as if there were none
    if (!a.gate_a && !a.up_a) ag.n = 0;
    if (!a.down_a) ad.n = 0;
    LowRank lx = {a.x, a.H, 2, 1, {a.gate_a, a.up_a}, s, part}, lh = {h, a.Is, 1, 0, {a.down_a, nullptr}, s, part};
    Product gu = {}, dn = {};
    gu.x = static_cast<const uint16_t *>(a.x); gu.K = a.H; gu.N = a.Is; gu.gather = 1;
    gu.w[0] = a.gate; gu.w[1] = a.up; gu.b[0] = a.gate_b; gu.b[1] = a.up_b; gu.s = s; gu.h = h; gu.hp = hp;
    dn.x = h; dn.K = a.Is; dn.N = a.H; dn.gather = 0;
    dn.w[0] = a.down; dn.b[0] = a.down_b; dn.s = s; dn.out = a.out; dn.out_bf16 = a.out_bf16;
    hipError_t e;
    if (small) {
        gu.x = u16(l.x);
        if (ad.n) lh.xv = gu.hrow = reinterpret_cast<float *>(base + l.hrow);
        if ((e = few_inputs(ag, lx, !a.x_bf16, xp, u16(l.x), st)) != hipSuccess) return e;
        if ((e = few<true>(ag, gu, xp, st)) != hipSuccess) return e;
        if (ad.n && low_rank_here(ad)) {
            dn.a = a.down_a;
            dn.hrow = gu.hrow;
        } else if ((e = few_inputs(ad, lh, true, hp, nullptr, st)) != hipSuccess) {
            return e;
        }
        return few<false>(ad, dn, hp, st);
    }
    if (!a.x_bf16) lx.xv = gu.x = u16(l.x);
    if (a.sorted) {
        a.perm = reinterpret_cast<int32_t *>(base + l.perm);
        a.plan_ad = reinterpret_cast<int32_t *>(base + l.ad);
        a.items = reinterpret_cast<int4 *>(base + l.items);
        a.n_items = reinterpret_cast<int32_t *>(base + l.n_items);
    }
    if (a.sorted || !a.x_bf16) {
        const int64_t quads = a.x_bf16 ? 0 : (int64_t)a.T * a.H / 4;
        hipLaunchKernelGGL(k_plan, dim3((unsigned)(a.sorted + (quads + PLAN_THREADS - 1) / PLAN_THREADS)), dim3(PLAN_THREADS),
                           0, st, a, u16(l.x), xp, a.sorted);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.sorted) {
        const int ng = ag.n, nd = ad.n;
        ag = ad = a;
        ag.n = ng;
        ad.n = nd;
    }
    if (ag.n && (e = many_low_rank(ag, lx, xp, st)) != hipSuccess) return e;
    if ((e = many<MODE_GATE_UP>(ag, gu, xp, st)) != hipSuccess) return e;
    if (ad.n && (e = many_low_rank(ad, lh, hp, st)) != hipSuccess) return e;
    return many<MODE_DOWN>(ad, dn, hp, st);
}

}  // namespace moe
