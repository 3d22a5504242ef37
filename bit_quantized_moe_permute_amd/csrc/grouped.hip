// Products over rows grouped by expert (moe_grouped_linear, moe_grouped_dgrad, moe_grouped_wgrad):
//
//   forward           out[o][n] = sum_k x[r][k] W_g[n][k]
//   input's gradient  dx[i][k]  = sum_n dy[o][n] W_g[n][k]
//   weights' gradient dW_g[n][k] = sum over the positions of g of dy[o][n] x[r][k]
//
// All on the bf16 matrix cores, with fp32 sums from the first to the last product; a bf16 output is rounded once, where it is
// stored. Few rows to an expert: every weight is read once, and that is the time (one token of 8 among 256 experts, 256 MiB of
// weights: 49 us, 5.4 TB/s; 2048 tokens of the same, all weights, 8.6 GB: 1742 us, 5.0 TB/s). Many rows: the products are (11709
// tokens of 8 among 32 experts: 2811 us, 1119 TFLOP/s, where a library product of 8192 x 8192 x 8192 makes 1346). A large copy
// moves 5.15 TB/s.
#include <type_traits>

#include "choice.h"
#include "groups.h"

using namespace moe;

namespace {

typedef __attribute__((address_space(3))) void *las_ptr;
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t *las_s16x4;
typedef const __attribute__((address_space(3))) u32x4_t *las_u32x4;

__device__ __forceinline__ f32x16_t mfma32(uint4 a, uint4 b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)a, (__bf16)b});
}

// Everything in LDS is read, up to N of this wave's loads are still under way, and the workgroup is here.
template <int N> __device__ __forceinline__ void wait_stage() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16 bytes at each lane's address -> 1 KiB of LDS at byte address `dst` (wave-uniform), in lane order. The destination goes
// through m0, which is put back: the compiler may count on its value.
__device__ __forceinline__ void load_to_lds(uint64_t from, uint32_t dst) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0) : "v"(from), "s"(dst) : "memory");
}

// ---------------------------------------------------------------------------
// A workgroup computes a tile of TP x TQ results, WP x WQ waves of FP x FQ fragments of 32 x 32. P is the side whose results lie
// one behind the other in memory (the weights' rows; for the gradients the columns of W and x), Q the rows of the output.
//
//              P                        Q                        summed over
//   forward    rows of W    [n][k]      rows of x    [r][k]      k
//   dgrad      columns of W [n][k]      rows of dy   [o][n]      n
//   wgrad      columns of x [r][k]      columns of dy [o][n]     positions
//
// Both pass through LDS in steps of BK = 64 or 32 of the sum, NST of them in a ring that direct-to-LDS loads fill. An operand
// whose rows run along the sum ("rows") keeps 2 BK bytes per row there: 16-byte chunk c of row r lies at c ^ (r / 2 % 8) (BK 32: c
// ^ (r / 4 % 4)), so that sixteen rows' reads of a chunk column touch every bank once. One whose rows run across it ("columns") is
// read with the transposing LDS loads, four steps of the sum x 16 columns by 16 lanes: piece u of 16 columns of row r lies at u ^
// swizzle(r).
// What is outside (rows behind the group, steps behind the sum, rows that an index puts outside) is read from a block of zeros.
//
// The loads are written as assembly: the compiler would otherwise wait for all of them before any LDS read. They have no
// register outputs; wait_stage() counts them and orders the workgroup. Nothing else of the loop loads through the vector memory
// pipe.
//
// What bounds it, forward: at 256 x 256 the loop runs like the library's, and ragged last tiles and the first loads of a tile are
// the rest; LDS gives two fragments of 32 x 32 x 16 in the time of two such products, so a wave has 4 x 2 of them. Input's gradient
// (2048 tokens of 8 among 32 experts of 4096 x 2048): 345 us, 790 TFLOP/s; 640 tiles are 2.5 rounds of the 256 units and take three.
// Weights' gradient (32 experts of 4096 x 4096, 512 rows each): 939 us; a tile has eight steps only, and its first loads (offsets,
// indices, rows, one behind the other) and its 256 KiB of results are not hidden behind another tile's products, since its ring and
// its sums fill the unit (with stores through the L2 1028 us, without the stores 765, without the loop 512). Workgroups that go on
// to a second tile by themselves took longer.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t swizzle(int r) { return ((r & 1) * 2) ^ ((r >> 1 & 1) * 5); }

template <int OP, int FP, int FQ, int WP, int WQ, int BK, int NST, bool SWIGLU>
__global__ __launch_bounds__(64 * WP * WQ, FP * FQ <= 8 ? 2 : 1) void k_tile(GroupedArgs a, int tiles_p, int tiles_q) {
    constexpr bool COLS_P = OP != GROUPED_FWD, COLS_Q = OP == GROUPED_WGRAD;
    constexpr int NW = WP * WQ, TP = 32 * FP * WP, TQ = 32 * FQ * WQ;
    constexpr int RK = 512 / BK, LP = TP / RK / NW, LQ = TQ / RK / NW, LOADS = LP + LQ;      // rows per KiB; loads of 1 KiB per wave and stage
    constexpr uint32_t STAGE = (TP + TQ) * 2 * BK;
    static_assert(LP * NW * RK == TP && LQ * NW * RK == TQ && (!COLS_P || TP >= 128) && (!COLS_Q || TQ >= 128), "");
    __shared__ __attribute__((aligned(1024))) uint8_t ring[NST * STAGE];
    // Weights' gradient: the rows of x and dy of the next WINDOW positions (-1: none, or behind the group).
    constexpr int WINDOW = OP == GROUPED_WGRAD ? 2048 : 1;
    __shared__ int table[OP == GROUPED_WGRAD ? 2 : 1][WINDOW];
    const int lane = threadIdx.x & 63, i32 = lane & 31, hh = lane >> 5;
    // Of the two waves that share a SIMD (w and w + 4 of eight), one has the first rows of the output and one the last: where a
    // tile is not full, the waves without rows leave the others the matrix cores.
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w4 = wave & 3, back = wave >> 2;
    static_assert(NW == 4 || (NW == 8 && (WQ == 2 || WQ == 4)), "");
    const int wp = NW == 4 ? wave / WQ : WQ == 4 ? w4 & 1 : (w4 >> 1) + 2 * back;
    const int wq = NW == 4 ? wave % WQ : WQ == 4 ? (back ? 3 - (w4 >> 1) : w4 >> 1) : (w4 + back) & 1;
    const int P = OP == GROUPED_FWD ? a.n_out : a.n_in;                               // results per row of the output
    // XCD-aware order: consecutive workgroups go to the eight XCDs in turn; each takes a run of tiles, in blocks of four tiles
    // along Q whose workgroups read the same rows on the other side
    int tp, group, begin, end, q0, last_q;
    if constexpr (OP == GROUPED_WGRAD) {
        const int total = tiles_p * tiles_q * a.g.n, per = (total + 7) / 8, id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
        if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
        group = id / (tiles_p * tiles_q);
        const int t = id - group * tiles_p * tiles_q;
        tp = t / tiles_q;
        q0 = (t - tp * tiles_q) * TQ;
        last_q = a.n_out;
        begin = group_edge(a.g, group);
        end = group_edge(a.g, group + 1);
        if (a.accumulate && end <= begin) return;            // stays as it is (-0 + 0 would be 0), and need not be read
    } else {
        const Tiles all = scan_tiles(a.g, TQ, tiles_q);
        const int total = all.total * tiles_p, per = (total + 7) / 8;
        const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
        if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
        const int block = id / (4 * tiles_p), in = id - block * 4 * tiles_p, height = min(4, all.total - 4 * block);
        tp = in / height;
        const Tile t = tile_at(a.g, all, TQ, 4 * block + in - tp * height);
        group = t.group;
        q0 = t.begin;
        last_q = t.end;
        begin = end = 0;
    }
    const int K = OP == GROUPED_FWD ? a.n_in : OP == GROUPED_DGRAD ? a.n_out : max(end - begin, 0);
    const int p0 = tp * (SWIGLU ? TP / 2 : TP), ns = (K + BK - 1) / BK;
    const uint64_t zero = (uint64_t)(uintptr_t)zeros;
    const uint64_t weights = (uint64_t)(uintptr_t)a.b + (uint64_t)group * a.n_out * a.n_in * (SWIGLU ? 4 : 2);

    // Load i of this wave, P's first: from[i] is this lane's 16 bytes in the next stage to load; inside says whether they are
    // any of the operand's, left is how far the sum goes from there.
    constexpr int RP = 512 / TP, RQ = 512 / TQ;              // columns: rows per load
    constexpr int CK = BK / 8;                               // rows: chunks of a row in a step
    auto place = [](int r, int c) { return BK == 64 ? c ^ (r >> 1 & 7) : c ^ (r >> 2 & 3); };
    uint64_t from[LOADS];
    int left[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const bool is_p = i < LP;
        const int l = is_p ? wave * LP + i : wave * LQ + i - LP;
        if (is_p ? !COLS_P : !COLS_Q) {
            const int r = RK * l + lane / CK, chunk = place(r, lane % CK);           // this lane's 8 of a step
            int row;
            if (is_p) {
                const int n = SWIGLU ? (r >> 6) * 32 + (r & 31) : r;
                row = p0 + n < P ? (SWIGLU && (r >> 5 & 1) ? P : 0) + p0 + n : -1;
            } else {
                const int p = q0 + r;
                row = p >= last_q ? -1 : OP == GROUPED_FWD ? in_row(a.g, p, a.a_rows) : out_row(a.g, p, a.a_rows);
            }
            from[i] = (is_p ? weights : (uint64_t)(uintptr_t)a.a) + 2 * ((uint64_t)(uint32_t)max(row, 0) * (uint32_t)K + 8 * chunk);
            left[i] = row < 0 ? 0 : K - 8 * chunk;
        } else {
            const int rows = is_p ? RP : RQ, per_row = 64 / rows, r = l * rows + lane / per_row, s = lane % per_row;
            const int c = ((int)((s >> 1) ^ swizzle(r)) << 1 | (s & 1)) * 8 + (is_p ? p0 : q0);      // first of 8 columns
            const int cols = is_p ? P : a.n_out;
            left[i] = c < cols ? K - r : 0;
            from[i] = 2 * (uint64_t)c + (OP == GROUPED_DGRAD ? weights + 2 * (uint64_t)r * (uint32_t)cols
                                                              : (uint64_t)(uintptr_t)(is_p ? a.a : a.b));
        }
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(las_ptr)ring;
    int step = 0;                                            // the sum's position of the stage to load next
    uint32_t idst = lds0;
    // Rows of positions first .. + count - 1 of the sum into the table.
    auto fill = [&](int first, int count) __attribute__((always_inline)) {
        if constexpr (OP == GROUPED_WGRAD) {
            for (int e = threadIdx.x; e < count; e += 64 * NW) {
                const int p = begin + first + e;
                const int x = first + e < K ? in_row(a.g, p, a.a_rows) : -1;
                const int dy = first + e < K ? out_row(a.g, p, a.b_rows) : -1;
                table[0][(first + e) % WINDOW] = dy < 0 ? -1 : x;        // without either the other may hold anything, NaN too
                table[1][(first + e) % WINDOW] = x < 0 ? -1 : dy;
            }
        }
    };
    int next_row[OP == GROUPED_WGRAD ? LOADS : 1];
    auto look_up = [&](int i) __attribute__((always_inline)) {                              // the row that load i will read, ahead of its issue
        if constexpr (OP == GROUPED_WGRAD) {
            const bool is_p = i < LP;
            const int rows = is_p ? RP : RQ, l = is_p ? wave * LP + i : wave * LQ + i - LP;
            next_row[i] = table[is_p ? 0 : 1][(step + l * rows + lane / (64 / rows)) % WINDOW];
        }
    };
    auto issue = [&](int i) __attribute__((always_inline)) {                                // i: load of this wave (compile-time)
        const bool is_p = i < LP;
        uint64_t at = from[i];
        bool in = step < left[i];
        if constexpr (OP == GROUPED_WGRAD) {
            in = in && next_row[i] >= 0;
            at += 2 * (uint64_t)(uint32_t)next_row[i] * (uint32_t)(is_p ? P : a.n_out);
        }
        const int l = is_p ? wave * LP + i : TP / RK + wave * LQ + i - LP;
        load_to_lds(in ? at : zero, idst + l * 1024u);
        if constexpr (OP == GROUPED_FWD) from[i] += 2 * BK;
        else if constexpr (OP == GROUPED_DGRAD) from[i] += is_p ? 2 * BK * (uint64_t)(uint32_t)P : 2 * BK;
    };
    auto next_stage = [&]() {
        step += BK;
        idst = idst == lds0 + (NST - 1) * STAGE ? lds0 : idst + STAGE;
    };
    f32x16_t acc[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

    // Fragment n of a 16-wide slice: lane l has its row (column) l % 32 and 8 (l / 32) .. + 7 of the sum.
    const int tr = 8 * hh + (lane >> 2 & 3);                 // columns: row of this lane's four values of the first read
    uint4 fp[2][FP], fq[2][FQ];
    auto read_one = [&](uint32_t stage, int kk, int b, int n) __attribute__((always_inline)) {
        const bool is_p = n < FP;
        const int f = is_p ? wp * FP + n : wq * FQ + n - FP;
        const uint32_t base = stage + (is_p ? 0 : TP * 2 * BK);
        uint4 v;
        if (is_p ? !COLS_P : !COLS_Q) {
            const uint32_t c = (uint32_t)place(i32, 2 * kk + hh);
            v = __builtin_bit_cast(uint4, *(las_u32x4)(uintptr_t)(base + (f * 32 + i32) * 2 * BK + c * 16));
        } else {
            const uint32_t pitch = 2 * (is_p ? TP : TQ), u = (uint32_t)(2 * f + (lane >> 4 & 1)) ^ swizzle(lane >> 2);
            const uint32_t at = base + (16 * kk + tr) * pitch + u * 32 + 8 * (lane & 3);
            const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((las_s16x4)(uintptr_t)at);
            const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((las_s16x4)(uintptr_t)(at + 4 * pitch));
            const uint2 l2 = __builtin_bit_cast(uint2, lo), h2 = __builtin_bit_cast(uint2, hi);
            v = make_uint4(l2.x, l2.y, h2.x, h2.y);
        }
        if (is_p) fp[b][n] = v;
        else fq[b][n - FP] = v;
    };
    // The products of one slice (buffer b). Between them go the reads of the next slice and part `part` of 2 of a stage's loads
    // (-1: none), so that the matrix cores have work while these are issued. A wave without results only loads.
    const bool works = p0 + wp * 32 * FP / (SWIGLU ? 2 : 1) < P && q0 + wq * 32 * FQ < last_q;
    auto slice = [&](auto working, int b, uint32_t next, int nkk, int part) __attribute__((always_inline)) {
        constexpr int M = FP * FQ, NR = FP + FQ;
        const int l0 = part * LOADS / 2, nl = part < 0 ? 0 : (part + 1) * LOADS / 2 - l0;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            if (i >= l0 && i < l0 + nl) look_up(i);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            if constexpr (decltype(working)::value) {
                acc[m / FQ][m % FQ] = mfma32(fp[b][m / FQ], fq[b][m % FQ], acc[m / FQ][m % FQ]);
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    if (n >= m * 2 * NR / M && n < (m + 1) * 2 * NR / M) read_one(next, nkk, b ^ 1, n);  // in the first half
            }
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                if (i >= l0 + m * nl / M && i < l0 + (m + 1) * nl / M) issue(i);                        // towards the end
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // All but one and a half of the ring's stages are loaded ahead. Before a stage's last slice: wait for the next stage (those
    // after it stay under way) and for the workgroup; from then on nobody reads the present stage, and it takes the loads of
    // the stage NST further on, in this slice and the next.
    constexpr int NS = BK / 16;                              // slices of a stage
    auto loop = [&](auto working) __attribute__((always_inline)) {
        uint32_t here = lds0;
        if constexpr (decltype(working)::value) {
#pragma unroll
            for (int n = 0; n < FP + FQ; ++n) read_one(here, 0, 0, n);
        }
        for (int s = 0; s < ns; ++s) {
#pragma unroll
            for (int k = 0; k < NS - 1; ++k) slice(working, k & 1, here, k + 1, k == 0 ? 1 : -1);
            next_stage();
            here = here == lds0 + (NST - 1) * STAGE ? lds0 : here + STAGE;
            wait_stage<(NST - 2) * LOADS>();
            // everybody has looked up the rows up to `step`: half of the table takes the ones behind the other half
            if constexpr (OP == GROUPED_WGRAD) {
                if (step % (WINDOW / 2) == 0 && step + WINDOW / 2 < K) {
                    fill(step + WINDOW / 2, WINDOW / 2);
                    __syncthreads();
                }
            }
            slice(working, 1, here, 0, 0);                   // behind the last stage: a read of zeros, not used
        }
    };
    if (ns > 0) {
        if constexpr (OP == GROUPED_WGRAD) {
            fill(0, min(K, WINDOW));
            __syncthreads();
        }
#pragma unroll
        for (int s = 0; s < NST - 1; ++s) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                look_up(i);
                issue(i);
            }
            next_stage();
        }
#pragma unroll
        for (int i = 0; i < LOADS / 2; ++i) {
            look_up(i);
            issue(i);
        }
        wait_stage<(NST - 2) * LOADS + LOADS / 2>();
        if (works) loop(std::true_type{});
        else loop(std::false_type{});
        wait_stage<0>();
    }
    if (!works) return;
    // Lane l has row l % 32 of a fragment of results, columns 8 (v / 4) + 4 (l / 32) + v % 4. Stored from there, every row would get
    // 16 or 8 bytes at a time (16384 x 4096 results: 50 us); through LDS, where the ring was, 32 rows of a wave go out as runs of
    // whole lines. 16-byte chunk c of row r lies at c ^ r. The weights' gradient is the largest thing that passes here and nothing of
    // the call reads it again: it leaves around the L2, which keeps x and dy (512 MiB matrices of 32 experts: 1028 -> 939 us; the
    // other outputs gain nothing from that, and what follows reads them).
    constexpr int FO = SWIGLU ? FP / 2 : FP, COLS = 32 * FO;
    static_assert(NW * 32 * COLS * 4 <= NST * STAGE, "");
    uint8_t *rows = ring + wave * (32 * COLS * 4);
    const int n0 = p0 + wp * COLS;
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
        const int q = q0 + (wq * FQ + j) * 32 + i32;
        int row = -1;
        if (q < last_q) row = OP == GROUPED_FWD ? out_row(a.g, q, a.out_rows) : OP == GROUPED_DGRAD ? in_slot(a.g, q, a.out_rows) : q;
        if (__ballot(row >= 0) == 0) continue;
        auto results = [&](auto bf16) __attribute__((always_inline)) {
            constexpr int SIZE = decltype(bf16)::value ? 2 : 4, CHUNKS = COLS * SIZE / 16, ROWS = 64 / CHUNKS, PER = 16 / SIZE;
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < FO; ++i)
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    float y[4];
                    if constexpr (SWIGLU) {
                        float g[4], u[4];
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            g[v] = acc[2 * i][j][4 * v4 + v];
                            u[v] = acc[2 * i + 1][j][4 * v4 + v];
                        }
                        swiglu(g, u, y);
                    } else {
#pragma unroll
                        for (int v = 0; v < 4; ++v) y[v] = acc[i][j][4 * v4 + v];
                    }
                    const int c = (i * 32 + 8 * v4 + 4 * hh) / PER;
                    uint8_t *to = rows + i32 * (COLS * SIZE) + (c ^ (i32 & (CHUNKS - 1))) * 16;
                    if constexpr (SIZE == 4) *reinterpret_cast<f32x4_t *>(to) = f32x4_t{y[0], y[1], y[2], y[3]};
                    else *reinterpret_cast<uint2 *>(to + 8 * hh) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
                }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
            const int c = lane % CHUNKS, n = n0 + c * PER;
#pragma unroll
            for (int k = 0; k < 32 / ROWS; ++k) {
                const int r = k * ROWS + lane / CHUNKS, to = __shfl(row, r, 64);
                u32x4_t y = *reinterpret_cast<const u32x4_t *>(rows + r * (COLS * SIZE) + (c ^ (r & (CHUNKS - 1))) * 16);
                if (to < 0 || n >= P) continue;
                const int64_t at = ((OP == GROUPED_WGRAD ? (int64_t)group * a.n_out : 0) + to) * P + n;
                if constexpr (SIZE == 2) {
                    u32x4_t *half = reinterpret_cast<u32x4_t *>(static_cast<uint16_t *>(a.out) + at);
                    if (OP == GROUPED_WGRAD) __builtin_nontemporal_store(y, half);
                    else *half = y;
                } else {
                    f32x4_t v = __builtin_bit_cast(f32x4_t, y);
                    uint2 *half = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at);
                    f32x4_t *full = reinterpret_cast<f32x4_t *>(static_cast<float *>(a.out) + at);
                    if (OP == GROUPED_WGRAD && a.accumulate) {
                        if (a.out_bf16) {
                            const uint2 w = *half;
                            v += f32x4_t{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                                         __uint_as_float(w.y & 0xFFFF0000u)};
                            *half = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
                            continue;
                        }
                        v += *full;
                    }
                    if (OP == GROUPED_WGRAD) __builtin_nontemporal_store(v, full);
                    else *full = v;
                }
            }
            asm volatile("" ::: "memory");
        };
        if (a.out_bf16 && !(OP == GROUPED_WGRAD && a.accumulate)) results(std::true_type{});
        else results(std::false_type{});
    }
}

// ---------------------------------------------------------------------------
// Few rows to an expert and few tiles of weights: a workgroup has 16 weight rows (SwiGLU: 16 of gate and the same of up) and up to
// 16 positions of a group, the matrix instruction's 16 x 16 results; its waves take pieces of 128 columns in turn, FEW_AHEAD of
// them loaded at once, and their sums meet in LDS. Lane l has weight row (x row) l % 16 and columns 8 (l / 16) .. + 7 of each 32.
// The weights' stream bounds it where there is one (4096 x 8192, one token: 12.0 us, 5.6 TB/s), the launch and the dependent loads
// of offsets, index, rows and weights where there is little (16 experts of 1024 x 1024, one token: 5.5 us).
// ---------------------------------------------------------------------------
constexpr int FEW_WAVES = 8, FEW_AHEAD = 2, FEW_COLS = 128;

template <bool SWIGLU> __global__ __launch_bounds__(64 * FEW_WAVES, 4) void k_few_rows(GroupedArgs a, int most, int tiles_n) {
    constexpr int R = SWIGLU ? 2 : 1;
    __shared__ __attribute__((aligned(16))) f32x4_t part[FEW_WAVES][R][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i16 = lane & 15, q = lane >> 4;
    const int N = a.n_out, K = a.n_in;
    Tile t;
    int n0;
    if (!place(a.g, 16, 16, most, tiles_n, t, n0)) return;
    const int xr = t.begin + i16 < t.end ? in_row(a.g, t.begin + i16, a.a_rows) : -1, x_end = xr < 0 ? 0 : K - 8 * q;
    const uint16_t *x = a.a + (int64_t)max(xr, 0) * K + 8 * q;
    const uint16_t *w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = a.b + (((int64_t)t.group * R + r) * N + min(n0 + i16, N - 1)) * K + 8 * q;
    f32x4_t acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int k0 = wave * FEW_COLS; k0 < K; k0 += FEW_AHEAD * FEW_WAVES * FEW_COLS) {
        uint4 v[FEW_AHEAD][4], u[FEW_AHEAD][R][4];
#pragma unroll
        for (int i = 0; i < FEW_AHEAD; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = k0 + i * FEW_WAVES * FEW_COLS + 32 * s;
#pragma unroll
                for (int r = 0; r < R; ++r) u[i][r][s] = load_or_zeros(w[r] + k, k + 8 * q < K);
                v[i][s] = load_or_zeros(x + k, k < x_end);
            }
#pragma unroll
        for (int i = 0; i < FEW_AHEAD; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int r = 0; r < R; ++r) acc[r] = mfma16(v[i][s], u[i][r][s], acc[r]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) part[wave][r][lane] = acc[r];
    __syncthreads();
    // lane l's four values are positions 4 (l / 16) .. + 3 of weight row l % 16
    const float *sums = reinterpret_cast<const float *>(part);
    const int e = threadIdx.x, n = e & 15, pos = e >> 4;
    if (pos >= 16 || t.begin + pos >= t.end || n0 + n >= N) return;
    const int row = out_row(a.g, t.begin + pos, a.out_rows);
    if (row < 0) return;
    float y[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        y[r] = 0.f;
#pragma unroll
        for (int j = 0; j < FEW_WAVES; ++j) y[r] += sums[((j * R + r) * 64 + n + 16 * (pos >> 2)) * 4 + (pos & 3)];
    }
    const float z = SWIGLU ? swiglu(y[0], y[R - 1]) : y[0];
    const int64_t o = (int64_t)row * N + n0 + n;
    if (a.out_bf16) static_cast<__bf16 *>(a.out)[o] = (__bf16)z;
    else static_cast<float *>(a.out)[o] = z;
}

}  // namespace

namespace moe {

template <int OP, int FP, int FQ, int WP, int WQ, int BK, int NST, bool SWIGLU>
static hipError_t launch_tile(const GroupedArgs &a, hipStream_t st) {
    constexpr int TP = 32 * FP * WP / (SWIGLU ? 2 : 1), TQ = 32 * FQ * WQ, threads = 64 * WP * WQ;
    const int64_t tp = ((OP == GROUPED_FWD ? a.n_out : a.n_in) + TP - 1) / TP;
    const int64_t tq = OP == GROUPED_WGRAD ? (a.n_out + TQ - 1) / TQ : most_tiles(a.g, TQ);
    const int64_t blocks = (tp * tq * (OP == GROUPED_WGRAD ? a.g.n : 1) + 7) / 8 * 8;
    if (!grid_fits(blocks, threads)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_tile<OP, FP, FQ, WP, WQ, BK, NST, SWIGLU>), dim3((unsigned)blocks), dim3(threads), 0, st, a, (int)tp, (int)tq);
    return hipGetLastError();
}

template <bool SWIGLU> static hipError_t launch_few_rows(const GroupedArgs &a, hipStream_t st) {
    const int64_t tn = (a.n_out + 15) / 16, most = most_tiles(a.g, 16), blocks = (most * tn + 7) / 8 * 8;
    if (!grid_fits(blocks, 64 * FEW_WAVES)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_few_rows<SWIGLU>), dim3((unsigned)blocks), dim3(64 * FEW_WAVES), 0, st, a, (int)most, (int)tn);
    return hipGetLastError();
}

// The rules between the kernels stand at grouped_choice() and wgrad_256(). Other tiles: 16384 slots of 64 rows, weights of 4096 x 4096,
// 1737 us with 256 x 128 of 4 waves (128 x 64: 1910); 512 tokens of one matrix 28 with 128 x 64 (128 x 128: 30, 256 x 128: 46 to 55),
// its ring of three steps of 64 (300 x 4 rows 11; six 11 to 12, four of 32 13); 11709 tokens of 8 among 32 experts 2826 with 256 x
// 256 (4 waves of 128 x 128: 2956, 256 x 128: 3406 to 3606). Weights' gradient of few tiles (8192 rows of one 1024 x 1024 matrix: 64
// workgroups, 80 us): their LDS reads bound it, a ring of four steps takes as long.
template <int OP, bool SWIGLU> static hipError_t launch_op(const GroupedArgs &a, hipStream_t st) {
    if constexpr (OP == GROUPED_WGRAD) {
        if (wgrad_256(a.g.n, a.n_out, a.n_in)) return launch_tile<OP, 4, 2, 2, 4, 64, 2, false>(a, st);
        return launch_tile<OP, 2, 1, 2, 4, 64, 3, false>(a, st);
    } else {
        switch (grouped_choice(OP == GROUPED_DGRAD, SWIGLU, a.g.n, a.g.rows, a.n_out, a.n_in)) {
            case TILE_256_256: return launch_tile<OP, 4, 2, 2, 4, 64, 2, SWIGLU>(a, st);
            case TILE_256_128_8: return launch_tile<OP, 2, 2, 4, 2, 64, 3, SWIGLU>(a, st);
            case TILE_256_128_4: return launch_tile<OP, 4, 2, 2, 2, 32, 3, SWIGLU>(a, st);
            case FEW_ROWS:
                if constexpr (OP == GROUPED_FWD) return launch_few_rows<SWIGLU>(a, st);
                break;
            case TILE_128_64: break;
        }
        return launch_tile<OP, 2, 1, 2, 2, 64, 3, SWIGLU>(a, st);
    }
}

hipError_t launch_grouped(int op, const GroupedArgs &a, hipStream_t st) {
    if (op == GROUPED_WGRAD) return launch_op<GROUPED_WGRAD, false>(a, st);
    if (op == GROUPED_DGRAD) return launch_op<GROUPED_DGRAD, false>(a, st);
    return a.swiglu ? launch_op<GROUPED_FWD, true>(a, st) : launch_op<GROUPED_FWD, false>(a, st);
}

}  // namespace moe
