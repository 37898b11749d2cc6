// MXFP4 x MXFP4 products with weights that depend on the row's group, for
// gfx950: the experts of a sparse layer.
//
//   p[s][r] = sum_b 2^(xs + ws - 254) sum_{i in b} e2m1(xq[s]) e2m1(w[e(s)][r])
//   y = p, or with the gate silu(p[s][j]) p[s][n/2 + j]
//
//  * A tile is up to 256 sorted rows of one group against 256 of its weight
//    rows (128 x 128 where such tiles fit the card at once, two to a compute
//    unit).  The grid is as large as any distribution of the slots over the
//    groups needs; a workgroup finds its group from the offsets.  The rows of x
//    are gathered through the order, y's are scattered.
//  * Rows come in any number: the waves that share a weight row take every
//    other 32 rows of x, and a tile of fewer rows runs a loop with as many
//    products as 64 rows need (32768 x 4096 x 2816 over 64 experts, 278 us
//    where whole tiles took 301).
//  * With the gate a wave has weight rows of each half, so that the two meet in
//    its registers.
//  * Codes and scales go to v_mfma_scale_f32_32x32x64_f8f6f4 as they are
//    stored, through LDS in stages of 256 k, double-buffered, in rows whose
//    16-byte chunks are permuted against bank conflicts; scales are staged for
//    512 k.  A row of x is read from LDS into the registers of the one that the
//    matrix cores have just taken, so that 128 x 64 results and everything on
//    its way fit a wave's 256 registers (one loop body a stage: an exit in the
//    middle of two doubled the results' registers and spilled).
//
// Bound by the operands' way and the clock: 32768 slots of 64 experts, 4096 x
// 2816 with the gate, 282 us = 2.7 PFLOP/s (266 to 286 by card and clock; 240
// of 279 without the stages' loads, 168 on constant operands and without
// stores; no LDS conflicts, 78% of the requests hit L2; the matrix cores are
// busy 34% of the launch's cycles, 95 us at 2.0 GHz, and 40% of those in which
// their compute unit had work).  7996 slots of 16, 1440 x 5120 to f32 76 us (72
// to 80; 32 of them its 164 MB of results at the copy's rate, and some 780 tiles
// are three rounds on 256 compute units and a few more).  Not kept, on the first:
// 128-k stages with two workgroups a compute unit 342 (of 278), two stages in
// registers with 192-row tiles 294 (of 295), a touch of the lines three stages
// ahead 323 to 349, four waves of 128 x 128 336 (of 283), raised priority and
// other places of the loads and LDS stores 284 to 286 (of 283).  Few rows an
// expert are bound by the weights: 288 slots of 64 experts, 77 us (5.1 TB/s).
#include <type_traits>

#include "grouped_gemm.h"

namespace bqm {

template <int Q>
__device__ __forceinline__ v16f gg_mfma(u32x4 a, u32x4 b, v16f c, int sa, int sb) {
    const v8i va = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const v8i vb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    // formats 4, 4: e2m1 on both sides; scale byte Q of each scale dword
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va, vb, c, 4, 4, Q, sa, Q, sb);
}

// Workgroups reach the eight XCDs round-robin; of each 256 consecutive ones (a
// round, one per compute unit) an XCD's 32 take items that follow each other,
// so that its L2 serves each operand row to several of them.
__device__ __forceinline__ int xcd_item(int id, int count) {
    const int base = id & ~255, r = id & 255;
    return base + 256 <= count ? base + (r & 7) * 32 + (r >> 3) : id;
}

// A wave's results to their slots: lane holds column r32 and rows 8 (v / 4) +
// 4 g + v % 4 of each 32 x 32.  Of 16-bit values two lanes swap, so that each
// has two columns of one of two rows: half as many stores.  Past the caches,
// where the operands keep their room (7996 slots, 1440 x 5120: 78 us for 94).
template <typename T, int WM, int TM, int TN, bool GLU>
__device__ __forceinline__ void store_tile(T *y, int outs, const v16f (&acc)[TM][TN], int te, const int *slots, int j0) {
    const int lane = threadIdx.x & 63, r32 = lane & 31, g = lane >> 5;
#pragma unroll
    for (int i = 0; i < TM; i++) {
        if (i >= te) break;
#pragma unroll
        for (int v = 0; v < 16; v += 4) {
            const v4i s = *reinterpret_cast<const v4i *>(slots + i * 32 * WM + 2 * v + 4 * g);
#pragma unroll
            for (int c = 0; c < TN; c += GLU ? 2 : 1) {
                const int j = j0 + c * (GLU ? 16 : 32) + r32;
                float out[4];
#pragma unroll
                for (int e = 0; e < 4; e++) out[e] = GLU ? silu(acc[i][c][v + e]) * acc[i][c + (GLU ? 1 : 0)][v + e] : acc[i][c][v + e];
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (s[e] >= 0 && j < outs) __builtin_nontemporal_store(out[e], y + (int64_t)s[e] * outs + j);
                } else {
                    // even lanes: columns j, j + 1 of row e; odd ones: j - 1, j of row e + 1
                    const bool odd = lane & 1;
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float give = odd ? out[e] : out[e + 1];
                        const float got = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, give), 0xB1, 0xF, 0xF, false));
                        const T lo = (T)(odd ? got : out[e]), hi = (T)(odd ? out[e + 1] : got);
                        const int slot = odd ? s[e + 1] : s[e], col = j - (odd ? 1 : 0);
                        T *const to = y + (int64_t)slot * outs + col;
                        if (slot < 0) continue;
                        if (outs % 2 == 0) {   // rows are aligned to two values, and no pair crosses their end
                            typedef T T2 __attribute__((ext_vector_type(2), aligned(2)));
                            if (col < outs) __builtin_nontemporal_store(T2{lo, hi}, reinterpret_cast<T2 *>(to));
                        } else {
                            if (col < outs) to[0] = lo;
                            if (col + 1 < outs) to[1] = hi;
                        }
                    }
                }
            }
        }
    }
}

constexpr int kGgBlocks = 8;                   // scale blocks of a stage: 256 k, 4 steps
constexpr int kGgRowBytes = 16 * kGgBlocks;    // of a row in LDS

// WM x WN waves, each TM x TN tiles of 32 x 32.
template <int WM, int WN, int TM, int TN, bool GLU>
__global__ __launch_bounds__(64 * WM * WN, 2) void grouped_gemm_kernel(GgArgs a) {
    constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN, NT = 64 * WM * WN, ROWS = BM + BN;
    constexpr int COLS = GLU ? BN / 2 : BN;             // columns of y
    constexpr int CA = BM * 8 / NT, CB = BN * 8 / NT;   // 16-byte chunks per thread and stage
    constexpr int RS = NT / 8;                          // rows between a thread's chunks
    constexpr int SR = (ROWS + NT - 1) / NT;            // scale rows per thread
    static_assert(!GLU || TN % 2 == 0, "a wave's tiles are the gate's and the other half's in turn");
    static_assert(CA % TM == 0 && CB >= 1, "a thread's chunks of x go by 32 WM rows");
    __shared__ __attribute__((aligned(16))) uint8_t st[2][ROWS * kGgRowBytes];
    __shared__ int sc[2][4][SR * NT];   // scale dword j (blocks 4j .. 4j+3 of the superstage) of each row
    __shared__ __attribute__((aligned(16))) int slot_of[BM];                    // -1: not a row of y
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int r32 = lane & 31, g = lane >> 5;

    const GroupTile t = find_group(a.q, BM, a.ntiles, xcd_item(blockIdx.x, gridDim.x));
    if (t.group > a.q.groups) return;
    const int mtiles = (t.rows + BM - 1) / BM;
    const int mt = t.local % mtiles, nt = t.local / mtiles;
    const int first = t.first + mt * BM, rows = min(BM, t.rows - mt * BM);
    const int j0 = nt * COLS;
    const bool none = t.group == a.q.groups;   // slots of no group
    const int64_t rb = a.k / 2;
    const int nblk = a.k / 32;
    const int stages = (nblk + kGgBlocks - 1) / kGgBlocks;
    // (of no group: nothing is read)
    const uint8_t *const w = a.w + (int64_t)t.group * a.n * rb, *const ws = a.ws + (int64_t)t.group * a.n * nblk;
    const int half = GLU ? a.outs : 0;

    // row tid / 8 (+ RS per chunk) of each operand, 16-byte chunk tid % 8 of the
    // stage, stored in a slot of its LDS row such that sixteen rows' reads of one
    // chunk meet all of LDS's 64 banks: two rows fill them once, so it is every
    // other row that takes the next slot
    const int chunk = tid & 7, row = tid >> 3;
    auto slot = [](int r, int c) { return 16 * (c ^ ((r >> 1) & 7)); };
    // Blocks past the row's end repeat its last one: their scales are 2^-127 on
    // both sides, whose products vanish in any f32 sum.
    auto offset = [&](int s) { return 16u * (uint32_t)min(kGgBlocks * s + chunk, nblk - 1); };
    struct Regs {
        u32x4 a[CA], b[CB];
    };
    Regs R;
    // the weight rows of a tile follow each other (with the gate those of each
    // half), so that one offset a thread does for them
    const int wrows = none ? 0 : min(COLS, a.outs - j0);
    const __amdgpu_buffer_rsrc_t rB0 = mx_rsrc(w + j0 * rb, wrows * rb);
    const __amdgpu_buffer_rsrc_t rB1 = mx_rsrc(w + (j0 + half) * rb, wrows * rb);
    auto load_b = [&](Regs &R, int s) {
        const uint32_t ob = (uint32_t)((GLU ? row & 31 : row) * rb) + offset(s);
        // the row step stays in the per-lane offset, which the range check
        // covers: the scalar offset is added past it, and a ragged tile's rows
        // past the last would be read
#pragma unroll
        for (int i = 0; i < CB; i++) {
            const uint32_t step = (uint32_t)((GLU ? (RS == 32 ? i >> 1 : i) * 32 : i * RS) * rb);
            const __amdgpu_buffer_rsrc_t rB = !GLU ? rB0 : (RS == 32 ? i & 1 : wave & 4) ? rB1 : rB0;
            R.b[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rB, ob + step, 0, 0));
        }
    };
    // the first weights are on their way while the slots are looked up
    load_b(R, 0);
    for (int i = tid; i < BM; i += NT) {
        const unsigned s = i < rows ? (unsigned)a.q.order[first + i] : ~0u;
        slot_of[i] = s < (unsigned)a.q.slots ? (int)s : -1;
    }
    __syncthreads();
    if (none) {
        for (int i = tid; i < rows * COLS; i += NT) {
            const int s = slot_of[i / COLS], j = j0 + i % COLS;
            if (s >= 0 && j < a.outs) store_as(a.y, (int64_t)s * a.outs + j, 0.0f, a.y_type);
        }
        return;
    }
    // the row of x of tile row i; rows that are none read row 0
    auto x_row = [&](int i) { return (int64_t)(max(slot_of[min(i, rows - 1)], 0) / a.top); };
    // the weight row of tile row i, past the last one the last one; with the
    // gate a wave's tiles of 32 rows are of either half in turn
    auto w_row = [&](int i) {
        if (GLU) {
            const int j = min(j0 + 32 * (i >> 6) + (i & 31), a.outs - 1);
            return (int64_t)(j + ((i >> 5) & 1) * half);
        }
        return (int64_t)min(j0 + i, a.outs - 1);
    };
    // x is at most 4 GiB, so a row's place in it is a 32-bit offset
    uint32_t pa[CA];
#pragma unroll
    for (int i = 0; i < CA; i++) pa[i] = (uint32_t)(x_row(row + i * RS) * rb);
    const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(a.xq), (short)0, (int)0xFFFFFFFF, 0x00020000);
    auto load_a = [&](Regs &R, int s, auto tes) {
        const uint32_t at = offset(s);
#pragma unroll
        for (int i = 0; i < CA * decltype(tes)::value / TM; i++) R.a[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rA, pa[i] + at, 0, 0));
    };
    const int at = row * kGgRowBytes + slot(row, chunk);
    auto store_a = [&](uint8_t *p, const Regs &R, auto tes) {
#pragma unroll
        for (int i = 0; i < CA * decltype(tes)::value / TM; i++) *reinterpret_cast<u32x4 *>(p + at + i * RS * kGgRowBytes) = R.a[i];
    };
    auto store_b = [&](uint8_t *p, const Regs &R) {
#pragma unroll
        for (int i = 0; i < CB; i++) *reinterpret_cast<u32x4 *>(p + at + (BM + i * RS) * kGgRowBytes) = R.b[i];
    };
    // Scales: a thread loads the 16 bytes of a row that 512 k need.
    const uint8_t *ps[SR];
#pragma unroll
    for (int i = 0; i < SR; i++) {
        const int rr = tid + i * NT;
        ps[i] = rr < BM ? a.xs + x_row(rr) * nblk : ws + w_row(min(rr - BM, BN - 1)) * nblk;
    }
    struct ScaleRegs {
        unsigned v[SR][4];
    };
    auto load_scales = [&](ScaleRegs &S, int super) {
        const int b0 = min(16 * super, (nblk - 1) / 16 * 16);   // past the end: not used
#pragma unroll
        for (int i = 0; i < SR; i++) scale_bytes(ps[i], b0, nblk, S.v[i]);
    };
    auto store_scales = [&](const ScaleRegs &S, int buf) {
#pragma unroll
        for (int i = 0; i < SR; i++)
#pragma unroll
            for (int q = 0; q < 4; q++) sc[buf][q][tid + i * NT] = (int)S.v[i][q];
    };

    v16f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++)
#pragma unroll
            for (int v = 0; v < 16; v++) acc[i][j][v] = 0.0f;

    // Lane half g takes chunks 4g .. 4g+3 of a stage, one per step, so its four
    // scales of a row are one dword.  Operands are read a step ahead: a row of
    // x into the registers of the one that this step has just multiplied, a
    // weight row into a second set.
    const int rowA = wm * 32 + r32, rowB = BM + wn * 32 * TN + r32;
    u32x4 va[TM], vb[2][TN];
    int ta[TM], tb[2][TN];
    auto read_a = [&](const uint8_t *p, auto q, int i) {
        constexpr int Q = decltype(q)::value;
        va[i] = *reinterpret_cast<const u32x4 *>(p + (rowA + 32 * WM * i) * kGgRowBytes + slot(r32, 4 * g + Q));
    };
    auto read_b = [&](const uint8_t *p, auto q, int j) {
        constexpr int Q = decltype(q)::value;
        vb[Q & 1][j] = *reinterpret_cast<const u32x4 *>(p + (rowB + 32 * j) * kGgRowBytes + slot(r32, 4 * g + Q));
    };
    auto scale = [&](int s, int r) { return sc[(s >> 1) & 1][2 * (s & 1) + g][r]; };   // of stage s, row r
    constexpr std::integral_constant<int, 0> q0{};
    constexpr std::integral_constant<int, 1> q1{};
    constexpr std::integral_constant<int, 2> q2{};
    constexpr std::integral_constant<int, 3> q3{};
    constexpr std::false_type no{};
    constexpr std::true_type yes{};

    // The tile's rows in 32 WM: the waves' share of x beyond them is left out.
    auto product = [&](auto tes) {
        constexpr int TE = decltype(tes)::value;
        ScaleRegs S;
        load_scales(S, 0);
        load_a(R, 0, tes);
        store_scales(S, 0);
        store_a(st[0], R, tes);
        store_b(st[0], R);
        load_a(R, 1, tes);
        load_b(R, 1);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TE; i++) {
            read_a(st[0], q0, i);
            ta[i] = scale(0, rowA + 32 * WM * i);
        }
#pragma unroll
        for (int j = 0; j < TN; j++) {
            read_b(st[0], q0, j);
            tb[0][j] = scale(0, rowB + 32 * j);
        }
        // Stage s is in st[s & 1], its first operands in registers, stage s + 1
        // on its way to R.  The barrier stands before the last step: by then
        // every wave has read this stage's operands and stored its share of the
        // next one.  The scales of the next two stages are loaded in an even
        // stage and stored in an odd one.
#pragma unroll 1
        for (int s = 0; s < stages; s++) {
            const uint8_t *const here = st[s & 1];
            uint8_t *const there = st[(s & 1) ^ 1];
            if (s & 1)
                store_scales(S, ((s >> 1) + 1) & 1);
            else
                load_scales(S, (s >> 1) + 1);
            auto step = [&](auto q, auto next, const uint8_t *p) {
                constexpr int Q = decltype(q)::value;
#pragma unroll
                for (int j = 0; j < TN; j++) read_b(p, next, j);
                if constexpr (Q == 3) {
#pragma unroll
                    for (int j = 0; j < TN; j++) tb[1][j] = scale(s + 1, rowB + 32 * j);
                }
#pragma unroll
                for (int i = 0; i < TE; i++) {
#pragma unroll
                    for (int j = 0; j < TN; j++) acc[i][j] = gg_mfma<Q>(va[i], vb[Q & 1][j], acc[i][j], ta[i], tb[0][j]);
                    read_a(p, next, i);
                    if constexpr (Q == 3) ta[i] = scale(s + 1, rowA + 32 * WM * i);
                }
            };
            // LDS accesses between the matrix products, W stores beside each row of x
            auto order = [&](auto scales_too, auto stores) {
                constexpr bool scales = decltype(scales_too)::value;
                constexpr int W = decltype(stores)::value;
                __builtin_amdgcn_sched_group_barrier(0x100, scales ? TN + (TN + 1) / 2 : TN, 0);
#pragma unroll
                for (int i = 0; i < TE; i++) {
                    __builtin_amdgcn_sched_group_barrier(0x008, TN, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, scales ? 2 : 1, 0);
                    if constexpr (W > 0) __builtin_amdgcn_sched_group_barrier(0x200, W, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            };
            constexpr std::integral_constant<int, 0> none{};
            constexpr std::integral_constant<int, (CA * TE / TM + CB + 2 * TE - 1) / (2 * TE)> some{};
            step(q0, q1, here);
            order(no, none);
            step(q1, q2, here);
            store_a(there, R, tes);
            order(no, some);
            step(q2, q3, here);
            store_b(there, R);
            order(no, some);
            load_a(R, s + 2, tes);
            load_b(R, s + 2);
            __syncthreads();
            step(q3, q0, there);
            order(yes, none);
#pragma unroll
            for (int j = 0; j < TN; j++) tb[0][j] = tb[1][j];
        }
    };
    const int te = (rows + 32 * WM - 1) / (32 * WM);
    if (TM >= 4 && te == 4)
        product(std::integral_constant<int, TM >= 4 ? 4 : TM>{});
    else if (TM >= 3 && te == 3)
        product(std::integral_constant<int, TM >= 3 ? 3 : TM>{});
    else if (TM >= 2 && te == 2)
        product(std::integral_constant<int, TM >= 2 ? 2 : TM>{});
    else
        product(std::integral_constant<int, 1>{});

    if (a.y_type == BQM_F32)
        store_tile<float, WM, TM, TN, GLU>(static_cast<float *>(a.y), a.outs, acc, te, slot_of + wm * 32, j0 + wn * (GLU ? 16 : 32) * TN);
    else if (a.y_type == BQM_F16)
        store_tile<_Float16, WM, TM, TN, GLU>(static_cast<_Float16 *>(a.y), a.outs, acc, te, slot_of + wm * 32, j0 + wn * (GLU ? 16 : 32) * TN);
    else
        store_tile<__bf16, WM, TM, TN, GLU>(static_cast<__bf16 *>(a.y), a.outs, acc, te, slot_of + wm * 32, j0 + wn * (GLU ? 16 : 32) * TN);
}

template <int WM, int WN, int TM, int TN, bool GLU>
static int launch_gg(GgArgs a, hipStream_t s) {
    constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN, NT = 64 * WM * WN, COLS = GLU ? BN / 2 : BN;
    a.ntiles = (int)(((int64_t)a.outs + COLS - 1) / COLS);
    const int64_t grid = most_tiles(a.q.slots, a.q.groups, BM) * a.ntiles;
    if (grid * NT > 0x7FFFFFFFll) return BQM_EUNSUPPORTED;   // work items that a dispatch counts
    hipLaunchKernelGGL((grouped_gemm_kernel<WM, WN, TM, TN, GLU>), dim3((unsigned)grid), dim3(NT), 0, s, a);
    return launch_status();
}

// Large tiles move the operands least often; where about as many small ones as
// the card takes at once do (two to a compute unit), those end sooner.
// Measured (large, small; us): 32768 x 4096 x 2816 of 64 278, 343; 4096 x 4096
// x 2816 of 16 62, 54; 2048 x 4096 x 4096 of 8 41, 45; 1024 x 2048 x 2048 of 16
// 20.5, 16.4; 64 slots x 1024 x 4096 of 16 12.2, 11.7; 32 x 4096 x 1024 of 8 17.4, 14.8.
// Where the small ones leave half of the card idle and k is long, waves that
// share k may do better (grouped_stream.hip).
template <bool GLU>
static int launch_gg_by_rows(const GgArgs &a, hipStream_t s) {
    const int64_t used = a.q.groups < a.q.slots ? a.q.groups : a.q.slots;
    const int64_t small = (a.q.slots / 128 + (used + 1) / 2) * (((int64_t)a.n + 127) / 128);
    const int cus = device_cus();
    if (grouped_stream_applies(a, small, cus)) return grouped_stream(a, cus, s);
    return small <= 2 * cus ? launch_gg<2, 2, 2, 2, GLU>(a, s) : launch_gg<2, 4, 4, 2, GLU>(a, s);
}

}  // namespace bqm

extern "C" int bqm_mxfp4_grouped_gemm(const uint8_t *w, const uint8_t *ws, const uint8_t *xq, const uint8_t *xs,
                                      const int *offsets, const int *order, void *y, int y_type, int glu, int rows,
                                      int slots, int groups, int k, int n, void *stream) {
    using namespace bqm;
    if (!w || !ws || !xq || !xs || !offsets || !order || !y || !type_known(y_type)) return BQM_EINVAL;
    if (rows < 1 || slots < 1 || slots % rows != 0 || groups < 1 || groups > BQM_MAX_GROUPS) return BQM_EINVAL;
    if (k < 32 || n < 1 || (glu && n % 2 != 0)) return BQM_EINVAL;
    if (k % 32 != 0 || !aligned(w, 16) || !aligned(xq, 16)) return BQM_EUNSUPPORTED;
    if (k > 1 << 22 || (int64_t)rows * (k / 2) > 0xFFFFFFF0ll) return BQM_EUNSUPPORTED;   // a tile's rows in 31 bits, x in 32
    if (!aligned(offsets, 4) || !aligned(order, 4) || !aligned(y, type_bytes(y_type))) return BQM_EUNSUPPORTED;
    hipStream_t s = as_stream(stream);
    const GgArgs a = {w, ws, xq, xs, y, {offsets, order, groups, slots}, y_type, slots / rows, k, n, glu ? n / 2 : n, 0};
    return glu ? launch_gg_by_rows<true>(a, s) : launch_gg_by_rows<false>(a, s);
}
