// MXFP4 x MXFP4 product for gfx950: codes of 4 bits with a power of two per
// 32 on both sides, f32 accumulation.
//
//   y[t][r] = sum_b 2^(xs[t][b] + ws[r][b] - 254) sum_{i in b} e2m1(xq) e2m1(w)
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes 32 x 64 codes of each side and one
// scale byte per row and 32 k, so codes and scales go to the matrix cores as
// they are stored: nothing is decoded and nothing folded.
//
//  * Large outputs: tiles of 192 tokens x 256 weight rows; small ones and what
//    is left of a round of those: 128 x 128 (large_columns).
//  * Codes pass through LDS in stages of 256 k, double-buffered, in rows whose
//    16-byte chunks are permuted against bank conflicts; the scales of 1024 k
//    are staged at once, one row a thread, whose bytes may be unaligned (odd
//    counts of blocks; loaded byte by byte they made 2137 x 7712 x 7399 take
//    273 us instead of 137).  A scale dword per lane and stage from memory
//    instead took a third of the time at 2048 x 8192 x 8192.
//  * y is stored past the caches.
//
// 512 x 4096 x 20480: 34 to 39 us (2.5 PFLOP/s at best); 3001 x 5120 x 17408:
// 167 to 178 us (3.2) a few at a time, 187 to 199 in long rows of calls, when
// the clock falls, the matrix cores busy 40% and 46% of the compute units'
// time.  Few tiles leave compute units idle (512 x 4096 x 4096, 128 tiles, 18.4
// us), and k runs in whole groups of four stages (512 x 4128 x 20480 55 us).
// 2048 x 8192 x 8192 takes 111 us (2.5 PFLOP/s), and 57 (4.8) with every
// load and LDS read taken out, on constant operands: what the matrix cores
// leave is the operands' way through LDS and the stores, which a workgroup does
// not overlap with its next tile.
#include <type_traits>

#include "mxfp4.h"

namespace bqm {

constexpr int kMgStage = 256;                 // k of an LDS stage: 8 scale blocks, 4 MFMA steps
constexpr int kMgRowBytes = kMgStage / 2;
constexpr int kMgSuper = 4;                   // stages whose scales are staged together: 32 bytes a row

constexpr int kMgLargeM = 192, kMgLargeN = 256;   // the large tile: 8 waves of 96 x 64
constexpr int kMgSmall = 128;                     // the small one: 4 waves of 64 x 64

template <int Q>
__device__ __forceinline__ v16f mg_mfma(u32x4 a, u32x4 b, v16f c, int sa, int sb) {
    const v8i va = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const v8i vb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    // formats 4, 4: e2m1 on both sides; scale byte Q of each scale dword
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va, vb, c, 4, 4, Q, sa, Q, sb);
}

// Tile of workgroup id.  Workgroups reach the eight XCDs round-robin; of each
// 256 consecutive ones (a round, one per compute unit) an XCD's 32 take tiles
// that follow each other down strips of eight tile rows, so that its L2 serves
// each operand row to several of them.
__device__ __forceinline__ void mg_tile(int id, int mtiles, int ntiles, int &mt, int &nt) {
    const int base = id & ~255, r = id & 255;
    if (base + 256 <= mtiles * ntiles) id = base + (r & 7) * 32 + (r >> 3);
    const int strip = id / (8 * ntiles), in = id - strip * 8 * ntiles;
    const int high = min(8, mtiles - 8 * strip);
    mt = 8 * strip + in % high;
    nt = in / high;
}

// WM x WN waves, each TM x TN tiles of 32 x 32 (tokens x weight rows).
// SW: scale rows are aligned to 16 bytes (16) or to nothing (1).
template <int WM, int WN, int TM, int TN, int SW>
__global__ __launch_bounds__(64 * WM * WN) void mxfp4_gemm_kernel(MgArgs a) {
    constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN, NT = 64 * WM * WN, ROWS = BM + BN;
    constexpr int CA = BM * 8 / NT, CB = BN * 8 / NT;   // 16-byte chunks per thread and stage
    constexpr int RS = NT / 8;                          // rows between a thread's chunks
    constexpr int SR = (ROWS + NT - 1) / NT;            // scale rows per thread
    __shared__ __attribute__((aligned(16))) uint8_t st[2][ROWS * kMgRowBytes];
    __shared__ int sc[2][2 * kMgSuper][SR * NT];   // scale dword j (blocks 4j .. 4j+3 of the superstage) of each row
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int r32 = lane & 31, g = lane >> 5;
    int mt, nt;
    mg_tile(blockIdx.x, a.mtiles, a.ntiles, mt, nt);
    const int64_t m0 = (int64_t)mt * BM, n0 = (int64_t)nt * BN;
    const int64_t rb = a.k / 2;
    const int nblk = a.k / 32;
    const int supers = (nblk + 8 * kMgSuper - 1) / (8 * kMgSuper);

    const int64_t rowsA = a.m - m0 < BM ? a.m - m0 : BM, rowsB = a.n - n0 < BN ? a.n - n0 : BN;
    const __amdgpu_buffer_rsrc_t rA = mx_rsrc(a.xq + m0 * rb, rowsA * rb);
    const __amdgpu_buffer_rsrc_t rB = mx_rsrc(a.w + n0 * rb, rowsB * rb);
    const __amdgpu_buffer_rsrc_t rSA = mx_rsrc(a.xs + m0 * nblk, rowsA * nblk);
    const __amdgpu_buffer_rsrc_t rSB = mx_rsrc(a.ws + n0 * nblk, rowsB * nblk);

    struct Regs {
        u32x4 a[CA], b[CB];
    };
    // thread: row tid / 8 (+ RS per chunk), 16-byte chunk tid % 8 of the stage,
    // stored at slot chunk ^ (row % 8) so that eight rows' reads of one chunk
    // meet eight different slots
    const int chunk = tid & 7, row = tid >> 3;
    // stages past the last read zeros
    auto load = [&](Regs &R, int s) {
        const uint32_t off = 8 * s + chunk < nblk ? (uint32_t)(row * rb + 16 * (8 * s + chunk)) : 0x80000000u;
#pragma unroll
        for (int i = 0; i < CA; i++)
            R.a[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rA, off + (uint32_t)(i * RS * rb), 0, 0));
#pragma unroll
        for (int i = 0; i < CB; i++)
            R.b[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rB, off + (uint32_t)(i * RS * rb), 0, 0));
    };
    auto store = [&](uint8_t *p, const Regs &R) {
        const int at = row * kMgRowBytes + 16 * (chunk ^ (row & 7));
#pragma unroll
        for (int i = 0; i < CA; i++) *reinterpret_cast<u32x4 *>(p + at + i * RS * kMgRowBytes) = R.a[i];
#pragma unroll
        for (int i = 0; i < CB; i++) *reinterpret_cast<u32x4 *>(p + at + (BM + i * RS) * kMgRowBytes) = R.b[i];
    };
    // Scales: a thread loads the 32 bytes of a row that four stages need.
    struct ScaleRegs {
        unsigned v[SR][2 * kMgSuper];
    };
    auto load_scales = [&](ScaleRegs &S, int super) {
        const int b0 = 8 * kMgSuper * super;
#pragma unroll
        for (int i = 0; i < SR; i++) {
            const int rr = tid + i * NT;
            const bool isA = rr < BM;   // uniform: BM is a multiple of the wave
            const __amdgpu_buffer_rsrc_t r = isA ? rSA : rSB;
            const uint32_t at = (uint32_t)((isA ? rr : rr - BM) * nblk + b0);
            if constexpr (SW == 16) {
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                        r, b0 + 16 * q < nblk ? at + 16 * q : 0x80000000u, 0, 0));
#pragma unroll
                    for (int e = 0; e < 4; e++) S.v[i][4 * q + e] = v[e];
                }
            } else if (b0 + 8 * kMgSuper <= nblk) {
                // 32 bytes at any alignment; a row past the last takes the last's
                const int64_t q0 = isA ? m0 + min((int64_t)rr, rowsA - 1) : n0 + min((int64_t)(rr - BM), rowsB - 1);
                const uint8_t *const p = (isA ? a.xs : a.ws) + q0 * nblk + b0;
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    u32x4 v;
                    __builtin_memcpy(&v, p + 16 * q, 16);
#pragma unroll
                    for (int e = 0; e < 4; e++) S.v[i][4 * q + e] = v[e];
                }
            } else {
                // the row's last few bytes
#pragma unroll
                for (int q = 0; q < 2 * kMgSuper; q++) {
                    S.v[i][q] = 0;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int b = 4 * q + e;
                        S.v[i][q] |= (unsigned)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                                         r, b0 + b < nblk ? at + b : 0x80000000u, 0, 0) << (8 * e);
                    }
                }
            }
        }
    };
    auto store_scales = [&](const ScaleRegs &S, int buf) {
#pragma unroll
        for (int i = 0; i < SR; i++)
#pragma unroll
            for (int q = 0; q < 2 * kMgSuper; q++) sc[buf][q][tid + i * NT] = (int)S.v[i][q];
    };

    v16f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++)
#pragma unroll
            for (int v = 0; v < 16; v++) acc[i][j][v] = 0.0f;

    // Operands of a step and scales of a stage, read one step ahead.  Lane half
    // g takes chunks 4g .. 4g+3 of a stage, one per step, so its four scales
    // of a row are one dword.
    const int rowA = wm * 32 * TM + r32, rowB = BM + wn * 32 * TN + r32;
    u32x4 va[2][TM], vb[2][TN];
    int ta[2][TM], tb[2][TN];
    auto read = [&](const uint8_t *p, auto q) {
        constexpr int Q = decltype(q)::value;
        const int slot = 16 * ((4 * g + Q) ^ (r32 & 7));
#pragma unroll
        for (int i = 0; i < TM; i++) va[Q & 1][i] = *reinterpret_cast<const u32x4 *>(p + (rowA + 32 * i) * kMgRowBytes + slot);
#pragma unroll
        for (int j = 0; j < TN; j++) vb[Q & 1][j] = *reinterpret_cast<const u32x4 *>(p + (rowB + 32 * j) * kMgRowBytes + slot);
    };
    auto read_scales = [&](const int (*scales)[SR * NT], int slot) {
#pragma unroll
        for (int i = 0; i < TM; i++) ta[slot][i] = scales[g][rowA + 32 * i];
#pragma unroll
        for (int j = 0; j < TN; j++) tb[slot][j] = scales[g][rowB + 32 * j];
    };
    auto multiply = [&](auto q, int slot) {
        constexpr int Q = decltype(q)::value;
#pragma unroll
        for (int i = 0; i < TM; i++)
#pragma unroll
            for (int j = 0; j < TN; j++) acc[i][j] = mg_mfma<Q>(va[Q & 1][i], vb[Q & 1][j], acc[i][j], ta[slot][i], tb[slot][j]);
    };
    constexpr std::integral_constant<int, 0> q0{};
    constexpr std::integral_constant<int, 1> q1{};
    constexpr std::integral_constant<int, 2> q2{};
    constexpr std::integral_constant<int, 3> q3{};

    Regs R;
    ScaleRegs S;
    load_scales(S, 0);
    load(R, 0);
    store_scales(S, 0);
    store(st[0], R);
    load(R, 1);
    __syncthreads();
    read(st[0], q0);
    read_scales(&sc[0][0], 0);
    // Stage s = 4 super + J is in st[J & 1], its first operands are in
    // registers, and stage s + 1 is on its way to R.  The
    // barrier stands before the last step: by then every wave has read this
    // stage's operands and stored its share of the next one, whose first
    // operands arrive while the last step multiplies.  The next superstage's
    // scales are loaded in a superstage's first stage and stored in its third.
    auto stage = [&](int s, auto pos, int super) {
        constexpr int J = decltype(pos)::value;
        uint8_t *const here = st[J & 1], *const there = st[(J + 1) & 1];
        if constexpr (J == 0) load_scales(S, super + 1);
        read(here, q1);
        multiply(q0, J & 1);
        read(here, q2);
        multiply(q1, J & 1);
        store(there, R);
        if constexpr (J == 2) store_scales(S, (super + 1) & 1);
        load(R, s + 2);
        read(here, q3);
        multiply(q2, J & 1);
        // LDS accesses between the MFMAs: an even share of the three steps'
        // reads after each, and of the writes after those of the last two
#pragma unroll
        for (int r = 0; r < 3 * TM * TN; r++) {
            if (r == 0) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, (TM + TN + TM * TN - 1) / (TM * TN), 0);
            if (r >= TM * TN) __builtin_amdgcn_sched_group_barrier(0x200, (CA + CB + 2 * TM * TN - 1) / (2 * TM * TN), 0);
        }
        __syncthreads();
        read(there, q0);
        read_scales(J == 3 ? &sc[(super + 1) & 1][0] : &sc[super & 1][2 * ((J + 1) & 3)], (J + 1) & 1);
        multiply(q3, J & 1);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
        for (int r = 0; r < TM * TN; r++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2 * (TM + TN) / (TM * TN) + 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);   // nothing of the next stage moves up
    };
    // whole superstages: the stages past the row's end multiply zeros
#pragma unroll 1
    for (int super = 0; super < supers; super++) {
        const int s = super * kMgSuper;
        stage(s, q0, super);
        stage(s + 1, q1, super);
        stage(s + 2, q2, super);
        stage(s + 3, q3, super);
    }

    // Lane: column r32, rows 8 (v / 4) + 4 g + v % 4.  y is written past the
    // caches: nothing here reads it again, and the operands keep their room.
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) {
            const int64_t col = n0 + wn * 32 * TN + j * 32 + r32;
            if (col >= a.n) continue;
#pragma unroll
            for (int v = 0; v < 16; v++) {
                const int64_t t = m0 + wm * 32 * TM + i * 32 + 8 * (v >> 2) + 4 * g + (v & 3);
                if (t < a.m) __builtin_nontemporal_store(acc[i][j][v], a.y + t * a.ldy + col);
            }
        }
}

template <int WM, int WN, int TM, int TN>
static int launch_mg(MgArgs a, hipStream_t s) {
    constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN, NT = 64 * WM * WN;
    a.mtiles = (a.m + BM - 1) / BM;
    a.ntiles = (a.n + BN - 1) / BN;
    const int64_t grid = (int64_t)a.mtiles * a.ntiles;
    if (scale_load(a.k / 32, a.ws, a.xs) == 16)
        hipLaunchKernelGGL((mxfp4_gemm_kernel<WM, WN, TM, TN, 16>), dim3((unsigned)grid), dim3(NT), 0, s, a);
    else
        hipLaunchKernelGGL((mxfp4_gemm_kernel<WM, WN, TM, TN, 1>), dim3((unsigned)grid), dim3(NT), 0, s, a);
    return launch_status();
}

// Estimated microseconds (measured at k = 4096, 5120 and 8192): the large tile
// takes 1.2 per stage and 11 besides for each round of one per compute unit;
// the small one, two to a compute unit, 0.65 and 1.2 for each that a compute
// unit gets, or 0.56 and 6 if it gets a single one (k = 4096 15 us, 8192 24,
// 16384 41, 17408 46).
static double large_cost(int64_t rounds, int stages) { return rounds * (1.2 * stages + 11.0); }
static double small_cost(int64_t each, int stages) {
    return each == 0 ? 0.0 : each == 1 ? 0.56 * stages + 6.0 : each * (0.65 * stages + 1.2);
}

static int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Columns of the output that the large tile takes, the small one taking the
// rest: all, none, or as many whole rounds of large tiles as fit, whichever
// is estimated to end first, at `best` us.
static int large_columns(int m, int k, int n, int cus, double &best) {
    const int stages = (int)up(k, 1024) * 4;
    const int64_t mt = up(m, kMgLargeM), nt = up(n, kMgLargeN), rounds = mt * nt / cus;
    const int64_t whole = rounds * cus / mt * kMgLargeN;   // columns of the whole rounds
    auto small = [&](int64_t cols) { return small_cost(up(up(m, kMgSmall) * up(cols, kMgSmall), cus), stages); };
    best = small(n);
    int cols = 0;
    if (rounds > 0 && whole < n && large_cost(rounds, stages) + small(n - whole) < best) {
        best = large_cost(rounds, stages) + small(n - whole);
        cols = (int)whole;
    }
    if (large_cost(up(mt * nt, cus), stages) < best) {
        best = large_cost(up(mt * nt, cus), stages);
        cols = n;
    }
    return cols;
}

}  // namespace bqm

extern "C" int bqm_mxfp4_gemm(const uint8_t *w, const uint8_t *ws, const uint8_t *xq, const uint8_t *xs, float *y,
                              int m, int k, int n, void *stream) {
    using namespace bqm;
    if (!w || !ws || !xq || !xs || !y) return BQM_EINVAL;
    if (m < 1 || k < 32 || n < 1) return BQM_EINVAL;
    if (k % 32 != 0 || !aligned(w, 16) || !aligned(xq, 16) || !aligned(y, 4)) return BQM_EUNSUPPORTED;
    if (k > 1 << 22) return BQM_EUNSUPPORTED;   // the rows of a tile in 31 bits
    // tile numbers in 32 bits, and the work items that a dispatch counts
    if (up(m, kMgSmall) * up(n, kMgSmall) * 512 > 0x7FFFFFFFll) return BQM_EUNSUPPORTED;
    hipStream_t s = as_stream(stream);
    MgArgs a = {w, ws, xq, xs, y, n, m, k, n, 0, 0};
    double cost;
    const int cols = large_columns(m, k, n, device_cus(), cost);
    // unaligned scale rows that end inside the last 32 bytes cost the tiles a
    // round of byte loads (463 x 288 x 91 12 us, 1302 x 8672 x 335 37, where the
    // estimate says 8 and 26)
    if (k / 32 % (8 * kMgSuper) != 0 && scale_load(k / 32, ws, xs) != 16) cost += 8.0;
    const int groups = mxfp4_stream_groups(m, k, n, device_cus(), cost);
    if (groups > 0) return mxfp4_stream(a, groups, s);
    if (cols > 0) {
        a.n = cols;
        const int rc = launch_mg<2, 4, 3, 2>(a, s);
        if (rc || cols == n) return rc;
        a.w += (int64_t)cols * (k / 2);
        a.ws += (int64_t)cols * (k / 32);
        a.y += cols;
        a.n = n - cols;
    }
    return launch_mg<2, 2, 2, 2>(a, s);
}
