// MXFP4 x MXFP4 products with weights that depend on the row's group, for
// gfx950: the experts of a sparse layer.
//
//   p[s][r] = sum_b 2^(xs + ws - 254) sum_{i in b} e2m1(xq[s]) e2m1(w[e(s)][r])
//   y = p, or with the gate silu(p[s][j]) p[s][n/2 + j]
//
// A tile is up to 32 TM WM sorted rows of one group against 32 TN WN of its
// weight rows; with the gate a wave has 32 rows of each half, so that the two
// meet in its registers.  The grid is as large as any distribution of the
// slots over the groups needs; a workgroup finds its group from the offsets.
// The rows of x are gathered through the order, y's are scattered.  Codes and
// scales go to v_mfma_scale_f32_32x32x64_f8f6f4 as they are stored, through
// LDS in stages of 256 k, double-buffered; scales are staged for 1024 k.
#include <type_traits>

#include "groups.h"

namespace bqm {

struct GgArgs {
    const uint8_t *w, *ws, *xq, *xs;
    void *y;
    Grouping q;
    int y_type, top;
    int k, n, outs;      // outs: columns of y
    int ntiles;
};

constexpr int kGgStage = 256;                 // k of an LDS stage: 8 scale blocks, 4 MFMA steps
constexpr int kGgRowBytes = kGgStage / 2;
constexpr int kGgSuper = 4;                   // stages whose scales are staged together: 32 bytes a row

template <int Q>
__device__ __forceinline__ v16f gg_mfma(u32x4 a, u32x4 b, v16f c, int sa, int sb) {
    const v8i va = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const v8i vb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    // formats 4, 4: e2m1 on both sides; scale byte Q of each scale dword
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va, vb, c, 4, 4, Q, sa, Q, sb);
}

// The 32 scale bytes from block b0 on of the row of nblk bytes at p, at any
// alignment; zeros past its end.
__device__ __forceinline__ void scale_bytes(const uint8_t *p, int b0, int nblk, unsigned (&v)[8]) {
    if (b0 + 32 <= nblk || nblk >= 32) {
        const int from = min(b0, nblk - 32), shift = b0 - from;   // uniform
#pragma unroll
        for (int q = 0; q < 2; q++) {
            u32x4 u;
            __builtin_memcpy(&u, p + from + 16 * q, 16);
#pragma unroll
            for (int e = 0; e < 4; e++) v[4 * q + e] = u[e];
        }
        if (shift > 0) {
#pragma unroll
            for (int d = 4; d >= 1; d /= 2)
                if ((shift >> 2) & d) {
#pragma unroll
                    for (int q = 0; q < 8; q++) v[q] = q + d < 8 ? v[q + d] : 0;
                }
#pragma unroll
            for (int q = 0; q < 8; q++) v[q] = __builtin_amdgcn_alignbyte(q < 7 ? v[q + 1] : 0, v[q], shift & 3);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; q++) {
            v[q] = 0;
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (4 * q + e < nblk - b0) v[q] |= (unsigned)p[b0 + 4 * q + e] << (8 * e);
        }
    }
}

template <int WM, int WN, int TM, int TN, bool GLU>
__global__ __launch_bounds__(64 * WM * WN) void grouped_gemm_kernel(GgArgs a) {
    constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN, NT = 64 * WM * WN, ROWS = BM + BN;
    constexpr int COLS = GLU ? BN / 2 : BN;             // columns of y
    constexpr int CA = BM * 8 / NT, CB = BN * 8 / NT;   // 16-byte chunks per thread and stage
    constexpr int RS = NT / 8;                          // rows between a thread's chunks
    constexpr int SR = (ROWS + NT - 1) / NT;            // scale rows per thread
    static_assert(!GLU || TN == 2, "a wave's two tiles are the gate's and the other half's");
    static_assert(CA >= 1 && RS % 32 == 0, "");
    __shared__ __attribute__((aligned(16))) uint8_t st[2][ROWS * kGgRowBytes];
    __shared__ int sc[2][2 * kGgSuper][SR * NT];   // scale dword j (blocks 4j .. 4j+3 of the superstage) of each row
    __shared__ int slot_of[BM];                    // -1: not a row of y
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int r32 = lane & 31, g = lane >> 5;

    const GroupTile t = find_group(a.q, BM, a.ntiles, blockIdx.x);
    if (t.group > a.q.groups) return;
    const int mtiles = (t.rows + BM - 1) / BM;
    const int mt = t.local % mtiles, nt = t.local / mtiles;
    const int first = t.first + mt * BM, rows = min(BM, t.rows - mt * BM);
    const int j0 = nt * COLS;
    for (int i = tid; i < BM; i += NT) {
        const unsigned s = i < rows ? (unsigned)a.q.order[first + i] : ~0u;
        slot_of[i] = s < (unsigned)a.q.slots ? (int)s : -1;
    }
    __syncthreads();
    if (t.group == a.q.groups) {   // slots of no group
        for (int i = tid; i < rows * COLS; i += NT) {
            const int s = slot_of[i / COLS], j = j0 + i % COLS;
            if (s >= 0 && j < a.outs) store_as(a.y, (int64_t)s * a.outs + j, 0.0f, a.y_type);
        }
        return;
    }

    const int64_t rb = a.k / 2;
    const int nblk = a.k / 32;
    const int stages = (nblk + 7) / 8;
    const uint8_t *const w = a.w + (int64_t)t.group * a.n * rb, *const ws = a.ws + (int64_t)t.group * a.n * nblk;
    const int half = GLU ? a.outs : 0;

    // row tid / 8 (+ RS per chunk) of each operand, 16-byte chunk tid % 8 of
    // the stage, stored at slot chunk ^ (row % 8) so that eight rows' reads of
    // one chunk meet eight different slots
    const int chunk = tid & 7, row = tid >> 3;
    // the row of x of tile row i; rows that are none read row 0
    auto x_row = [&](int i) { return (int64_t)(max(slot_of[min(i, rows - 1)], 0) / a.top); };
    // the weight row of tile row i, past the last one the last one
    auto w_row = [&](int i) {
        if (GLU) {
            const int j = min(j0 + 32 * (i >> 6) + (i & 31), a.outs - 1);
            return (int64_t)(j + ((i >> 5) & 1) * half);
        }
        return (int64_t)min(j0 + i, a.outs - 1);
    };
    const uint8_t *pa[CA], *pb[CB];
#pragma unroll
    for (int i = 0; i < CA; i++) pa[i] = a.xq + x_row(row + i * RS) * rb;
#pragma unroll
    for (int i = 0; i < CB; i++) pb[i] = w + w_row(row + i * RS) * rb;
    struct Regs {
        u32x4 a[CA], b[CB];
    };
    // blocks past the row's end repeat its last one in x and are zeros in w
    auto load = [&](Regs &R, int s) {
        const int c = 8 * s + chunk;
        const int at = 16 * min(c, nblk - 1);
#pragma unroll
        for (int i = 0; i < CA; i++) R.a[i] = *reinterpret_cast<const u32x4 *>(pa[i] + at);
#pragma unroll
        for (int i = 0; i < CB; i++) R.b[i] = *reinterpret_cast<const u32x4 *>(pb[i] + at);
        if (c >= nblk) {
#pragma unroll
            for (int i = 0; i < CB; i++) R.b[i] = u32x4{0, 0, 0, 0};
        }
    };
    auto store = [&](uint8_t *p, const Regs &R) {
        const int at = row * kGgRowBytes + 16 * (chunk ^ (row & 7));
#pragma unroll
        for (int i = 0; i < CA; i++) *reinterpret_cast<u32x4 *>(p + at + i * RS * kGgRowBytes) = R.a[i];
#pragma unroll
        for (int i = 0; i < CB; i++) *reinterpret_cast<u32x4 *>(p + at + (BM + i * RS) * kGgRowBytes) = R.b[i];
    };
    // Scales: a thread loads the 32 bytes of a row that four stages need.
    const uint8_t *ps[SR];
#pragma unroll
    for (int i = 0; i < SR; i++) {
        const int rr = tid + i * NT;
        ps[i] = rr < BM ? a.xs + x_row(rr) * nblk : ws + w_row(min(rr - BM, BN - 1)) * nblk;
    }
    struct ScaleRegs {
        unsigned v[SR][2 * kGgSuper];
    };
    auto load_scales = [&](ScaleRegs &S, int super) {
        const int b0 = 8 * kGgSuper * super;
        if (b0 >= nblk) return;
#pragma unroll
        for (int i = 0; i < SR; i++) scale_bytes(ps[i], b0, nblk, S.v[i]);
    };
    auto store_scales = [&](const ScaleRegs &S, int buf) {
#pragma unroll
        for (int i = 0; i < SR; i++)
#pragma unroll
            for (int q = 0; q < 2 * kGgSuper; q++) sc[buf][q][tid + i * NT] = (int)S.v[i][q];
    };

    v16f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++)
#pragma unroll
            for (int v = 0; v < 16; v++) acc[i][j][v] = 0.0f;

    // Lane half g takes chunks 4g .. 4g+3 of a stage, one per step, so its four
    // scales of a row are one dword.
    const int rowA = wm * 32 * TM + r32, rowB = BM + wn * 32 * TN + r32;
    auto step = [&](const uint8_t *p, const int (&ta)[TM], const int (&tb)[TN], auto q) {
        constexpr int Q = decltype(q)::value;
        const int slot = 16 * ((4 * g + Q) ^ (r32 & 7));
        u32x4 va[TM], vb[TN];
#pragma unroll
        for (int i = 0; i < TM; i++) va[i] = *reinterpret_cast<const u32x4 *>(p + (rowA + 32 * i) * kGgRowBytes + slot);
#pragma unroll
        for (int j = 0; j < TN; j++) vb[j] = *reinterpret_cast<const u32x4 *>(p + (rowB + 32 * j) * kGgRowBytes + slot);
#pragma unroll
        for (int i = 0; i < TM; i++)
#pragma unroll
            for (int j = 0; j < TN; j++) acc[i][j] = gg_mfma<Q>(va[i], vb[j], acc[i][j], ta[i], tb[j]);
    };
    Regs R;
    ScaleRegs S;
    load_scales(S, 0);
    load(R, 0);
    store_scales(S, 0);
    store(st[0], R);
    __syncthreads();
#pragma unroll 1
    for (int s = 0; s < stages; s++) {
        const int super = s / kGgSuper, in = s % kGgSuper;
        load(R, s + 1);
        if (in == 0) load_scales(S, super + 1);
        int ta[TM], tb[TN];
        const int(*const scales)[SR * NT] = &sc[super & 1][2 * in + g];
#pragma unroll
        for (int i = 0; i < TM; i++) ta[i] = scales[0][rowA + 32 * i];
#pragma unroll
        for (int j = 0; j < TN; j++) tb[j] = scales[0][rowB + 32 * j];
        const uint8_t *const p = st[s & 1];
        step(p, ta, tb, std::integral_constant<int, 0>{});
        step(p, ta, tb, std::integral_constant<int, 1>{});
        step(p, ta, tb, std::integral_constant<int, 2>{});
        step(p, ta, tb, std::integral_constant<int, 3>{});
        store(st[(s + 1) & 1], R);
        if (in == 0) store_scales(S, (super + 1) & 1);
        __syncthreads();
    }

    // Lane: column r32, rows 8 (v / 4) + 4 g + v % 4.
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int v = 0; v < 16; v++) {
            const int s = slot_of[wm * 32 * TM + i * 32 + 8 * (v >> 2) + 4 * g + (v & 3)];
            if (s < 0) continue;
            if constexpr (GLU) {
                const int j = j0 + wn * 32 + r32;
                if (j < a.outs) store_as(a.y, (int64_t)s * a.outs + j, silu(acc[i][0][v]) * acc[i][1][v], a.y_type);
            } else {
#pragma unroll
                for (int c = 0; c < TN; c++) {
                    const int j = j0 + wn * 32 * TN + c * 32 + r32;
                    if (j < a.outs) store_as(a.y, (int64_t)s * a.outs + j, acc[i][c][v], a.y_type);
                }
            }
        }
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

template <bool GLU>
static int launch_gg_by_rows(const GgArgs &a, hipStream_t s) {
    return launch_gg<2, 2, 2, 2, GLU>(a, s);
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
    if (!aligned(offsets, 4) || !aligned(order, 4) || !aligned(y, type_bytes(y_type))) return BQM_EUNSUPPORTED;
    hipStream_t s = as_stream(stream);
    const GgArgs a = {w, ws, xq, xs, y, {offsets, order, groups, slots}, y_type, slots / rows, k, n, glu ? n / 2 : n, 0};
    return glu ? launch_gg_by_rows<true>(a, s) : launch_gg_by_rows<false>(a, s);
}
