// MXFP4 x MXFP4 product for gfx950: codes of 4 bits with a power of two per
// 32 on both sides, f32 accumulation.
//
//   y[t][r] = sum_b 2^(xs[t][b] + ws[r][b] - 254) sum_{i in b} e2m1(xq) e2m1(w)
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes 32 x 64 codes of each side and one
// scale byte per row and 32 k, so codes and scales go to the matrix cores as
// they are stored: nothing is decoded and nothing folded.
#include <type_traits>

#include "values.h"

namespace bqm {

constexpr int kMgStage = 256;                 // k of an LDS stage: 8 scale blocks, 4 MFMA steps
constexpr int kMgRowBytes = kMgStage / 2;
constexpr int kMgRowStride = kMgRowBytes + 16;   // padded LDS row: conflict-free 16-byte reads

struct MgArgs {
    const uint8_t *w, *ws, *xq, *xs;
    float *y;
    int m, k, n;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mg_rsrc(const void *base, int64_t bytes) {
    const uint32_t b = bytes <= 0 ? 0u : bytes > 0x7FFFFFF0ll ? 0x7FFFFFF0u : (uint32_t)bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)b, 0x00020000);
}

template <int Q>
__device__ __forceinline__ v16f mg_mfma(u32x4 a, u32x4 b, v16f c, int sa, int sb) {
    const v8i va = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const v8i vb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    // formats 4, 4: e2m1 on both sides; scale byte Q of each scale dword
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va, vb, c, 4, 4, Q, sa, Q, sb);
}

// WM x WN waves, each TM x TN tiles of 32 x 32 (tokens x weight rows).
// WIDE: scale rows are whole, aligned dwords (k % 128 == 0); else bytes.
template <int WM, int WN, int TM, int TN, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN) void mxfp4_gemm_kernel(MgArgs a) {
    constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN, NT = 64 * WM * WN;
    constexpr int CA = BM * 8 / NT, CB = BN * 8 / NT;   // 16-byte chunks per thread and stage
    constexpr int RS = NT / 8;                          // rows between a thread's chunks
    __shared__ __attribute__((aligned(16))) uint8_t st[2][(BM + BN) * kMgRowStride];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int r32 = lane & 31, g = lane >> 5;
    const int64_t m0 = (int64_t)blockIdx.y * BM, n0 = (int64_t)blockIdx.x * BN;
    const int64_t rb = a.k / 2;
    const int nblk = a.k / 32;
    const int stages = (nblk + 7) / 8;

    const int64_t rowsA = a.m - m0 < BM ? a.m - m0 : BM, rowsB = a.n - n0 < BN ? a.n - n0 : BN;
    const __amdgpu_buffer_rsrc_t rA = mg_rsrc(a.xq + m0 * rb, rowsA * rb);
    const __amdgpu_buffer_rsrc_t rB = mg_rsrc(a.w + n0 * rb, rowsB * rb);
    const __amdgpu_buffer_rsrc_t rSA = mg_rsrc(a.xs + m0 * nblk, rowsA * nblk);
    const __amdgpu_buffer_rsrc_t rSB = mg_rsrc(a.ws + n0 * nblk, rowsB * nblk);

    // thread: row tid / 8 (+ RS per chunk), 16-byte chunk tid % 8 of the stage
    const int chunk = tid & 7, row = tid >> 3;
    u32x4 ca[CA], cb[CB];
    auto load = [&](int s) {
        // chunks past the row's end are read as zeros
        const uint32_t off = 8 * s + chunk < nblk ? (uint32_t)(row * rb + 16 * (8 * s + chunk)) : 0x80000000u;
#pragma unroll
        for (int i = 0; i < CA; i++)
            ca[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rA, off + (uint32_t)(i * RS * rb), 0, 0));
#pragma unroll
        for (int i = 0; i < CB; i++)
            cb[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rB, off + (uint32_t)(i * RS * rb), 0, 0));
    };
    auto store = [&](uint8_t *p) {
        const int at = row * kMgRowStride + 16 * chunk;
#pragma unroll
        for (int i = 0; i < CA; i++) *reinterpret_cast<u32x4 *>(p + at + i * RS * kMgRowStride) = ca[i];
#pragma unroll
        for (int i = 0; i < CB; i++) *reinterpret_cast<u32x4 *>(p + at + (BM + i * RS) * kMgRowStride) = cb[i];
    };
    // lane half g takes scale blocks 4g .. 4g+3 of a stage, one per step, so
    // its four scales of a row are one dword
    auto scales = [&](const __amdgpu_buffer_rsrc_t &r, int row0, int s) {
        const int b = 8 * s + 4 * g;
        const uint32_t at = (uint32_t)((row0 + r32) * nblk + b);
        if constexpr (WIDE) {
            return (int)__builtin_amdgcn_raw_buffer_load_b32(r, b < nblk ? at : 0x80000000u, 0, 0);
        } else {
            unsigned v = 0;
#pragma unroll
            for (int q = 0; q < 4; q++)
                v |= (unsigned)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, b + q < nblk ? at + q : 0x80000000u, 0, 0) << (8 * q);
            return (int)v;
        }
    };
    int sa[TM], sb[TN];
    auto load_scales = [&](int s) {
#pragma unroll
        for (int i = 0; i < TM; i++) sa[i] = scales(rSA, wm * 32 * TM + 32 * i, s);
#pragma unroll
        for (int j = 0; j < TN; j++) sb[j] = scales(rSB, wn * 32 * TN + 32 * j, s);
    };

    v16f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++)
#pragma unroll
            for (int v = 0; v < 16; v++) acc[i][j][v] = 0.0f;

    load(0);
    load_scales(0);
    store(st[0]);
    __syncthreads();
    for (int s = 0; s < stages; s++) {
        const uint8_t *const pa = st[s & 1] + (wm * 32 * TM + r32) * kMgRowStride + 64 * g;
        const uint8_t *const pb = st[s & 1] + (BM + wn * 32 * TN + r32) * kMgRowStride + 64 * g;
        int ta[TM], tb[TN];
#pragma unroll
        for (int i = 0; i < TM; i++) ta[i] = sa[i];
#pragma unroll
        for (int j = 0; j < TN; j++) tb[j] = sb[j];
        if (s + 1 < stages) {
            load(s + 1);
            load_scales(s + 1);
        }
        auto step = [&](auto q) {
            constexpr int Q = decltype(q)::value;
            u32x4 va[TM], vb[TN];
#pragma unroll
            for (int i = 0; i < TM; i++) va[i] = *reinterpret_cast<const u32x4 *>(pa + i * 32 * kMgRowStride + 16 * Q);
#pragma unroll
            for (int j = 0; j < TN; j++) vb[j] = *reinterpret_cast<const u32x4 *>(pb + j * 32 * kMgRowStride + 16 * Q);
#pragma unroll
            for (int i = 0; i < TM; i++)
#pragma unroll
                for (int j = 0; j < TN; j++) acc[i][j] = mg_mfma<Q>(va[i], vb[j], acc[i][j], ta[i], tb[j]);
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
        if (s + 1 < stages) store(st[(s + 1) & 1]);
        __syncthreads();
    }

#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) {
            const int64_t col = n0 + wn * 32 * TN + j * 32 + r32;
            if (col >= a.n) continue;
#pragma unroll
            for (int v = 0; v < 16; v++) {
                const int64_t t = m0 + wm * 32 * TM + i * 32 + 8 * (v >> 2) + 4 * g + (v & 3);
                if (t < a.m) a.y[t * a.n + col] = acc[i][j][v];
            }
        }
}

template <int WM, int WN, int TM, int TN>
static int launch_mg(const MgArgs &a, hipStream_t s) {
    constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN;
    const dim3 grid((a.n + BN - 1) / BN, (a.m + BM - 1) / BM);
    // the dispatch counts rows of tiles in 16 bits and work items in 32
    if (grid.y > 65535 || (int64_t)grid.x * (64 * WM * WN) > 0xFFFFFFFFll) return BQM_EUNSUPPORTED;
    if (a.k % 128 == 0 && aligned(a.ws, 4) && aligned(a.xs, 4))
        hipLaunchKernelGGL((mxfp4_gemm_kernel<WM, WN, TM, TN, true>), grid, dim3(64 * WM * WN), 0, s, a);
    else
        hipLaunchKernelGGL((mxfp4_gemm_kernel<WM, WN, TM, TN, false>), grid, dim3(64 * WM * WN), 0, s, a);
    return launch_status();
}

}  // namespace bqm

extern "C" int bqm_mxfp4_gemm(const uint8_t *w, const uint8_t *ws, const uint8_t *xq, const uint8_t *xs, float *y,
                              int m, int k, int n, void *stream) {
    using namespace bqm;
    if (!w || !ws || !xq || !xs || !y) return BQM_EINVAL;
    if (m < 1 || k < 32 || n < 1) return BQM_EINVAL;
    if (k % 32 != 0 || !aligned(w, 16) || !aligned(xq, 16) || !aligned(y, 4)) return BQM_EUNSUPPORTED;
    if (k > 1 << 22) return BQM_EUNSUPPORTED;   // the rows of a tile in 31 bits
    const MgArgs a = {w, ws, xq, xs, y, m, k, n};
    return launch_mg<2, 4, 2, 2>(a, as_stream(stream));
}
