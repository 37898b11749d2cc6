// Root-mean-square norm with the residual's addition for gfx950, written as
// plain values or as the 8-bit operands of the projection matmuls.
//
//   s = x + res (f32),  h = s rounded to x's type,
//   y = s * (1 / sqrt(sum(s^2) / k + eps)) * gain,
// then q8_1 per 32 values or e4m3 per 128 values of the f32 y.
//
// HBM-bound: x and res are read once and h and y written once, so a row stays
// in registers between the sum of squares and the scaling.
//  * A row is cut into pieces of four values; thread i of the row's NT owns
//    pieces i, i + NT, ... (four of them).  A wave has a row of k <= 1024 to
//    itself (no barrier); otherwise a workgroup of k/16 threads, rounded up
//    to whole waves, has it (k <= 16384); beyond that the workgroup reads the
//    row twice, the second time mostly from its L2.
//  * The sum of squares is one fma chain per thread (16 values), a DPP tree
//    over the wave, then the waves' sums in order: f32, the order a function
//    of k alone, so a token's norm is the same bits in decode and in prefill.
//  * A 32-value block is 8 neighbouring lanes and a 128-value block 32 of
//    them, so the block maxima are DPP steps on values already in registers.
//  * ALN: rows aligned to four elements move in 16-byte (f32) or 8-byte
//    pieces; otherwise the same pieces move element by element, with the same
//    arithmetic, for odd k and odd strides.
#include "values.h"

namespace bqm {

enum { kOutF32, kOutSame, kOutQ81, kOutE4m3 };

constexpr int kNormPieces = 4;          // pieces of four values per thread
constexpr int kNormMaxThreads = 1024;
constexpr int kNormWaveK = 64 * 4 * kNormPieces;
constexpr int kNormRegK = kNormMaxThreads * 4 * kNormPieces;
constexpr int kNormMaxGrid = 1 << 20;   // rows beyond it are taken in turn
constexpr int kNormMaxK = 1 << 30;      // 32-bit positions within a row

struct NormArgs {
    const void *x, *res;
    const float *gain;
    void *h, *y;
    float *scale;   // xds (q8_1) or xs (e4m3)
    int64_t ldx, ldr, ldh;
    float eps;
    int m, k;
};

template <typename T, bool ALN>
__device__ __forceinline__ v4f load4(const T *p, int i, int k) {
    v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (ALN) {
        if (i < k) v = __builtin_convertvector(*reinterpret_cast<const typename Vec<T>::x4 *>(p + i), v4f);
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (i + e < k) v[e] = (float)p[i + e];
    }
    return v;
}

template <typename T, bool ALN>
__device__ __forceinline__ void store4(T *p, int i, int k, v4f v) {
    if constexpr (ALN) {
        if (i < k) *reinterpret_cast<typename Vec<T>::x4 *>(p + i) = __builtin_convertvector(v, typename Vec<T>::x4);
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (i + e < k) p[i + e] = (T)v[e];
    }
}

__device__ __forceinline__ float clamp448n(float v) { return fminf(fmaxf(v, -448.0f), 448.0f); }

// One piece of y: values i .. i+3 of row t.  Every lane of the wave takes
// part (block maxima); lanes past k hold zeros and store nothing.
template <typename T, int OUT, bool ALN>
__device__ __forceinline__ void emit(const NormArgs &a, int64_t t, int i, v4f y) {
    const int64_t at = t * a.k;
    if constexpr (OUT == kOutF32) {
        store4<float, ALN>(static_cast<float *>(a.y) + at, i, a.k, y);
    } else if constexpr (OUT == kOutSame) {
        store4<T, ALN>(static_cast<T *>(a.y) + at, i, a.k, y);
    } else if constexpr (OUT == kOutQ81) {
        const Q81Lane r = q8_1_block_lane(make_float4(y[0], y[1], y[2], y[3]));
        int sum = r.qsum;
        sum += __builtin_amdgcn_update_dpp(0, sum, 0xB1, 0xF, 0xF, false);
        sum += __builtin_amdgcn_update_dpp(0, sum, 0x4E, 0xF, 0xF, false);
        sum += __builtin_amdgcn_update_dpp(0, sum, 0x141, 0xF, 0xF, false);
        if (i < a.k) {
            static_cast<unsigned *>(a.y)[(at + i) >> 2] = r.packed;
            if ((threadIdx.x & 7) == 0)
                reinterpret_cast<float2 *>(a.scale)[(at + i) >> 5] = make_float2(r.d, r.d * (float)sum);
        }
    } else {
        float big = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
        big = swap16_max(dpp_absmax16(big));
        float mul = 0.0f, s = 0.0f;
        if (big > 0.0f) {
            mul = 448.0f / big;
            s = big / 448.0f;
        }
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448n(y[0] * mul), clamp448n(y[1] * mul), 0, false);
        const int q = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448n(y[2] * mul), clamp448n(y[3] * mul), lo, true);
        if (i < a.k) {
            static_cast<int *>(a.y)[(at + i) >> 2] = q;
            if ((threadIdx.x & 31) == 0) a.scale[t * ((a.k + 127) >> 7) + (i >> 7)] = s;
        }
    }
}

// Sum over the workgroup, on every thread; `red` is a buffer that nobody has
// read since the last barrier but one.
__device__ __forceinline__ float block_sum(float v, float *red) {
    v = wave_sum(v);
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < waves; i++) v += red[i];
    return v;
}

__device__ __forceinline__ float inv_rms(float sum, int k, float eps) { return 1.0f / sqrtf(sum / (float)k + eps); }

__device__ __forceinline__ float squares(v4f v, float acc) {
#pragma unroll
    for (int e = 0; e < 4; e++) acc = __builtin_fmaf(v[e], v[e], acc);
    return acc;
}

// WAVE: a wave per row; else a workgroup per row.  LONG: the row is longer
// than the registers hold and is read twice.
template <typename T, int OUT, bool ALN, bool WAVE, bool LONG>
__global__ __launch_bounds__(WAVE ? 256 : kNormMaxThreads) void norm_kernel(NormArgs a) {
    __shared__ float red[2][kNormMaxThreads / 64];
    const int lane = WAVE ? threadIdx.x & 63 : threadIdx.x;
    const int nt = WAVE ? 64 : blockDim.x;
    const int64_t step = (int64_t)gridDim.x * (WAVE ? 4 : 1);
    int64_t t = (int64_t)blockIdx.x * (WAVE ? 4 : 1) + (WAVE ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0);
    for (int turn = 0; t < a.m; t += step, turn ^= 1) {
        const T *x = static_cast<const T *>(a.x) + t * a.ldx;
        const T *res = a.res ? static_cast<const T *>(a.res) + t * a.ldr : nullptr;
        T *h = static_cast<T *>(a.h) + t * a.ldh;
        float acc = 0.0f;
        if constexpr (!LONG) {
            v4f s[kNormPieces], g[kNormPieces];
#pragma unroll
            for (int c = 0; c < kNormPieces; c++) s[c] = load4<T, ALN>(x, 4 * (lane + c * nt), a.k);
            if (res) {
                v4f r[kNormPieces];
#pragma unroll
                for (int c = 0; c < kNormPieces; c++) r[c] = load4<T, ALN>(res, 4 * (lane + c * nt), a.k);
#pragma unroll
                for (int c = 0; c < kNormPieces; c++) s[c] += r[c];
            }
#pragma unroll
            for (int c = 0; c < kNormPieces; c++)
                g[c] = a.gain ? load4<float, ALN>(a.gain, 4 * (lane + c * nt), a.k) : v4f{1.0f, 1.0f, 1.0f, 1.0f};
#pragma unroll
            for (int c = 0; c < kNormPieces; c++) acc = squares(s[c], acc);
            if (res) {
#pragma unroll
                for (int c = 0; c < kNormPieces; c++) store4<T, ALN>(h, 4 * (lane + c * nt), a.k, s[c]);
            }
            const float inv = inv_rms(WAVE ? wave_sum(acc) : block_sum(acc, red[turn]), a.k, a.eps);
#pragma unroll
            for (int c = 0; c < kNormPieces; c++) {
                if (4 * c * nt < a.k) emit<T, OUT, ALN>(a, t, 4 * (lane + c * nt), s[c] * inv * g[c]);
            }
        } else {
            for (int i = 4 * lane; i - 4 * lane < a.k; i += 4 * nt) {
                v4f s = load4<T, ALN>(x, i, a.k);
                if (res) s += load4<T, ALN>(res, i, a.k);
                acc = squares(s, acc);
            }
            const float inv = inv_rms(block_sum(acc, red[turn]), a.k, a.eps);
            // h may be x or res: each value is read and then written by one thread
            for (int i = 4 * lane; i - 4 * lane < a.k; i += 4 * nt) {
                v4f s = load4<T, ALN>(x, i, a.k);
                if (res) {
                    s += load4<T, ALN>(res, i, a.k);
                    store4<T, ALN>(h, i, a.k, s);
                }
                const v4f g = a.gain ? load4<float, ALN>(a.gain, i, a.k) : v4f{1.0f, 1.0f, 1.0f, 1.0f};
                emit<T, OUT, ALN>(a, t, i, s * inv * g);
            }
        }
    }
}

template <typename T, int OUT, bool ALN>
static int launch_norm(const NormArgs &a, hipStream_t s) {
    const int64_t rows = a.m;
    if (a.k <= kNormWaveK) {
        const int64_t grid = (rows + 3) / 4;
        hipLaunchKernelGGL((norm_kernel<T, OUT, ALN, true, false>), dim3((unsigned)(grid < kNormMaxGrid ? grid : kNormMaxGrid)),
                           dim3(256), 0, s, a);
        return launch_status();
    }
    const unsigned grid = (unsigned)(rows < kNormMaxGrid ? rows : kNormMaxGrid);
    if (a.k <= kNormRegK) {
        const int nt = (a.k + 64 * 4 * kNormPieces - 1) / (64 * 4 * kNormPieces) * 64;
        hipLaunchKernelGGL((norm_kernel<T, OUT, ALN, false, false>), dim3(grid), dim3(nt), 0, s, a);
    } else {
        hipLaunchKernelGGL((norm_kernel<T, OUT, ALN, false, true>), dim3(grid), dim3(kNormMaxThreads), 0, s, a);
    }
    return launch_status();
}

template <typename T, int OUT>
static int launch_aligned(const NormArgs &a, hipStream_t s) {
    const uintptr_t in = 4 * sizeof(T);
    const uintptr_t out = OUT == kOutF32 ? 16 : OUT == kOutSame ? in : 1;
    const bool rows4 = a.m == 1 || (a.ldx % 4 == 0 && (!a.res || (a.ldr % 4 == 0 && a.ldh % 4 == 0)));
    const bool aln = a.k % 4 == 0 && rows4 && aligned(a.x, in) && aligned(a.res, in) && aligned(a.h, in) &&
                     aligned(a.gain, 16) && aligned(a.y, out);
    return aln ? launch_norm<T, OUT, true>(a, s) : launch_norm<T, OUT, false>(a, s);
}

template <int OUT>
static int launch_typed(const NormArgs &a, int x_type, hipStream_t s) {
    if (x_type == BQM_F16) return launch_aligned<_Float16, OUT>(a, s);
    if (x_type == BQM_BF16) return launch_aligned<__bf16, OUT>(a, s);
    return launch_aligned<float, OUT>(a, s);
}

// The checks that every form shares, in the order of the return codes.
static int norm_check(const NormArgs &a, int x_type) {
    if (!a.x || !a.y || !a.res != !a.h) return BQM_EINVAL;
    if (a.m < 1 || a.k < 1 || !type_known(x_type)) return BQM_EINVAL;
    if (!(a.eps >= 0.0f) || a.eps > 3.4e38f) return BQM_EINVAL;
    if (a.k > kNormMaxK) return BQM_EUNSUPPORTED;
    if (a.m > 1 && (a.ldx < a.k || (a.res && (a.ldr < a.k || a.ldh < a.k)))) return BQM_EUNSUPPORTED;
    const uintptr_t e = type_bytes(x_type);
    if (!aligned(a.x, e) || !aligned(a.res, e) || !aligned(a.h, e) || !aligned(a.gain, 4)) return BQM_EUNSUPPORTED;
    return BQM_OK;
}

}  // namespace bqm

extern "C" int bqm_add_rmsnorm(const void *x, int64_t ldx, const void *res, int64_t ldr, const float *gain, float eps,
                               void *h, int64_t ldh, void *y, int x_type, int y_type, int m, int k, void *stream) {
    using namespace bqm;
    const NormArgs a = {x, res, gain, h, y, nullptr, ldx, ldr, ldh, eps, m, k};
    const int rc = norm_check(a, x_type);
    if (rc) return rc;
    if (!type_known(y_type)) return BQM_EINVAL;
    if (y_type != BQM_F32 && y_type != x_type) return BQM_EUNSUPPORTED;
    if (!aligned(y, type_bytes(y_type))) return BQM_EUNSUPPORTED;
    hipStream_t s = as_stream(stream);
    if (y_type == BQM_F32) return launch_typed<kOutF32>(a, x_type, s);
    return x_type == BQM_F16 ? launch_aligned<_Float16, kOutSame>(a, s) : launch_aligned<__bf16, kOutSame>(a, s);
}

extern "C" int bqm_add_rmsnorm_q8_1(const void *x, int64_t ldx, const void *res, int64_t ldr, const float *gain,
                                    float eps, void *h, int64_t ldh, int8_t *xq, float *xds, int x_type, int m, int k,
                                    void *stream) {
    using namespace bqm;
    const NormArgs a = {x, res, gain, h, xq, xds, ldx, ldr, ldh, eps, m, k};
    const int rc = norm_check(a, x_type);
    if (rc) return rc;
    if (!xds || k < kQK) return BQM_EINVAL;
    if (k % kQK != 0 || !aligned(xq, 4) || !aligned(xds, 8)) return BQM_EUNSUPPORTED;
    return launch_typed<kOutQ81>(a, x_type, as_stream(stream));
}

extern "C" int bqm_add_rmsnorm_e4m3_blk(const void *x, int64_t ldx, const void *res, int64_t ldr, const float *gain,
                                        float eps, void *h, int64_t ldh, uint8_t *xq, float *xs, int x_type, int m,
                                        int k, void *stream) {
    using namespace bqm;
    const NormArgs a = {x, res, gain, h, xq, xs, ldx, ldr, ldh, eps, m, k};
    const int rc = norm_check(a, x_type);
    if (rc) return rc;
    if (!xs || k < 16) return BQM_EINVAL;
    if (k % 16 != 0 || !aligned(xq, 4) || !aligned(xs, 4)) return BQM_EUNSUPPORTED;
    return launch_typed<kOutE4m3>(a, x_type, as_stream(stream));
}
