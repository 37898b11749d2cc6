// Root-mean-square norm with the residual's addition for gfx950, written as
// plain values or as the 8-bit operands of the projection matmuls.
//
//   s = x + res (f32),  h = s rounded to x's type,
//   y = s * (1 / sqrt(sum(s^2) / k + eps)) * gain,
// then q8_1 per 32 values or e4m3 per 128 values of the f32 y.
//
// HBM-bound: x and res are read once and h and y written once, so a row stays
// in registers between the sum of squares and the scaling.
//  * A row is cut into pieces of 16 bytes (four f32 or eight 16-bit values);
//    thread i of the row's NT owns pieces i, i + NT, ... (kNormPieces of them).
//    A wave has a row of up to 128 pieces to itself (no barrier); otherwise a
//    workgroup, as many whole waves as the row needs, has it (up to 2048
//    pieces); beyond that the workgroup reads the row twice, the second time
//    mostly from its L2.  Two pieces per thread, measured against one and four
//    at 8192 x 5120 bf16 -> e4m3 (56.9, 65.5, 65.7 us; 5.2 TB/s) and at
//    64 x 8192 (5.1, 4.6, 6.9 us): more waves on a row shorten its chain of
//    load, sum, barrier and store, fewer leave each enough loads in flight.
//  * The sum of squares is one fma chain per thread, a DPP tree over the wave,
//    then the waves' sums in order: f32, the order a function of k and the type
//    alone, so a token's norm is the same bits in decode and in prefill.
//  * The lanes of a 32- or 128-value block are neighbours in a row of 16 or 32
//    lanes, so the block maxima are DPP steps on values already in registers.
//  * The q8_1 rule rounds the correctly rounded quotient x / d.  Here the
//    product with an approximate reciprocal decides wherever it is further
//    from a half than its error, and only a wave that holds a value nearer
//    than that divides: the quants are the same, for a tenth of the divisions.
//  * ALN: rows aligned to a piece; otherwise the same pieces move in 16-byte
//    accesses at any alignment, the row's last one element by element, with
//    the same arithmetic, for odd k and odd strides: 8192 x 5121 f16 80 us (4.2
//    TB/s; 254 if every piece moves by elements) against 61 for 8192 x 5120.
//    Stores through the caches there: neighbouring rows share lines.
//  * Aligned rows are stored past the caches: each output is larger than they are
//    by the time it is read, where time counts.
#include "values.h"

namespace bqm {

enum { kOutF32, kOutSame, kOutQ81, kOutE4m3 };

constexpr int kNormPieces = 2;          // pieces per thread
constexpr int kNormMaxThreads = 1024;
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

// A piece of T: W values.
template <typename T>
struct Piece {
    static constexpr int W = 16 / sizeof(T);
    typedef float f __attribute__((ext_vector_type(W)));
};

template <typename T, int W, bool ALN>
__device__ __forceinline__ auto load_piece(const T *p, int i, int k) {
    typedef float f __attribute__((ext_vector_type(W)));
    typedef typename Packed<T, W, ALN ? 16 : sizeof(T)>::v tv;
    f v = {};
    if (i + W <= k) {
        v = __builtin_convertvector(*reinterpret_cast<const tv *>(p + i), f);
    } else if constexpr (!ALN) {
#pragma unroll
        for (int e = 0; e < W; e++)
            if (i + e < k) v[e] = (float)p[i + e];
    }
    return v;
}

template <typename T, int W, bool ALN, typename F>
__device__ __forceinline__ void store_piece(T *p, int i, int k, F v) {
    typedef T plain __attribute__((ext_vector_type(W)));
    typedef typename Packed<T, W, ALN ? 16 : sizeof(T)>::v tv;
    if (i + W <= k) {
        if constexpr (ALN)
            __builtin_nontemporal_store(__builtin_convertvector(v, plain), reinterpret_cast<tv *>(p + i));
        else
            *reinterpret_cast<tv *>(p + i) = __builtin_convertvector(v, plain);
    } else if constexpr (!ALN) {
#pragma unroll
        for (int e = 0; e < W; e++)
            if (i + e < k) p[i + e] = (T)v[e];
    }
}

__device__ __forceinline__ float clamp448n(float v) { return fminf(fmaxf(v, -448.0f), 448.0f); }

// Largest magnitude over groups of LANES neighbouring lanes, on every lane.
template <int LANES>
__device__ __forceinline__ float group_absmax(float v) {
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, false)));
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, false)));
    if constexpr (LANES >= 8)
        v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xF, 0xF, false)));
    if constexpr (LANES >= 16)
        v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xF, 0xF, false)));
    if constexpr (LANES >= 32) v = swap16_max(v);
    return v;
}

// One piece of y: values i .. i+W-1 of row t.  Every lane of the wave takes
// part (block maxima); lanes past k hold zeros and store nothing.
template <typename T, int OUT, bool ALN, typename F>
__device__ __forceinline__ void emit(const NormArgs &a, int64_t t, int i, F y) {
    constexpr int W = Piece<T>::W;
    typedef int words __attribute__((ext_vector_type(W / 4)));
    const int64_t at = t * a.k;
    if constexpr (OUT == kOutF32) {
        store_piece<float, W, ALN>(static_cast<float *>(a.y) + at, i, a.k, y);
        return;
    }
    if constexpr (OUT == kOutSame) {
        store_piece<T, W, ALN>(static_cast<T *>(a.y) + at, i, a.k, y);
        return;
    }
    // from the first value, not from zero: a block of NaN alone keeps it, as in
    // the quantizers (a NaN beside numbers is dropped)
    float big = fabsf(y[0]);
#pragma unroll
    for (int e = 1; e < W; e++) big = fmaxf(big, fabsf(y[e]));
    words q;
    if constexpr (OUT == kOutQ81) {
        big = group_absmax<32 / W>(big);
        const float d = big / 127.0f;
        const bool nz = d > 0.0f;
        const float inv = __builtin_amdgcn_rcpf(d);
        // |y * inv| is within 127 * 3 * 2^-24 < 2.4e-5 of the quotient, and the
        // correctly rounded one within 7.6e-6; a tiny d has no reciprocal
        bool near = !(d > 1e-30f) && nz;
        float r[W];
#pragma unroll
        for (int e = 0; e < W; e++) {
            const float v = fabsf(y[e] * inv);
            const float whole = floorf(v);
            near |= !(fabsf(v - whole - 0.5f) > 1e-4f) && nz;   // a NaN too
            r[e] = copysignf(fminf(floorf(v + 0.5f), 127.0f), y[e]);
        }
        if (__ballot(near) != 0) {
#pragma unroll
            for (int e = 0; e < W; e++) r[e] = (float)q8_1_quant1(y[e], d, nz);
        }
        int sum = 0;
#pragma unroll
        for (int w = 0; w < W / 4; w++) {
            unsigned b = 0;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int one = nz ? (int)r[4 * w + e] : 0;
                sum += one;
                b |= (unsigned)(one & 0xFF) << (8 * e);
            }
            q[w] = (int)b;
        }
        sum += __builtin_amdgcn_update_dpp(0, sum, 0xB1, 0xF, 0xF, false);
        sum += __builtin_amdgcn_update_dpp(0, sum, 0x4E, 0xF, 0xF, false);
        if constexpr (W == 4) sum += __builtin_amdgcn_update_dpp(0, sum, 0x141, 0xF, 0xF, false);
        if (i < a.k && (threadIdx.x & (32 / W - 1)) == 0)
            reinterpret_cast<float2 *>(a.scale)[(at + i) >> 5] = make_float2(d, d * (float)sum);
    } else {
        big = group_absmax<128 / W>(big);
        float mul = 0.0f, s = 0.0f;
        if (big > 0.0f) {
            mul = 448.0f / big;
            s = big / 448.0f;
        }
#pragma unroll
        for (int w = 0; w < W / 4; w++) {
            const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448n(y[4 * w] * mul), clamp448n(y[4 * w + 1] * mul), 0, false);
            q[w] = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448n(y[4 * w + 2] * mul), clamp448n(y[4 * w + 3] * mul), lo, true);
        }
        if (i < a.k && (threadIdx.x & (128 / W - 1)) == 0) a.scale[t * ((a.k + 127) >> 7) + (i >> 7)] = s;
    }
    // codes: k and so every piece's place is a multiple of W (k % 16 == 0)
    if (i < a.k) {
        int *const p = reinterpret_cast<int *>(static_cast<uint8_t *>(a.y) + at + i);
        if constexpr (ALN) {
            __builtin_nontemporal_store(q, reinterpret_cast<words *>(p));
        } else {
#pragma unroll
            for (int w = 0; w < W / 4; w++) p[w] = q[w];
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

template <int W, typename F>
__device__ __forceinline__ float squares(F v, float acc) {
#pragma unroll
    for (int e = 0; e < W; e++) acc = __builtin_fmaf(v[e], v[e], acc);
    return acc;
}

// WAVE: a wave per row; else a workgroup per row.  LONG: the row is longer
// than the registers hold and is read twice.
template <typename T, int OUT, bool ALN, bool WAVE, bool LONG>
__global__ __launch_bounds__(WAVE ? 256 : kNormMaxThreads) void norm_kernel(NormArgs a) {
    constexpr int W = Piece<T>::W;
    typedef typename Piece<T>::f F;
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
            F s[kNormPieces];
#pragma unroll
            for (int c = 0; c < kNormPieces; c++) s[c] = load_piece<T, W, ALN>(x, W * (lane + c * nt), a.k);
            if (res) {
                F r[kNormPieces];
#pragma unroll
                for (int c = 0; c < kNormPieces; c++) r[c] = load_piece<T, W, ALN>(res, W * (lane + c * nt), a.k);
#pragma unroll
                for (int c = 0; c < kNormPieces; c++) s[c] += r[c];
            }
            // f32: the gain is on its way during the sum (16-bit pieces have twice
            // the values, and the registers go to more rows in flight)
            F g[W == 4 ? kNormPieces : 1];
            auto load_gain = [&](int c) {
                F v = F(1.0f);
                if (a.gain) v = load_piece<float, W, ALN>(a.gain, W * (lane + c * nt), a.k);
                return v;
            };
            if constexpr (W == 4) {
#pragma unroll
                for (int c = 0; c < kNormPieces; c++) g[c] = load_gain(c);
            }
#pragma unroll
            for (int c = 0; c < kNormPieces; c++) acc = squares<W>(s[c], acc);
            if (res) {
#pragma unroll
                for (int c = 0; c < kNormPieces; c++) store_piece<T, W, ALN>(h, W * (lane + c * nt), a.k, s[c]);
            }
            const float inv = inv_rms(WAVE ? wave_sum(acc) : block_sum(acc, red[turn]), a.k, a.eps);
#pragma unroll
            for (int c = 0; c < kNormPieces; c++) {
                if (W * c * nt < a.k) {
                    if constexpr (W != 4) g[0] = load_gain(c);
                    emit<T, OUT, ALN>(a, t, W * (lane + c * nt), s[c] * inv * g[W == 4 ? c : 0]);
                }
            }
        } else {
            for (int i = W * lane; i - W * lane < a.k; i += W * nt) {
                F s = load_piece<T, W, ALN>(x, i, a.k);
                if (res) s += load_piece<T, W, ALN>(res, i, a.k);
                acc = squares<W>(s, acc);
            }
            const float inv = inv_rms(block_sum(acc, red[turn]), a.k, a.eps);
            // h may be x or res: each value is read and then written by one thread
            for (int i = W * lane; i - W * lane < a.k; i += W * nt) {
                F s = load_piece<T, W, ALN>(x, i, a.k);
                if (res) {
                    s += load_piece<T, W, ALN>(res, i, a.k);
                    store_piece<T, W, ALN>(h, i, a.k, s);
                }
                F g = F(1.0f);
                if (a.gain) g = load_piece<float, W, ALN>(a.gain, i, a.k);
                emit<T, OUT, ALN>(a, t, i, s * inv * g);
            }
        }
    }
}

template <typename T, int OUT, bool ALN>
static int launch_norm(const NormArgs &a, hipStream_t s) {
    constexpr int kWaveK = 64 * Piece<T>::W * kNormPieces;   // a wave's row at most
    const int64_t rows = a.m;
    if (a.k <= kWaveK) {
        const int64_t grid = (rows + 3) / 4;
        hipLaunchKernelGGL((norm_kernel<T, OUT, ALN, true, false>), dim3((unsigned)(grid < kNormMaxGrid ? grid : kNormMaxGrid)),
                           dim3(256), 0, s, a);
        return launch_status();
    }
    const unsigned grid = (unsigned)(rows < kNormMaxGrid ? rows : kNormMaxGrid);
    if (a.k <= kWaveK * (kNormMaxThreads / 64)) {
        const int nt = (a.k + kWaveK - 1) / kWaveK * 64;
        hipLaunchKernelGGL((norm_kernel<T, OUT, ALN, false, false>), dim3(grid), dim3(nt), 0, s, a);
    } else {
        hipLaunchKernelGGL((norm_kernel<T, OUT, ALN, false, true>), dim3(grid), dim3(kNormMaxThreads), 0, s, a);
    }
    return launch_status();
}

template <typename T, int OUT>
static int launch_aligned(const NormArgs &a, hipStream_t s) {
    constexpr int W = Piece<T>::W;
    const uintptr_t out = OUT == kOutF32 || OUT == kOutSame ? 16 : W;
    const bool rows = a.m == 1 || (a.ldx % W == 0 && (!a.res || (a.ldr % W == 0 && a.ldh % W == 0)));
    const bool aln = a.k % W == 0 && rows && aligned(a.x, 16) && aligned(a.res, 16) && aligned(a.h, 16) &&
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
