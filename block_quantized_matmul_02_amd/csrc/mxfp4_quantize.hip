// MXFP4 quantization and dequantization for gfx950 (OCP Microscaling Formats
// v1.0: e2m1 values, one E8M0 scale per 32).
//
// The scale is a power of two taken from the exponent field of the block's
// largest magnitude, so dividing by it is one exact multiplication and only
// the conversion to e2m1 rounds (v_cvt_scalef32_pk_fp4_f32 with scale 1, to
// nearest even; values are clamped to +-6 first).
//
// HBM-bound both ways.  A lane holds eight values and four neighbouring lanes
// a block: the block maximum is two DPP steps, an item is one or two 16-byte
// accesses on the wide side and one dword of codes, and a wave's accesses are
// contiguous: 5.6 TB/s for 5120 x 17408 bf16 (40 us, 225 MB).  The dequantized
// values, four to eight times the codes, are stored past the caches (33 us
// against 46).  The maximum is taken over the magnitudes' bit patterns as
// whole numbers, which order infinities and NaN above every finite value.
#include "values.h"

namespace bqm {

constexpr int kMxThreads = 256;

struct MxShape {
    int64_t items;   // eight values each
    int64_t ld;      // elements between rows of x
    unsigned per_row;   // items in a row
    int dense;       // rows of x follow each other
};

template <typename T>
__device__ __forceinline__ v8f load8(const T *p) {
    return __builtin_convertvector(*reinterpret_cast<const typename Packed<T, 8, 16>::v *>(p), v8f);
}

template <typename T>
__global__ __launch_bounds__(kMxThreads) void mxfp4_quantize_kernel(const T *__restrict__ x,
                                                                  unsigned *__restrict__ codes,
                                                                  uint8_t *__restrict__ scales, MxShape g) {
    const int64_t item = (int64_t)blockIdx.x * kMxThreads + threadIdx.x;
    // items are a multiple of four, so a block's four lanes are all inside or all outside
    if (item >= g.items) return;
    int64_t at = item * 8;
    if (!g.dense) {
        const int64_t row = item / g.per_row;
        at = row * g.ld + (item - row * g.per_row) * 8;
    }
    const v8f v = load8(x + at);
    unsigned big = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const float one = v[e];   // a bit cast of a vector element would read the first element
        big = max(big, __builtin_bit_cast(unsigned, one) & 0x7FFFFFFFu);
    }
    big = max(big, (unsigned)__builtin_amdgcn_update_dpp(0, (int)big, 0xB1, 0xF, 0xF, false));
    big = max(big, (unsigned)__builtin_amdgcn_update_dpp(0, (int)big, 0x4E, 0xF, 0xF, false));
    const int field = (int)(big >> 23);   // exponent field: 0 for zero and subnormals, 255 for inf and NaN
    const int s = field == 255 ? 255 : max(field - 2, 0);
    // 2^(127 - s): s is at most 252 here, so the factor is a normal number
    const float mul = __builtin_bit_cast(float, (unsigned)(254 - s) << 23);
    unsigned q = 0;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float a = fminf(fmaxf(v[2 * e] * mul, -6.0f), 6.0f);
        const float b = fminf(fmaxf(v[2 * e + 1] * mul, -6.0f), 6.0f);
        switch (e) {   // the byte of the result is part of the instruction
            case 0: q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a, b, 1.0f, 0); break;
            case 1: q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a, b, 1.0f, 1); break;
            case 2: q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a, b, 1.0f, 2); break;
            default: q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a, b, 1.0f, 3); break;
        }
    }
    codes[item] = field == 255 ? 0u : q;
    if ((item & 3) == 0) scales[item >> 2] = (uint8_t)s;
}

// An E8M0 byte as f32: 2^(s - 127); 255 is NaN, 0 is the subnormal 2^-127.
__device__ __forceinline__ float e8m0_to_float(unsigned s) {
    return __builtin_bit_cast(float, s == 255 ? 0x7FC00000u : s == 0 ? 0x00400000u : s << 23);
}

template <typename T>
__global__ __launch_bounds__(kMxThreads) void mxfp4_dequantize_kernel(const unsigned *__restrict__ codes,
                                                                    const uint8_t *__restrict__ scales,
                                                                    T *__restrict__ y, int64_t items) {
    const int64_t item = (int64_t)blockIdx.x * kMxThreads + threadIdx.x;
    if (item >= items) return;
    const unsigned q = codes[item];
    const float s = e8m0_to_float(scales[item >> 2]);
    v8f v;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const auto p = e == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0)
                       : e == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1)
                       : e == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2)
                                : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
        v[2 * e] = p[0] * s;
        v[2 * e + 1] = p[1] * s;
    }
    typedef T plain __attribute__((ext_vector_type(8)));
    __builtin_nontemporal_store(__builtin_convertvector(v, plain), reinterpret_cast<typename Packed<T, 8, 16>::v *>(y + item * 8));
}

static bool mx_grid(int64_t items, unsigned *grid) {
    const int64_t b = (items + kMxThreads - 1) / kMxThreads;
    // the dispatch counts work items in 32 bits
    if (b * kMxThreads > 0xFFFFFFFFll) return false;
    *grid = (unsigned)b;
    return true;
}

}  // namespace bqm

extern "C" int bqm_mxfp4_quantize(const void *x, int64_t ldx, uint8_t *codes, uint8_t *scales, int x_type, int m,
                                  int k, void *stream) {
    using namespace bqm;
    if (!x || !codes || !scales) return BQM_EINVAL;
    if (m < 1 || k < 32 || !type_known(x_type)) return BQM_EINVAL;
    if (k % 32 != 0 || !aligned(x, 16) || !aligned(codes, 4)) return BQM_EUNSUPPORTED;
    if (m > 1 && (ldx < k || ldx * type_bytes(x_type) % 16 != 0)) return BQM_EUNSUPPORTED;
    const MxShape g = {(int64_t)m * k / 8, ldx, (unsigned)(k / 8), m == 1 || ldx == k};
    unsigned grid;
    if (!mx_grid(g.items, &grid)) return BQM_EUNSUPPORTED;
    hipStream_t s = as_stream(stream);
    unsigned *c = reinterpret_cast<unsigned *>(codes);
    if (x_type == BQM_F32)
        hipLaunchKernelGGL(mxfp4_quantize_kernel<float>, dim3(grid), dim3(kMxThreads), 0, s, static_cast<const float *>(x), c, scales, g);
    else if (x_type == BQM_F16)
        hipLaunchKernelGGL(mxfp4_quantize_kernel<_Float16>, dim3(grid), dim3(kMxThreads), 0, s, static_cast<const _Float16 *>(x), c, scales, g);
    else
        hipLaunchKernelGGL(mxfp4_quantize_kernel<__bf16>, dim3(grid), dim3(kMxThreads), 0, s, static_cast<const __bf16 *>(x), c, scales, g);
    return launch_status();
}

extern "C" int bqm_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, void *y, int y_type, int m, int k,
                                    void *stream) {
    using namespace bqm;
    if (!codes || !scales || !y) return BQM_EINVAL;
    if (m < 1 || k < 32 || !type_known(y_type)) return BQM_EINVAL;
    if (k % 32 != 0 || !aligned(codes, 4) || !aligned(y, 16)) return BQM_EUNSUPPORTED;
    const int64_t items = (int64_t)m * k / 8;
    unsigned grid;
    if (!mx_grid(items, &grid)) return BQM_EUNSUPPORTED;
    hipStream_t s = as_stream(stream);
    const unsigned *c = reinterpret_cast<const unsigned *>(codes);
    if (y_type == BQM_F32)
        hipLaunchKernelGGL(mxfp4_dequantize_kernel<float>, dim3(grid), dim3(kMxThreads), 0, s, c, scales, static_cast<float *>(y), items);
    else if (y_type == BQM_F16)
        hipLaunchKernelGGL(mxfp4_dequantize_kernel<_Float16>, dim3(grid), dim3(kMxThreads), 0, s, c, scales, static_cast<_Float16 *>(y), items);
    else
        hipLaunchKernelGGL(mxfp4_dequantize_kernel<__bf16>, dim3(grid), dim3(kMxThreads), 0, s, c, scales, static_cast<__bf16 *>(y), items);
    return launch_status();
}
