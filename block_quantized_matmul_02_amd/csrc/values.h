// Typed loads and stores of the kernels that take f32, fp16 or bf16 values.
#pragma once

#include "bqmm_internal.h"
#include "bqmm_layer.h"

namespace bqm {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v8f __attribute__((ext_vector_type(8)));

// W values of T at an address aligned to A bytes; the vector's own alignment,
// its whole size, may be more than the 16 bytes that pointers are checked for.
template <typename T, int W, int A>
struct Packed {
    typedef T v __attribute__((ext_vector_type(W), aligned(A)));
};

// A buffer whose reads past `bytes` give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_rsrc(const void *base, int64_t bytes) {
    const uint32_t b = bytes <= 0 ? 0u : bytes > 0x7FFFFFF0ll ? 0x7FFFFFF0u : (uint32_t)bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)b, 0x00020000);
}

inline int type_bytes(int type) { return type == BQM_F32 ? 4 : 2; }
inline bool type_known(int type) { return type == BQM_F32 || type == BQM_F16 || type == BQM_BF16; }

// Largest magnitude over a row of 16 lanes, on every lane (magnitudes only:
// a NaN operand is dropped).
__device__ __forceinline__ float dpp_absmax16(float v) {
    v = q8_1_max8(v);
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xF, 0xF, false)));
}

// Sum over the wave, on every lane.
__device__ __forceinline__ float wave_sum(float v) { return swap32_sum(swap16_sum(dpp_sum16(v))); }

}  // namespace bqm
