// Shared by the kernels of the grouped MXFP4 product.
#pragma once

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

// The 16 scale bytes from block b0 on of the row of nblk bytes at p, at any
// alignment; zeros past its end.
__device__ __forceinline__ void scale_bytes(const uint8_t *p, int b0, int nblk, unsigned (&v)[4]) {
    if (nblk >= 16) {
        const int from = min(b0, nblk - 16), shift = b0 - from;   // uniform
        u32x4 u;
        __builtin_memcpy(&u, p + from, 16);
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = u[e];
        if (shift > 0) {
#pragma unroll
            for (int d = 2; d >= 1; d /= 2)
                if ((shift >> 2) & d) {
#pragma unroll
                    for (int q = 0; q < 4; q++) v[q] = q + d < 4 ? v[q + d] : 0;
                }
#pragma unroll
            for (int q = 0; q < 4; q++) v[q] = __builtin_amdgcn_alignbyte(q < 3 ? v[q + 1] : 0, v[q], shift & 3);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 4; q++) {
            v[q] = 0;
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (4 * q + e < nblk - b0) v[q] |= (unsigned)p[b0 + 4 * q + e] << (8 * e);
        }
    }
}

// The product of few slots a group (grouped_stream.hip): whether it takes a
// shape of about so many tiles of 128 x 128, and its launch.
bool grouped_stream_applies(const GgArgs &a, int64_t tiles, int cus);
int grouped_stream(const GgArgs &a, int cus, hipStream_t s);

}  // namespace bqm
