// Shared by the kernels of the MXFP4 products.
#pragma once

#include "values.h"

namespace bqm {

struct MgArgs {
    const uint8_t *w, *ws, *xq, *xs;
    float *y;
    int64_t ldy;          // floats between rows of y
    int m, k, n;
    int mtiles, ntiles;
};

// Widest aligned loads of scale rows of `nblk` bytes: 16, 4 or 1.
inline int scale_load(int nblk, const void *a, const void *b) {
    if (nblk % 16 == 0 && aligned(a, 16) && aligned(b, 16)) return 16;
    return nblk % 4 == 0 && aligned(a, 4) && aligned(b, 4) ? 4 : 1;
}

// The product for few tokens (mxfp4_stream.hip): the groups of 16 tokens at a
// time with which it takes a shape, 0 if the tiles (tile_cost us) should, and
// its launch (arguments already checked by the GEMM entry).
int mxfp4_stream_groups(int m, int k, int n, int cus, double tile_cost);
int mxfp4_stream(const MgArgs &a, int groups, hipStream_t s);

}  // namespace bqm
