// MXFP4 decode / verify product for gfx950: weights of 4 bits with a power of
// two per 32, f32 activations, m = 1..16.
//
//   y[t][r] = sum_b 2^(ws[r][b] - 127) * sum_{i in b} x[t][i] * e2m1(w[r][i])
//
// HBM-bound: 17/32 byte per weight, read once.  At two weights a byte the
// VALU could not keep up with a few tokens (a conversion and one fma per
// weight and token), so the bf16 matrix cores do it at every m:
//  * An f32 is the sum of three bf16 numbers exactly (its significand cut
//    into three bytes), and a scaled e2m1 value is a bf16 exactly, so the
//    products are exact and only the f32 accumulation rounds.
//  * The three parts of a token are three rows of the 16-row operand, so five
//    tokens make one MFMA per 16 weight rows x 32 k (G = 1), ten two, sixteen
//    three.  Rows do not mix: a token's result is the same bits at every m.
//  * A wave owns 512 k (16 scale blocks) and keeps its x operands for them in
//    registers (64 VGPRs per 16 operand rows); the workgroup's waves cover up
//    to 4096 k and the k beyond them in further passes, which add to y.
//  * Weight rows stream through registers into a wave's own LDS tile (16 rows
//    x 256 bytes, loaded 256 contiguous bytes per row, two tiles ahead), from
//    which a lane reads the 16-byte block of its row: lane group g holds
//    blocks 4g .. 4g+3 of the 512 k, so that its four scales are one dword.
//    The order of k inside a step is the same for x, and free.
//  * The waves' partial tiles meet in LDS, added in wave order.
#include "values.h"

namespace bqm {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kMvRows = 16;           // weight rows of a tile
constexpr int kMvSlice = 512;         // k of a wave
constexpr int kMvBlocks = kMvSlice / 32;
constexpr int kMvMaxWaves = 8;
constexpr int kMvRowStride = kMvSlice / 2 + 16;           // LDS row of a weight tile
constexpr int kMvXStride = kMvSlice * 2 + 16;             // LDS row of the x operand
constexpr int kMvTileBytes = kMvRows * kMvRowStride;

struct MvArgs {
    const uint8_t *w, *ws;
    const float *x;
    float *y;
    int m, k, n;
    int parts;     // waves along k
    int groups;    // row tiles of a workgroup at a time
    int passes;    // rounds over k
};

struct MvTile {
    u32x4 c[4];
    unsigned s;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_rsrc(const void *base, int64_t bytes) {
    const uint32_t b = bytes <= 0 ? 0u : bytes > 0x7FFFFFF0ll ? 0x7FFFFFF0u : (uint32_t)bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)b, 0x00020000);
}

// Two codes of byte `sel` of q, scaled, as bf16.
template <int SEL>
__device__ __forceinline__ v2bf two(unsigned q, float s) { return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, SEL); }

__device__ __forceinline__ v8bf eight(unsigned q, float s) {
    const v2bf a = two<0>(q, s), b = two<1>(q, s), c = two<2>(q, s), d = two<3>(q, s);
    return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The three bf16 parts of eight f32 values, by cutting: each part is the
// upper half of what the earlier ones left, and the last is what remains.
__device__ __forceinline__ void three_parts(const float *v, u32x4 (&p)[3]) {
    unsigned h[3][8];
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const float a = v[e];
        const float b = a - __builtin_bit_cast(float, __builtin_bit_cast(unsigned, a) & 0xFFFF0000u);
        const float c = b - __builtin_bit_cast(float, __builtin_bit_cast(unsigned, b) & 0xFFFF0000u);
        h[0][e] = __builtin_bit_cast(unsigned, a);
        h[1][e] = __builtin_bit_cast(unsigned, b);
        h[2][e] = __builtin_bit_cast(unsigned, c);
    }
#pragma unroll
    for (int i = 0; i < 3; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) p[i][e] = (h[i][2 * e] >> 16) | (h[i][2 * e + 1] & 0xFFFF0000u);
}

// WIDE: scale rows are whole, aligned dwords (k % 128 == 0); else bytes.
template <int G, bool WIDE>
__global__ __launch_bounds__(kMvMaxWaves * 64, G == 1 ? (WIDE ? 4 : 3) : 2) void mxfp4_gemv_kernel(MvArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = wave % a.parts, group = wave / a.parts;
    const int waves = a.parts * a.groups;
    const int r16 = lane & 15, g4 = lane >> 4;
    const int nblk = a.k / 32;               // scale blocks of a row
    const int64_t row_bytes = a.k / 2;
    const int tiles = (a.n + kMvRows - 1) / kMvRows;
    const int stride = gridDim.x * a.groups;
    const int rounds = (tiles + stride - 1) / stride;

    // LDS: first each wave's x operand, then (the same memory) each wave's
    // weight tile and, behind the tiles, two sets of partial results
    uint8_t *const tile = lds + wave * kMvTileBytes;
    float *const red = reinterpret_cast<float *>(lds + waves * kMvTileBytes);
    constexpr int kRed = G * 256;   // floats of a wave's partial result

    for (int pass = 0; pass < a.passes; pass++) {
        const int blk0 = (pass * a.parts + part) * kMvBlocks;   // first scale block of this wave's k

        auto load = [&](MvTile &t, int round) {
            const int64_t row0 = ((int64_t)round * stride + blockIdx.x * a.groups + group) * kMvRows;
            const int64_t rows = a.n - row0 < kMvRows ? a.n - row0 : kMvRows;   // may be <= 0: nothing is read
            const __amdgpu_buffer_rsrc_t rw = mx_rsrc(a.w + row0 * row_bytes, rows * row_bytes);
            const __amdgpu_buffer_rsrc_t rs = mx_rsrc(a.ws + row0 * nblk, rows * nblk);
            // blocks past the row's end are read as zeros
            const uint32_t off = blk0 + r16 < nblk ? (uint32_t)(g4 * row_bytes + 16 * (blk0 + r16)) : 0x80000000u;
#pragma unroll
            for (int i = 0; i < 4; i++)
                t.c[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, off + (uint32_t)(4 * i * row_bytes), 0, 0));
            const int b = blk0 + 4 * g4;
            if constexpr (WIDE) {
                t.s = __builtin_amdgcn_raw_buffer_load_b32(rs, b < nblk ? (uint32_t)(r16 * nblk + b) : 0x80000000u, 0, 0);
            } else {
                t.s = 0;
#pragma unroll
                for (int q = 0; q < 4; q++)
                    t.s |= (unsigned)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                               rs, b + q < nblk ? (uint32_t)(r16 * nblk + b + q) : 0x80000000u, 0, 0) << (8 * q);
            }
        };

        MvTile t0, t1;
        load(t0, 0);
        load(t1, 1);

        // x operands: a token's 512 values are eight per lane, its three parts
        // three rows; a lane then takes row 16 * grp + r16 of the operand
        v8bf xop[G][16];
        {
            uint8_t *const xs = lds + wave * (16 * kMvXStride);
#pragma unroll
            for (int grp = 0; grp < G; grp++) {
                const int k0 = 32 * blk0 + 8 * lane;
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                for (int tok = (16 * grp) / 3; tok < a.m && 3 * tok < 16 * grp + 16; tok++) {
                    float v[8];
                    const bool in = k0 < a.k;   // k % 32 == 0: eight values are in or out together
                    const float4 lo = in ? *reinterpret_cast<const float4 *>(a.x + (int64_t)tok * a.k + k0) : make_float4(0, 0, 0, 0);
                    const float4 hi = in ? *reinterpret_cast<const float4 *>(a.x + (int64_t)tok * a.k + k0 + 4) : make_float4(0, 0, 0, 0);
                    v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
                    v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
                    u32x4 p[3];
                    three_parts(v, p);
#pragma unroll
                    for (int i = 0; i < 3; i++) {
                        const int row = 3 * tok + i - 16 * grp;
                        if (row >= 0 && row < 16) *reinterpret_cast<u32x4 *>(xs + row * kMvXStride + 16 * lane) = p[i];
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                const bool used = 16 * grp + r16 < 3 * a.m;
#pragma unroll
                for (int st = 0; st < 16; st++) {
                    // step 4q + d: values 8d .. 8d+7 of block 4 * g4 + q
                    const int at = (4 * g4 + (st >> 2)) * 64 + (st & 3) * 16;
                    u32x4 q = {0, 0, 0, 0};
                    if (used) q = *reinterpret_cast<const u32x4 *>(xs + r16 * kMvXStride + at);
                    xop[grp][st] = __builtin_bit_cast(v8bf, q);
                }
            }
        }
        __syncthreads();   // the x operands' LDS becomes the weight tiles'

        auto compute = [&](const MvTile &t, int round) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                *reinterpret_cast<u32x4 *>(tile + (4 * i + g4) * kMvRowStride + 16 * r16) = t.c[i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            v4f acc[G];
#pragma unroll
            for (int grp = 0; grp < G; grp++) acc[grp] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const u32x4 c = *reinterpret_cast<const u32x4 *>(tile + r16 * kMvRowStride + (4 * g4 + q) * 16);
                const float s = __builtin_bit_cast(float, ((t.s >> (8 * q)) & 255u) << 23);
#pragma unroll
                for (int d = 0; d < 4; d++) {
                    const v8bf b = eight(c[d], s);
#pragma unroll
                    for (int grp = 0; grp < G; grp++)
                        acc[grp] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xop[grp][4 * q + d], b, acc[grp], 0, 0, 0);
                }
            }
            // lane: weight row r16, operand rows 4 * g4 + v of each group
            float *const mine = red + ((round & 1) * waves + wave) * kRed;
#pragma unroll
            for (int grp = 0; grp < G; grp++)
#pragma unroll
                for (int v = 0; v < 4; v++) mine[(16 * grp + 4 * g4 + v) * 16 + r16] = acc[grp][v];
            __syncthreads();
            const int64_t row0 = ((int64_t)round * stride + blockIdx.x * a.groups + group) * kMvRows;
            const float *const set = red + ((round & 1) * waves + group * a.parts) * kRed;
            for (int o = part * 64 + lane; o < 16 * a.m; o += 64 * a.parts) {
                const int tok = o >> 4, col = o & 15;
                float v = 0.0f;
                for (int p = 0; p < a.parts; p++) {
                    const float *q = set + p * kRed + 48 * tok + col;
                    v += (q[32] + q[16]) + q[0];   // the smallest part first
                }
                if (row0 + col < a.n) {
                    float *const y = a.y + (int64_t)tok * a.n + row0 + col;
                    *y = pass == 0 ? v : *y + v;
                }
            }
        };
        for (int round = 0; round < rounds; round += 2) {
            compute(t0, round);
            load(t0, round + 2);
            if (round + 1 < rounds) {
                compute(t1, round + 1);
                load(t1, round + 3);
            }
        }
        __syncthreads();   // the tiles' LDS becomes the next pass's x operands'
    }
}

template <int G, bool WIDE>
static int launch_mv(MvArgs a, hipStream_t s) {
    static LaunchCache cache;
    const void *fn = reinterpret_cast<const void *>(&mxfp4_gemv_kernel<G, WIDE>);
    const int waves = a.parts * a.groups;
    const int stream_bytes = waves * (kMvTileBytes + 2 * G * 1024);
    const int x_bytes = waves * 16 * kMvXStride;
    const int bytes = stream_bytes > x_bytes ? stream_bytes : x_bytes;
    const int rc = raise_lds_limit(cache, fn, 160 * 1024);
    if (rc) return rc;
    const int tiles = (a.n + kMvRows - 1) / kMvRows;
    const int units = (tiles + a.groups - 1) / a.groups;
    const int most = device_cus() * blocks_per_cu(cache, fn, waves * 64, bytes, 4);
    const int rounds = (units + most - 1) / most;
    const int grid = (units + rounds - 1) / rounds;
    hipLaunchKernelGGL((mxfp4_gemv_kernel<G, WIDE>), dim3(grid), dim3(waves * 64), bytes, s, a);
    return launch_status();
}

template <int G>
static int launch_mv_scales(const MvArgs &a, hipStream_t s) {
    return a.k % 128 == 0 && aligned(a.ws, 4) ? launch_mv<G, true>(a, s) : launch_mv<G, false>(a, s);
}

}  // namespace bqm

extern "C" int bqm_mxfp4_gemv(const uint8_t *w, const uint8_t *ws, const float *x, float *y, int m, int k, int n,
                              void *stream) {
    using namespace bqm;
    if (!w || !ws || !x || !y) return BQM_EINVAL;
    if (m < 1 || m > BQM_MXFP4_GEMV_MAX_M || k < 32 || n < 1) return BQM_EINVAL;
    if (k % 32 != 0 || !aligned(w, 16) || !aligned(x, 16) || !aligned(y, 4)) return BQM_EUNSUPPORTED;
    if (k > 1 << 27) return BQM_EUNSUPPORTED;   // 16 rows in 31 bits
    MvArgs a = {w, ws, x, y, m, k, n, 0, 0, 0};
    const int slices = (k + kMvSlice - 1) / kMvSlice;
    a.passes = (slices + kMvMaxWaves - 1) / kMvMaxWaves;
    a.parts = (slices + a.passes - 1) / a.passes;
    a.groups = kMvMaxWaves / a.parts;
    hipStream_t s = as_stream(stream);
    if (m <= 5) return launch_mv_scales<1>(a, s);
    if (m <= 10) return launch_mv_scales<2>(a, s);
    return launch_mv_scales<3>(a, s);
}
