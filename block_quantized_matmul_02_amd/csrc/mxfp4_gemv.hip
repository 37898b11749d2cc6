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
//    three (the last in the rows that five of a group leave).  Rows do not mix: a token's result is the same bits at every m.
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
__device__ __forceinline__ void three_parts(const u32x4 (&v)[2], u32x4 (&p)[3]) {
    unsigned h[3][8];
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const unsigned u = v[e >> 2][e & 3];
        const float a = __builtin_bit_cast(float, u);
        const float b = a - __builtin_bit_cast(float, u & 0xFFFF0000u);
        const float c = b - __builtin_bit_cast(float, __builtin_bit_cast(unsigned, b) & 0xFFFF0000u);
        h[0][e] = u;
        h[1][e] = __builtin_bit_cast(unsigned, b);
        h[2][e] = __builtin_bit_cast(unsigned, c);
    }
#pragma unroll
    for (int i = 0; i < 3; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) p[i][e] = (h[i][2 * e] >> 16) | (h[i][2 * e + 1] & 0xFFFF0000u);
}

// Operand row of part h of the group's token i: tokens 0..3 have rows 4i + h,
// which are values 0..2 of one lane's result, and token 4 rows 4h + 3.  The
// sixteenth token has row 15 of the three groups.
__device__ __forceinline__ int operand_row(int i, int h) { return i < 4 ? 4 * i + h : 4 * h + 3; }

// A token's sum from the lanes' results of a wave's tile (r: column 0's lane
// plus the column): its three parts, the smallest first.
__device__ __forceinline__ float token_sum(const float2 *r, int tok) {
    if (tok == 15) return (r[128 + 48].y + r[64 + 48].y) + r[48].y;
    r += (tok / 5) * 64;
    const int i = tok % 5;
    return i < 4 ? r[16 * i].x : (r[32].y + r[16].y) + r[0].y;
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
    // weight tile and, behind the tiles, two sets of two tiles' partial results
    uint8_t *const tile = lds + wave * kMvTileBytes;
    float2 *const red = reinterpret_cast<float2 *>(lds + waves * kMvTileBytes);
    constexpr int kRed = G * 64;   // of a wave's tile: per group and lane (its token's sum, token 4's part)

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

        // x operands: a token's 512 values are eight per lane, its three parts
        // three rows; a lane then takes row r16 of each group's operand.  The
        // first group's values are asked for before the first weights.
        MvTile t0, t1;
        v8bf xop[G][16];
        {
            uint8_t *const xs = lds + wave * (16 * kMvXStride);
            const __amdgpu_buffer_rsrc_t rx = mx_rsrc(a.x, 4ll * a.m * a.k);
            // k % 32 == 0: a lane's eight values are in or out of the row together
            const uint32_t off = 32 * blk0 + 8 * lane < a.k ? (uint32_t)(4 * (32 * blk0 + 8 * lane)) : 0x80000000u;
#pragma unroll
            for (int grp = 0; grp < G; grp++) {
                // the group's five tokens and, of three groups, the sixteenth
                constexpr int kTok = G == 3 ? 6 : 5;
                u32x4 raw[kTok][2];
#pragma unroll
                for (int i = 0; i < kTok; i++) {
                    // tokens past the last read zeros
                    const uint32_t at = off + (uint32_t)(4 * a.k) * (i < 5 ? 5 * grp + i : 15);
                    raw[i][0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, at, 0, 0));
                    raw[i][1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, at + 16, 0, 0));
                }
                if (grp == 0) {
                    load(t0, 0);
                    load(t1, 1);
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                for (int i = 0; i < kTok; i++) {
                    if ((i < 5 ? 5 * grp + i : 15) >= a.m) continue;
                    u32x4 p[3];
                    three_parts(raw[i], p);
                    if (i == 5) {
                        *reinterpret_cast<u32x4 *>(xs + 15 * kMvXStride + 16 * lane) = p[grp];
                        continue;
                    }
#pragma unroll
                    for (int h = 0; h < 3; h++)
                        *reinterpret_cast<u32x4 *>(xs + operand_row(i, h) * kMvXStride + 16 * lane) = p[h];
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                const bool used = (r16 == 15 ? 15 : 5 * grp + ((r16 & 3) < 3 ? r16 >> 2 : 4)) < a.m;
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

        auto multiply = [&](const MvTile &t, float2 *out) {
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
            // lane: weight row r16, operand rows 4 * g4 + v; the smallest part first
#pragma unroll
            for (int grp = 0; grp < G; grp++)
                out[grp * 64 + lane] = make_float2((acc[grp][2] + acc[grp][1]) + acc[grp][0], acc[grp][3]);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        };
        // Two tiles to a barrier, and always two, so that the loads in flight
        // are the same number on every path; a tile past the last reads nothing
        // and stores nothing.
#pragma unroll 1
        for (int round = 0; round < rounds; round += 2) {
            float2 *const set = red + (round & 2) * waves * kRed;   // [2 tiles][waves][kRed], alternating
            // output o: tile o / (16 m), token, column; a later pass adds to y
            // (with more than one pass there are at least five waves along k,
            // and a thread has at most two outputs)
            auto where = [&](int o, int &tok, int &col, int64_t &at) {
                const int second = o >= 16 * a.m;
                col = o & 15;
                tok = (o >> 4) - (second ? a.m : 0);
                const int64_t row = ((int64_t)(round + second) * stride + blockIdx.x * a.groups + group) * kMvRows + col;
                at = (int64_t)tok * a.n + row;
                return row < a.n;
            };
            float old[2] = {0.0f, 0.0f};
            if (pass > 0) {
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    int tok, col;
                    int64_t at;
                    const int o = part * 64 + lane + i * 64 * a.parts;
                    if (o < 32 * a.m && where(o, tok, col, at)) old[i] = a.y[at];
                }
            }
            multiply(t0, set + wave * kRed);
            load(t0, round + 2);
            multiply(t1, set + (waves + wave) * kRed);
            load(t1, round + 3);
            __syncthreads();
            for (int o = part * 64 + lane, i = 0; o < 32 * a.m; o += 64 * a.parts, i++) {
                int tok, col;
                int64_t at;
                if (!where(o, tok, col, at)) continue;
                const float2 *const q = set + ((o >= 16 * a.m ? waves : 0) + group * a.parts) * kRed + col;
                float v[kMvMaxWaves];
#pragma unroll
                for (int p = 0; p < kMvMaxWaves; p++) {
                    const float2 *const r = q + (p < a.parts ? p : 0) * kRed;
                    const float one = token_sum(r, tok);
                    v[p] = p < a.parts ? one : 0.0f;
                }
                float sum = v[0];
#pragma unroll
                for (int p = 1; p < kMvMaxWaves; p++) sum += v[p];
                a.y[at] = pass > 0 ? (i == 0 ? old[0] : old[1]) + sum : sum;
            }
        }
        __syncthreads();   // the tiles' LDS becomes the next pass's x operands'
    }
}

// Up to five tokens whose operand fits in LDS.  The whole workgroup cuts x once
// into [3 m rows][k] bf16 and each step's operand is read from there (a few
// lanes' worth), so a wave goes through any number of 512-k slices: items
// (tile, slice) in order, kMvAhead of them loaded ahead, each slice's result
// kept apart in LDS so that they are added in the same order as the passes
// above add them, whatever k is.
constexpr int kMvAhead = 4;

struct MvDecode {
    MvArgs a;
    int slices;     // 512-k slices of a row
    int per_wave;   // slices of a wave: ceil(slices / 8)
    int batch;      // tiles between barriers
    int two_sets;   // results have two sets in LDS; else a second barrier
};

template <bool WIDE>
__global__ __launch_bounds__(kMvMaxWaves * 64, WIDE ? 4 : 2) void mxfp4_decode_kernel(MvDecode d) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const MvArgs &a = d.a;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int nblk = a.k / 32;
    const int64_t row_bytes = a.k / 2;
    const int tiles = (a.n + kMvRows - 1) / kMvRows;
    const int xstride = d.slices * kMvSlice * 2 + 16;

    uint8_t *const xs = lds;
    uint8_t *const tile = lds + 3 * a.m * xstride + wave * kMvTileBytes;
    float2 *const red = reinterpret_cast<float2 *>(lds + 3 * a.m * xstride + kMvMaxWaves * kMvTileBytes);
    const int set_size = d.batch * d.slices * 64;

    // item j of this wave: tile (j / per_wave) of this workgroup's, slice wave + 8 (j % per_wave)
    int next_tile = blockIdx.x, next_s = 0;
    MvTile t[kMvAhead];
    auto load = [&](MvTile &q) {
        const int64_t row0 = (int64_t)next_tile * kMvRows;
        const int64_t rows = a.n - row0 < kMvRows ? a.n - row0 : kMvRows;   // may be <= 0: nothing is read
        const int blk0 = (wave + kMvMaxWaves * next_s) * kMvBlocks;
        const __amdgpu_buffer_rsrc_t rw = mx_rsrc(a.w + row0 * row_bytes, rows * row_bytes);
        const __amdgpu_buffer_rsrc_t rs = mx_rsrc(a.ws + row0 * nblk, rows * nblk);
        const uint32_t off = blk0 + r16 < nblk ? (uint32_t)(g4 * row_bytes + 16 * (blk0 + r16)) : 0x80000000u;
#pragma unroll
        for (int i = 0; i < 4; i++)
            q.c[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, off + (uint32_t)(4 * i * row_bytes), 0, 0));
        const int b = blk0 + 4 * g4;
        if constexpr (WIDE) {
            q.s = __builtin_amdgcn_raw_buffer_load_b32(rs, b < nblk ? (uint32_t)(r16 * nblk + b) : 0x80000000u, 0, 0);
        } else {
            q.s = 0;
#pragma unroll
            for (int e = 0; e < 4; e++)
                q.s |= (unsigned)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                           rs, b + e < nblk ? (uint32_t)(r16 * nblk + b + e) : 0x80000000u, 0, 0) << (8 * e);
        }
        if (++next_s == d.per_wave) {
            next_s = 0;
            next_tile += gridDim.x;
        }
    };

    // x: eight values a thread and turn; zeros up to a whole slice
    const int per_row = d.slices * 64;
    const __amdgpu_buffer_rsrc_t rx = mx_rsrc(a.x, 4ll * a.m * a.k);
    auto load_x = [&](int i, u32x4 (&v)[2], int &tok, int &at) {
        tok = i / per_row;
        at = i - tok * per_row;
        const uint32_t off = 8 * at < a.k ? (uint32_t)(4 * (tok * a.k + 8 * at)) : 0x80000000u;
        v[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, off, 0, 0));
        v[1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, off + 16, 0, 0));
    };
    {
        u32x4 v[2];
        int tok, at;
        load_x(threadIdx.x, v, tok, at);
#pragma unroll
        for (int i = 0; i < kMvAhead; i++) load(t[i]);
        for (int i = threadIdx.x;;) {
            u32x4 p[3];
            three_parts(v, p);
            if (i < a.m * per_row) {
#pragma unroll
                for (int h = 0; h < 3; h++) *reinterpret_cast<u32x4 *>(xs + (3 * tok + h) * xstride + 16 * at) = p[h];
            }
            i += kMvMaxWaves * 64;
            if (i - (int)threadIdx.x >= a.m * per_row) break;
            load_x(i, v, tok, at);
        }
    }
    __syncthreads();

    // this lane's operand row: rows 4i + h and 4h + 3 of the sixteen, as above
    const int tok = (r16 & 3) < 3 ? r16 >> 2 : 4, part = (r16 & 3) < 3 ? r16 & 3 : r16 >> 2;
    const bool used = tok < a.m && r16 != 15;
    const uint8_t *const xrow = xs + (used ? 3 * tok + part : 0) * xstride + 4 * g4 * 64;

    int s = 0, b = 0, first = blockIdx.x, set = 0;   // slice turn, tile of the batch, the batch's first tile
    const int mine = (tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x * d.per_wave;
    auto item = [&](MvTile &q, int j) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            *reinterpret_cast<u32x4 *>(tile + (4 * i + g4) * kMvRowStride + 16 * r16) = q.c[i];
        const unsigned sc = q.s;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        load(q);
        const int slice = wave + kMvMaxWaves * s;
        const uint8_t *const xp = xrow + (slice < d.slices ? slice : 0) * (kMvSlice * 2);
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int qq = 0; qq < 4; qq++) {
            const u32x4 c = *reinterpret_cast<const u32x4 *>(tile + r16 * kMvRowStride + (4 * g4 + qq) * 16);
            const float f = __builtin_bit_cast(float, ((sc >> (8 * qq)) & 255u) << 23);
            u32x4 xv[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                xv[e] = u32x4{0, 0, 0, 0};
                if (used) xv[e] = *reinterpret_cast<const u32x4 *>(xp + qq * 64 + e * 16);
            }
#pragma unroll
            for (int e = 0; e < 4; e++)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, xv[e]), eight(c[e], f), acc, 0, 0, 0);
        }
        if (slice < d.slices)
            red[set * set_size + (b * d.slices + slice) * 64 + lane] = make_float2((acc[2] + acc[1]) + acc[0], acc[3]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (++s < d.per_wave) return;
        s = 0;
        if (++b < d.batch && j + 1 < mine) return;
        __syncthreads();
        for (int o = threadIdx.x; o < 16 * a.m * b; o += kMvMaxWaves * 64) {
            const int col = o & 15, tk = (o >> 4) % a.m, tl = (o >> 4) / a.m;
            const int64_t row = ((int64_t)first + (int64_t)tl * gridDim.x) * kMvRows + col;
            const float2 *r = red + set * set_size + tl * d.slices * 64 + col;
            float y = 0.0f;
            for (int p0 = 0; p0 < d.slices; p0 += a.parts) {
                float sum = token_sum(r + p0 * 64, tk);
                for (int p = 1; p < a.parts && p0 + p < d.slices; p++) sum += token_sum(r + (p0 + p) * 64, tk);
                y = p0 == 0 ? sum : y + sum;
            }
            if (row < a.n) a.y[(int64_t)tk * a.n + row] = y;
        }
        b = 0;
        first += d.batch * gridDim.x;
        if (d.two_sets)
            set ^= 1;
        else
            __syncthreads();
    };
#pragma unroll 1
    for (int j = 0; j < mine; j += kMvAhead) {
        item(t[0], j);
        if (j + 1 < mine) item(t[1], j + 1);
        if (j + 2 < mine) item(t[2], j + 2);
        if (j + 3 < mine) item(t[3], j + 3);
    }
}

template <bool WIDE>
static int launch_decode(MvDecode d, int cus, hipStream_t s) {
    static LaunchCache cache;
    const void *fn = reinterpret_cast<const void *>(&mxfp4_decode_kernel<WIDE>);
    const int rc = raise_lds_limit(cache, fn, 160 * 1024);
    if (rc) return rc;
    const int fixed = 3 * d.a.m * (d.slices * kMvSlice * 2 + 16) + kMvMaxWaves * kMvTileBytes;
    const int tiles = (d.a.n + kMvRows - 1) / kMvRows;
    const int each = (tiles + cus - 1) / cus;
    d.per_wave = (d.slices + kMvMaxWaves - 1) / kMvMaxWaves;
    d.batch = each < 4 ? each : 4;
    if (d.batch > 4 / d.per_wave) d.batch = d.per_wave >= 4 ? 1 : 4 / d.per_wave;
    const int set_bytes = d.batch * d.slices * 64 * (int)sizeof(float2);
    d.two_sets = fixed + 2 * set_bytes <= 160 * 1024;
    const int bytes = fixed + (d.two_sets ? 2 : 1) * set_bytes;
    const int most = cus * blocks_per_cu(cache, fn, kMvMaxWaves * 64, bytes, 2);
    const int rounds = (tiles + most - 1) / most;
    const int grid = (tiles + rounds - 1) / rounds;
    hipLaunchKernelGGL((mxfp4_decode_kernel<WIDE>), dim3(grid), dim3(kMvMaxWaves * 64), bytes, s, d);
    return launch_status();
}

template <int G, bool WIDE>
static int launch_mv(MvArgs a, hipStream_t s) {
    static LaunchCache cache;
    const void *fn = reinterpret_cast<const void *>(&mxfp4_gemv_kernel<G, WIDE>);
    const int waves = a.parts * a.groups;
    const int stream_bytes = waves * (kMvTileBytes + 4 * G * 64 * (int)sizeof(float2));
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
    if (k > 1 << 24) return BQM_EUNSUPPORTED;   // 16 rows of x and of w in 31 bits
    MvArgs a = {w, ws, x, y, m, k, n, 0, 0, 0};
    const int slices = (k + kMvSlice - 1) / kMvSlice;
    a.passes = (slices + kMvMaxWaves - 1) / kMvMaxWaves;
    a.parts = (slices + a.passes - 1) / a.passes;
    a.groups = kMvMaxWaves / a.parts;
    hipStream_t s = as_stream(stream);
    // up to five tokens: in one pass if x, the tiles and one batch's results fit in LDS
    if (m <= 5 && (int64_t)slices * (3 * m * kMvSlice * 2 + 512) + 3 * m * 16 + kMvMaxWaves * kMvTileBytes <= 160 * 1024) {
        const MvDecode d = {a, slices, 0, 0, 0};
        return k % 128 == 0 && aligned(ws, 4) ? launch_decode<true>(d, device_cus(), s) : launch_decode<false>(d, device_cus(), s);
    }
    if (m <= 5) return launch_mv_scales<1>(a, s);
    if (m <= 10) return launch_mv_scales<2>(a, s);
    return launch_mv_scales<3>(a, s);
}
