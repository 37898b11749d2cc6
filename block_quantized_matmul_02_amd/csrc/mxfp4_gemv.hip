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
//    three (the last in the rows that five of a group leave).  Rows do not
//    mix: a token's result is the same bits at every m.
//  * A wave owns 512 k (16 scale blocks) and keeps its x operands for them in
//    registers (64 VGPRs per 16 operand rows); the workgroup's waves cover up
//    to 4096 k and the k beyond them in further passes, which add to y.
//  * Weight rows stream through registers into a wave's own LDS tile (16 rows
//    x 256 bytes, loaded 256 contiguous bytes per row, two tiles ahead), from
//    which a lane reads the 16-byte block of its row: lane group g holds
//    blocks 4g .. 4g+3 of the 512 k, so that its four scales are one dword.
//    The order of k inside a step is the same for x, and free.
//    (Straight from memory into the operand registers, four lanes to 64
//    contiguous bytes, is slower at most sizes: 1 x 4096 x 64448 41.2 us
//    against 28.9, 4 x 5120 x 17408 32.3 against 24.1; at 16 x 4096 x 4096
//    13.7 against 14.2.)
//  * The waves' partial tiles meet in LDS, added in wave order.
//
// Weights from HBM: 1 x 4096 x 4096 7.2 us (latency), 1 x 4096 x 64448 28.9 us
// (4.9 TB/s), 9 x 4096 x 64448 32.8 us (4.3 TB/s), 5 x 17408 x 5120 28.1 us.
// Long rows are further from the weights' time (1 x 17408 x 5120 24.1 us, 9.3
// for its bytes): 320 tiles are two rounds of 256 workgroups, 34 slices five
// turns of eight waves, and x is cut first.  G = 3 fills the registers and
// spills 6 (11 with unaligned scales) to scratch: 16 x 4096 x 64448 43 us.
#include "mxfp4.h"

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

// Where a token's sum stands among the lanes' results of a wave's tile (as
// floats, column 0): tokens 0..3 of a group in one place, its token 4 and the
// sixteenth token in three, which are added the smallest part first.  Without
// branches, so that the reads of several waves' results overlap.
struct TokenSum {
    int a, b, c;
    bool split;

    __device__ __forceinline__ explicit TokenSum(int tok) {
        const int i = tok % 5, at = 2 * 64 * (tok / 5);
        split = tok == 15 || i == 4;
        a = tok == 15 ? 2 * 48 + 1 : i < 4 ? at + 2 * 16 * i : at + 1;
        b = tok == 15 ? 2 * (64 + 48) + 1 : i < 4 ? a : a + 2 * 16;
        c = tok == 15 ? 2 * (128 + 48) + 1 : i < 4 ? a : a + 2 * 32;
    }
    __device__ __forceinline__ float operator()(const float2 *r) const {
        const float *const f = reinterpret_cast<const float *>(r);
        const float x = f[a], y = f[b], z = f[c];
        return split ? (z + y) + x : x;
    }
};

// WIDE: scale rows are whole, aligned dwords (k % 128 == 0); else bytes.
template <int G, bool WIDE>
__global__ __launch_bounds__(kMvMaxWaves * 64, 2) void mxfp4_gemv_kernel(MvArgs a) {
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
        // values are asked for before the first weights, all at once.
        MvTile t0, t1;
        v8bf xop[G][16];
        {
            uint8_t *const xs = lds + wave * (16 * kMvXStride);
            const __amdgpu_buffer_rsrc_t rx = mx_rsrc(a.x, 4ll * a.m * a.k);
            // k % 32 == 0: a lane's eight values are in or out of the row together
            const uint32_t off = 32 * blk0 + 8 * lane < a.k ? (uint32_t)(4 * (32 * blk0 + 8 * lane)) : 0x80000000u;
            // a group's five tokens and, of three groups, the sixteenth
            constexpr int kTok = G == 3 ? 6 : 5;
            u32x4 all[G][kTok][2];
#pragma unroll
            for (int grp = 0; grp < G; grp++)
#pragma unroll
                for (int i = 0; i < kTok; i++) {
                    // tokens past the last read zeros
                    const uint32_t at = off + (uint32_t)(4 * a.k) * (i < 5 ? 5 * grp + i : 15);
                    all[grp][i][0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, at, 0, 0));
                    all[grp][i][1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, at + 16, 0, 0));
                }
            load(t0, 0);
            if constexpr (G < 3) load(t1, 1);
#pragma unroll
            for (int grp = 0; grp < G; grp++) {
                const auto &raw = all[grp];
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

        auto multiply = [&](MvTile &t, int next, float2 *out) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                *reinterpret_cast<u32x4 *>(tile + (4 * i + g4) * kMvRowStride + 16 * r16) = t.c[i];
            const unsigned sc = t.s;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            load(t, next);
            v4f acc[G];
#pragma unroll
            for (int grp = 0; grp < G; grp++) acc[grp] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const u32x4 c = *reinterpret_cast<const u32x4 *>(tile + r16 * kMvRowStride + (4 * g4 + q) * 16);
                const float s = __builtin_bit_cast(float, ((sc >> (8 * q)) & 255u) << 23);
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
            if constexpr (G < 3) {
                multiply(t0, round + 2, set + wave * kRed);
                multiply(t1, round + 3, set + (waves + wave) * kRed);
            } else {
                multiply(t0, round + 1, set + wave * kRed);
                multiply(t0, round + 2, set + (waves + wave) * kRed);
            }
            __syncthreads();
            for (int o = part * 64 + lane, i = 0; o < 32 * a.m; o += 64 * a.parts, i++) {
                int tok, col;
                int64_t at;
                if (!where(o, tok, col, at)) continue;
                const float2 *const q = set + ((o >= 16 * a.m ? waves : 0) + group * a.parts) * kRed + col;
                const TokenSum token(tok);
                float v[kMvMaxWaves];
#pragma unroll
                for (int p = 0; p < kMvMaxWaves; p++) {
                    const float2 *const r = q + (p < a.parts ? p : 0) * kRed;
                    const float one = token(r);
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
// lanes' worth), so a wave goes through any number of 512-k slices.  An item is
// one slice of R tiles of 16 weight rows, which share the operand and give R
// independent chains of MFMAs; kAhead items are on their way.  Each slice's
// result is kept apart in LDS, so that they are added as the passes above add
// them: a token's bits do not depend on which kernel ran.
struct MvDecode {
    MvArgs a;
    int slices;     // 512-k slices of a row
    int parts;      // waves along k: min(slices, 8)
    int subs;       // groups of tiles of a workgroup at a time: 8 / parts
    int per_wave;   // slices of a wave: ceil(slices / parts)
    int batch;      // groups of R tiles between barriers
    int two_sets;   // results have two sets in LDS; else a second barrier
};

template <int R, bool WIDE>
__global__ __launch_bounds__(kMvMaxWaves * 64, R == 2 && WIDE ? 4 : 2) void mxfp4_decode_kernel(MvDecode d) {
    constexpr int kAhead = R == 1 ? 4 : 1;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const MvArgs &a = d.a;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int nblk = a.k / 32;
    const int64_t row_bytes = a.k / 2;
    const int groups = (a.n + R * kMvRows - 1) / (R * kMvRows);   // groups of R tiles
    const int xstride = d.slices * kMvSlice * 2 + 16;

    uint8_t *const xs = lds;
    uint8_t *const tile = lds + 3 * a.m * xstride + wave * kMvTileBytes;
    float2 *const red = reinterpret_cast<float2 *>(lds + 3 * a.m * xstride + kMvMaxWaves * kMvTileBytes);
    const int set_size = d.subs * d.batch * R * d.slices * 64;
    const int sub = wave / d.parts, wpart = wave % d.parts;   // with sub == subs: a wave without work
    const int hop = gridDim.x * d.subs;

    // item j of this wave: its group j / per_wave, slice wpart + parts (j % per_wave)
    int next_group = sub < d.subs ? blockIdx.x * d.subs + sub : groups, next_s = 0;
    struct Item {
        MvTile t[R];
    };
    Item it[kAhead];
    auto load = [&](Item &q) {
        const int64_t row0 = (int64_t)next_group * (R * kMvRows);
        const int64_t rows = a.n - row0 < R * kMvRows ? a.n - row0 : R * kMvRows;   // may be <= 0: nothing is read
        const int blk0 = (wpart + d.parts * next_s) * kMvBlocks;
        const __amdgpu_buffer_rsrc_t rw = mx_rsrc(a.w + row0 * row_bytes, rows * row_bytes);
        const __amdgpu_buffer_rsrc_t rs = mx_rsrc(a.ws + row0 * nblk, rows * nblk);
        const uint32_t off = blk0 + r16 < nblk ? (uint32_t)(g4 * row_bytes + 16 * (blk0 + r16)) : 0x80000000u;
        const int b = blk0 + 4 * g4;
#pragma unroll
        for (int h = 0; h < R; h++) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                q.t[h].c[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, off + (uint32_t)((16 * h + 4 * i) * row_bytes), 0, 0));
            if constexpr (WIDE) {
                q.t[h].s = __builtin_amdgcn_raw_buffer_load_b32(rs, b < nblk ? (uint32_t)((16 * h + r16) * nblk + b) : 0x80000000u, 0, 0);
            } else {
                q.t[h].s = 0;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    q.t[h].s |= (unsigned)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                                    rs, b + e < nblk ? (uint32_t)((16 * h + r16) * nblk + b + e) : 0x80000000u, 0, 0) << (8 * e);
            }
        }
        if (++next_s == d.per_wave) {
            next_s = 0;
            next_group += hop;
        }
    };

    // x: eight values a thread and turn; zeros up to a whole slice
    const int per_row = d.slices * 64;
    const __amdgpu_buffer_rsrc_t rx = mx_rsrc(a.x, 4ll * a.m * a.k);
    auto load_x = [&](int i, u32x4 (&v)[2]) {
        const int tok = i / per_row, at = i - tok * per_row;
        const uint32_t off = 8 * at < a.k ? (uint32_t)(4 * (tok * a.k + 8 * at)) : 0x80000000u;
        v[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, off, 0, 0));
        v[1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, off + 16, 0, 0));
    };
    auto store_x = [&](int i, const u32x4 (&v)[2]) {
        const int tok = i / per_row, at = i - tok * per_row;
        u32x4 p[3];
        three_parts(v, p);
        if (i < a.m * per_row) {
#pragma unroll
            for (int h = 0; h < 3; h++) *reinterpret_cast<u32x4 *>(xs + (3 * tok + h) * xstride + 16 * at) = p[h];
        }
    };
    {
        // the values are asked for before the first weights, all at once: what
        // fits in LDS is at most five turns
        constexpr int T = kMvMaxWaves * 64, kTurns = 5;
        const int turns = (a.m * per_row + T - 1) / T;
        u32x4 v[kTurns][2];
#pragma unroll
        for (int u = 0; u < kTurns; u++)
            if (u < turns) load_x(threadIdx.x + u * T, v[u]);
#pragma unroll
        for (int i = 0; i < kAhead; i++) load(it[i]);
#pragma unroll
        for (int u = 0; u < kTurns; u++)
            if (u < turns) store_x(threadIdx.x + u * T, v[u]);
    }
    __syncthreads();

    // this lane's operand row: rows 4i + h and 4h + 3 of the sixteen, as above
    const int tok = (r16 & 3) < 3 ? r16 >> 2 : 4, part = (r16 & 3) < 3 ? r16 & 3 : r16 >> 2;
    const bool used = tok < a.m && r16 != 15;
    const uint8_t *const xrow = xs + (used ? 3 * tok + part : 0) * xstride + 4 * g4 * 64;

    int s = 0, b = 0, first = blockIdx.x * d.subs, set = 0;   // slice turn, group of the batch, the batch's first group
    const int mine = (groups - first + hop - 1) / hop * d.per_wave;   // items, the same for all waves
    auto item = [&](Item &q, int j) {
        u32x4 c[R][4];
        unsigned sc[R];
#pragma unroll
        for (int h = 0; h < R; h++) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                *reinterpret_cast<u32x4 *>(tile + (4 * i + g4) * kMvRowStride + 16 * r16) = q.t[h].c[i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int i = 0; i < 4; i++) c[h][i] = *reinterpret_cast<const u32x4 *>(tile + r16 * kMvRowStride + (4 * g4 + i) * 16);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            sc[h] = q.t[h].s;
        }
        load(q);
        const int slice = wpart + d.parts * s;
        const uint8_t *const xp = xrow + (slice < d.slices ? slice : 0) * (kMvSlice * 2);
        v4f acc[R];
#pragma unroll
        for (int h = 0; h < R; h++) acc[h] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int qq = 0; qq < 4; qq++) {
            u32x4 xv[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                xv[e] = u32x4{0, 0, 0, 0};
                if (used) xv[e] = *reinterpret_cast<const u32x4 *>(xp + qq * 64 + e * 16);
            }
#pragma unroll
            for (int e = 0; e < 4; e++)
#pragma unroll
                for (int h = 0; h < R; h++) {
                    const float f = __builtin_bit_cast(float, ((sc[h] >> (8 * qq)) & 255u) << 23);
                    acc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, xv[e]), eight(c[h][qq][e], f), acc[h], 0, 0, 0);
                }
        }
        if (slice < d.slices && sub < d.subs) {
#pragma unroll
            for (int h = 0; h < R; h++)
                red[set * set_size + (((b * d.subs + sub) * R + h) * d.slices + slice) * 64 + lane] = make_float2((acc[h][2] + acc[h][1]) + acc[h][0], acc[h][3]);
        }
        if (++s < d.per_wave) return;
        s = 0;
        if (++b < d.batch && j + 1 < mine) return;
        __syncthreads();
        // A pass's waves are added in wave order, then the passes.  With more
        // than one pass, four lanes share an output, a pass each in turn, and
        // the first adds what they find.
        const int per = d.slices > a.parts ? 4 : 1;
        for (int o = threadIdx.x; o < 16 * R * a.m * b * d.subs * per; o += kMvMaxWaves * 64) {
            const int col = o & 15, unit = (o >> 4) / per, lead = per == 1 ? 0 : (o >> 4) & 3;
            const int tk = unit % a.m, tl = unit / a.m, gr = tl / R;   // group gr % subs of the batch's gr / subs
            const int64_t row = (((int64_t)first + (int64_t)(gr / d.subs) * hop + gr % d.subs) * R + tl % R) * kMvRows + col;
            const float2 *r = red + set * set_size + tl * d.slices * 64 + col;
            const TokenSum token(tk);
            auto pass_sum = [&](int p0) {
                float v[kMvMaxWaves];
#pragma unroll
                for (int p = 0; p < kMvMaxWaves; p++) {
                    const bool in = p < a.parts && p0 + p < d.slices;
                    const float one = token(r + (in ? p0 + p : 0) * 64);
                    v[p] = in ? one : 0.0f;
                }
                float sum = v[0];
#pragma unroll
                for (int p = 1; p < kMvMaxWaves; p++) sum += v[p];
                return sum;
            };
            float y = pass_sum(lead * a.parts);
            if (per == 4) {
                // 16 outputs x 4 lanes are a wave's, whole (16 R m b subs per is a multiple of 64)
                const int src = lane & 15;
                float all = 0.0f;
                for (int p0 = 0; p0 < a.passes; p0 += 4) {
                    const float mine_sum = p0 == 0 ? y : pass_sum((p0 + lead) * a.parts);
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const float one = __shfl(mine_sum, src + 16 * q);
                        if (p0 + q < a.passes) all = p0 + q == 0 ? one : all + one;
                    }
                }
                y = all;
            }
            if (row < a.n && lead == 0) a.y[(int64_t)tk * a.n + row] = y;
        }
        b = 0;
        first += d.batch * hop;
        if (d.two_sets)
            set ^= 1;
        else
            __syncthreads();
    };
#pragma unroll 1
    for (int j = 0; j < mine; j += kAhead) {
        item(it[0], j);
        if constexpr (kAhead == 4) {
            if (j + 1 < mine) item(it[1], j + 1);
            if (j + 2 < mine) item(it[2], j + 2);
            if (j + 3 < mine) item(it[3], j + 3);
        }
    }
}

// LDS of the operand and the waves' tiles.
static int decode_lds(int m, int slices) { return 3 * m * (slices * kMvSlice * 2 + 16) + kMvMaxWaves * kMvTileBytes; }

template <int R, bool WIDE>
static int launch_decode_r(MvDecode d, int cus, hipStream_t s) {
    static LaunchCache cache;
    const void *fn = reinterpret_cast<const void *>(&mxfp4_decode_kernel<R, WIDE>);
    const int rc = raise_lds_limit(cache, fn, 160 * 1024);
    if (rc) return rc;
    const int fixed = decode_lds(d.a.m, d.slices);
    const int groups = (d.a.n + R * kMvRows - 1) / (R * kMvRows);
    d.parts = d.slices < kMvMaxWaves ? d.slices : kMvMaxWaves;
    d.subs = kMvMaxWaves / d.parts;
    d.per_wave = (d.slices + d.parts - 1) / d.parts;
    const int one = d.subs * R * d.slices * 64 * (int)sizeof(float2);
    d.batch = 4 / R / d.per_wave;
    const int units = (groups + d.subs - 1) / d.subs, each = (units + cus - 1) / cus;
    if (d.batch > each) d.batch = each;
    if (d.batch < 1) d.batch = 1;
    while (d.batch > 1 && fixed + d.batch * one > 160 * 1024) d.batch--;
    d.two_sets = fixed + 2 * d.batch * one <= 160 * 1024;
    const int bytes = fixed + (d.two_sets ? 2 : 1) * d.batch * one;
    const int most = cus * blocks_per_cu(cache, fn, kMvMaxWaves * 64, bytes, 2);
    hipLaunchKernelGGL((mxfp4_decode_kernel<R, WIDE>), dim3(units < most ? units : most), dim3(kMvMaxWaves * 64), bytes, s, d);
    return launch_status();
}

// Two tiles an item where every compute unit gets some and their results fit.
template <bool WIDE>
static int launch_decode(const MvDecode &d, int cus, hipStream_t s) {
    const int one = d.slices < kMvMaxWaves ? kMvMaxWaves * 64 * 8 : d.slices * 64 * 8;   // bytes of a tile's results, at most
    const bool fits = decode_lds(d.a.m, d.slices) + 2 * one <= 160 * 1024;
    return fits && d.a.n >= 32 * cus ? launch_decode_r<2, WIDE>(d, cus, s) : launch_decode_r<1, WIDE>(d, cus, s);
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
    if (n > 0x7FFFFFFF - 2 * kMvRows) return BQM_EUNSUPPORTED;   // whole tiles, two at a time, in 31 bits
    MvArgs a = {w, ws, x, y, m, k, n, 0, 0, 0};
    const int slices = (k + kMvSlice - 1) / kMvSlice;
    a.passes = (slices + kMvMaxWaves - 1) / kMvMaxWaves;
    a.parts = (slices + a.passes - 1) / a.passes;
    a.groups = kMvMaxWaves / a.parts;
    hipStream_t s = as_stream(stream);
    // up to five tokens: in one pass if x, the tiles and one batch's results fit in LDS
    if (m <= 5 && slices * m <= 40 && decode_lds(m, slices) + (slices < kMvMaxWaves ? kMvMaxWaves : slices) * 512 <= 160 * 1024) {
        const MvDecode d = {a, slices, 0, 0, 0, 0, 0};
        return k % 128 == 0 && aligned(ws, 4) ? launch_decode<true>(d, device_cus(), s) : launch_decode<false>(d, device_cus(), s);
    }
    if (m <= 5) return launch_mv_scales<1>(a, s);
    if (m <= 10) return launch_mv_scales<2>(a, s);
    return launch_mv_scales<3>(a, s);
}
