// The MXFP4 x MXFP4 product for few tokens (up to 64, as long as their codes
// fit in registers or LDS): HBM-bound, every weight read once.  And for more
// tokens in chunks, where the output has too few tiles for the other kernel to
// fill the card: the waves share k (98 x 12512 x 320 12 us against 47, 512 x
// 17408 x 512 27 against 46).
//
//  * Up to k = 4096 a wave has one 512-k slice of every tile and keeps the
//    tokens' operand for it in registers.  Beyond, the workgroup keeps the
//    tokens' codes and scales in LDS, in the order in which the matrix cores
//    take them: a lane's 16 bytes of each 16-token group and 128-k step follow
//    the lane before's, and its four scales of 512 k are one dword.
//  * A wave streams tiles of 16 weight rows, 512 k at a time, straight from
//    memory into the operand registers of v_mfma_scale_f32_16x16x128 (lane:
//    row r = l % 16, block 4 i + l / 16 of step i), kAhead items ahead.
//  * The workgroup's waves share a tile's k (`parts` of them), or where a row
//    has fewer than eight slices several tiles; parts meet in LDS, added in
//    wave order.
//
// Weights from HBM: 16 x 4096 x 5152 8.0 us (latency: at 136 registers one
// workgroup a compute unit, so 66 of the 256 take a second of the 322 tiles),
// 16 x 4096 x 64448 30.2 us (4.8 TB/s), 16 x 17408 x 20480 44 us (4.3 TB/s).
#include <type_traits>

#include "mxfp4.h"

namespace bqm {

constexpr int kMsWaves = 8;
constexpr int kMsMaxGroups = 4;             // of 16 tokens
constexpr int kMsLds = 160 * 1024;
constexpr int kMsMaxChunks = 65535;         // of tokens: workgroups along y

struct MsArgs {
    MgArgs a;
    int slices;     // 512-k slices of a row
    int parts;      // waves along k
    int subs;       // tiles of a workgroup at a time: 8 / parts
    int per_wave;   // slices of a wave
};

// Bytes of LDS: codes, scales, one tile's partial results.
static int64_t ms_lds(int groups, int slices) { return (int64_t)groups * slices * (4096 + 256) + kMsWaves * 1024; }

template <int Q>
__device__ __forceinline__ v4f ms_mfma(u32x4 a, u32x4 b, v4f c, int sa, int sb) {
    const v8i va = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const v8i vb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, Q, sa, Q, sb);
}

// G: groups of 16 tokens; SW: scale rows in aligned 16-byte pieces (16) or bytes (1).
// XREG: a wave has one slice (k <= 4096), whose operand stays in its registers.
template <int G, int SW, bool XREG>
__global__ __launch_bounds__(kMsWaves * 64, G == 1 && !XREG ? 4 : 2) void mxfp4_stream_kernel(MsArgs d) {
    constexpr int kAhead = 3;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    MgArgs a = d.a;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int nblk = a.k / 32;
    const int64_t rb = a.k / 2;
    const int tiles = (a.n + 15) / 16;
    const int sub = wave / d.parts, wpart = wave % d.parts;   // with sub == subs: a wave without work
    const int hop = gridDim.x * d.subs;

    // this workgroup's tokens
    const int t0 = blockIdx.y * (16 * G);
    a.m = a.m - t0 < 16 * G ? a.m - t0 : 16 * G;
    a.xq += t0 * rb;
    a.xs += (int64_t)t0 * nblk;
    a.y += t0 * a.ldy;

    uint8_t *const xc = lds;                                              // [G][slices][4 steps][64 lanes][16]
    int *const xsc = reinterpret_cast<int *>(lds + G * d.slices * 4096);  // [G][slices][64 lanes]
    v4f *const red = reinterpret_cast<v4f *>(lds + (XREG ? 0 : G * d.slices * (4096 + 256)));   // [waves][64 lanes]

    struct Tile {
        u32x4 c[4];
        unsigned s[4];   // SW == 16: the row's 16 scales; else this lane's four
    };
    int next_tile = sub < d.subs ? blockIdx.x * d.subs + sub : tiles, next_s = 0;
    auto load = [&](Tile &q) {
        const int64_t row0 = (int64_t)next_tile * 16;
        const int64_t rows = a.n - row0 < 16 ? a.n - row0 : 16;   // may be <= 0: nothing is read
        const __amdgpu_buffer_rsrc_t rw = mx_rsrc(a.w + row0 * rb, rows * rb);
        const __amdgpu_buffer_rsrc_t rs = mx_rsrc(a.ws + row0 * nblk, rows * nblk);
        const int blk0 = (wpart + d.parts * next_s) * 16;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int b = blk0 + 4 * i + g4;   // blocks past the row's end are read as zeros
            q.c[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                         rw, b < nblk ? (uint32_t)(r16 * rb + 16 * b) : 0x80000000u, 0, 0));
        }
        if constexpr (SW == 16) {
            const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                rs, blk0 < nblk ? (uint32_t)(r16 * nblk + blk0) : 0x80000000u, 0, 0));
#pragma unroll
            for (int i = 0; i < 4; i++) q.s[i] = v[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int b = blk0 + 4 * i + g4;
                q.s[i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rs, b < nblk ? (uint32_t)(r16 * nblk + b) : 0x80000000u, 0, 0);
            }
        }
        if (++next_s == d.per_wave) {
            next_s = 0;
            next_tile += hop;
        }
    };
    // this lane's four scales, one a byte, from what SW loads
    auto scales = [&](const unsigned (&s)[4]) {
        if constexpr (SW == 16) {
            // byte g4 of each dword
            const unsigned sel = 0x0C0C0400u + 0x0101u * (unsigned)g4;
            const unsigned lo = __builtin_amdgcn_perm(s[1], s[0], sel), hi = __builtin_amdgcn_perm(s[3], s[2], sel);
            return (int)(lo | hi << 16);
        } else {
            return (int)(s[0] | s[1] << 8 | s[2] << 16 | s[3] << 24);
        }
    };

    // The tokens' codes and scales; tokens and blocks past the ends are zeros.
    const __amdgpu_buffer_rsrc_t rx = mx_rsrc(a.xq, a.m * rb), rxs = mx_rsrc(a.xs, (int64_t)a.m * nblk);
    auto x_codes = [&](int grp, int b, bool in) {
        return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                   rx, in && b < nblk ? (uint32_t)((16 * grp + r16) * rb + 16 * b) : 0x80000000u, 0, 0));
    };
    auto x_scales = [&](unsigned (&s)[4], int grp, int slice, bool in) {
        if constexpr (SW == 16) {
            const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                rxs, in && 16 * slice < nblk ? (uint32_t)((16 * grp + r16) * nblk + 16 * slice) : 0x80000000u, 0, 0));
#pragma unroll
            for (int i = 0; i < 4; i++) s[i] = v[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int b = 16 * slice + 4 * i + g4;
                s[i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rxs, in && b < nblk ? (uint32_t)((16 * grp + r16) * nblk + b) : 0x80000000u, 0, 0);
            }
        }
    };
    u32x4 xr[XREG ? G : 1][4];
    unsigned xrs[XREG ? G : 1][4];
    Tile it[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; i++) load(it[i]);
    if constexpr (XREG) {
#pragma unroll
        for (int grp = 0; grp < G; grp++) {
#pragma unroll
            for (int i = 0; i < 4; i++) xr[grp][i] = x_codes(grp, 16 * wpart + 4 * i + g4, sub < d.subs);
            x_scales(xrs[grp], grp, wpart, sub < d.subs);
        }
    }
    if constexpr (!XREG) {
        // several loads of a thread at a time
        constexpr int U = 8;
        const int steps = G * d.slices * 4, per = d.slices * 4;   // a wave writes a step's 1 KiB
        for (int st0 = wave; st0 < steps; st0 += U * kMsWaves) {
            u32x4 v[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int st = st0 + u * kMsWaves, grp = st / per;
                v[u] = x_codes(grp, (st - grp * per) * 4 + g4, st < steps);
            }
#pragma unroll
            for (int u = 0; u < U; u++)
                if (st0 + u * kMsWaves < steps) *reinterpret_cast<u32x4 *>(xc + (st0 + u * kMsWaves) * 1024 + 16 * lane) = v[u];
        }
        constexpr int V = 4;
        for (int sl0 = wave; sl0 < G * d.slices; sl0 += V * kMsWaves) {
            unsigned v[V][4];
#pragma unroll
            for (int u = 0; u < V; u++) {
                const int sl = sl0 + u * kMsWaves, grp = sl / d.slices;
                x_scales(v[u], grp, sl - grp * d.slices, sl < G * d.slices);
            }
#pragma unroll
            for (int u = 0; u < V; u++)
                if (sl0 + u * kMsWaves < G * d.slices) xsc[(sl0 + u * kMsWaves) * 64 + lane] = scales(v[u]);
        }
        __syncthreads();
    }

    v4f acc[G] = {};
    int s = 0, first = blockIdx.x * d.subs;   // slice turn, the workgroup's current first tile
    const int mine = (tiles - first + hop - 1) / hop * d.per_wave;   // items, the same for all waves
    auto item = [&](Tile &q) {
        // a tile's first slice starts from zero (a select: no branch splits the
        // accumulators' lifetime)
        const float keep = s == 0 ? 0.0f : 1.0f;
#pragma unroll
        for (int grp = 0; grp < G; grp++)
#pragma unroll
            for (int e = 0; e < 4; e++) acc[grp][e] = keep != 0.0f ? acc[grp][e] : 0.0f;
        const int slice = wpart + d.parts * s;
        const int at = slice < d.slices ? slice : 0;   // past the end: zero weights
        const int sb = scales(q.s);
#pragma unroll
        for (int grp = 0; grp < G; grp++) {
            int sa;
            if constexpr (XREG)
                sa = scales(xrs[grp]);
            else
                sa = xsc[(grp * d.slices + at) * 64 + lane];
            const uint8_t *const p = xc + (grp * d.slices + at) * 4096 + 16 * lane;
            auto step = [&](auto qq) {
                constexpr int Q = decltype(qq)::value;
                u32x4 x;
                if constexpr (XREG)
                    x = xr[grp][Q];
                else
                    x = *reinterpret_cast<const u32x4 *>(p + Q * 1024);
                acc[grp] = ms_mfma<Q>(x, q.c[Q], acc[grp], sa, sb);
            };
            step(std::integral_constant<int, 0>{});
            step(std::integral_constant<int, 1>{});
            step(std::integral_constant<int, 2>{});
            step(std::integral_constant<int, 3>{});
        }
        load(q);
        if (++s < d.per_wave) return;
        s = 0;
        // lane: weight row r16, tokens 4 g4 + v of each group
#pragma unroll
        for (int grp = 0; grp < G; grp++) {
            if (d.parts > 1) {
                red[wave * 64 + lane] = acc[grp];
                __syncthreads();
                if (wpart == 0 && sub < d.subs) {
                    const v4f *const q0 = red + sub * d.parts * 64 + lane;
                    v4f v[kMsWaves];
#pragma unroll
                    for (int p = 0; p < kMsWaves; p++) v[p] = q0[(p < d.parts ? p : 0) * 64];
#pragma unroll
                    for (int p = 1; p < kMsWaves; p++)
                        if (p < d.parts) v[0] += v[p];
                    acc[grp] = v[0];
                }
                __syncthreads();
            }
            if (wpart == 0 && sub < d.subs) {
                const int64_t row = (int64_t)(first + sub) * 16 + r16;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (row < a.n && 16 * grp + 4 * g4 + e < a.m) a.y[(16 * grp + 4 * g4 + e) * a.ldy + row] = acc[grp][e];
            }
        }
        first += hop;
    };
#pragma unroll 1
    for (int j = 0; j < mine; j += kAhead) {
        item(it[0]);
        if (j + 1 < mine) item(it[1]);
        if (j + 2 < mine) item(it[2]);
    }
}

template <int G, int SW, bool XREG>
static int launch_ms(MsArgs d, int cus, hipStream_t s) {
    static LaunchCache cache;
    const void *fn = reinterpret_cast<const void *>(&mxfp4_stream_kernel<G, SW, XREG>);
    const int rc = raise_lds_limit(cache, fn, kMsLds);
    if (rc) return rc;
    const int tiles = (d.a.n + 15) / 16;
    d.slices = (d.a.k + 511) / 512;
    d.parts = d.slices < kMsWaves ? d.slices : kMsWaves;
    d.subs = kMsWaves / d.parts;
    d.per_wave = (d.slices + d.parts - 1) / d.parts;
    const int bytes = (int)ms_lds(XREG ? 0 : G, d.slices);
    const int units = (tiles + d.subs - 1) / d.subs;
    const int chunks = (d.a.m + 16 * G - 1) / (16 * G);
    int most = cus * blocks_per_cu(cache, fn, kMsWaves * 64, bytes, 2) / chunks;
    if (most < 1) most = 1;
    hipLaunchKernelGGL((mxfp4_stream_kernel<G, SW, XREG>), dim3(units < most ? units : most, chunks), dim3(kMsWaves * 64), bytes, s, d);
    return launch_status();
}

template <int G>
static int launch_ms_g(const MgArgs &a, hipStream_t s) {
    const MsArgs d = {a, 0, 0, 0, 0};
    const int cus = device_cus();
    const bool wide = scale_load(a.k / 32, a.ws, a.xs) == 16;
    if (a.k <= kMsWaves * 512) return wide ? launch_ms<G, 16, true>(d, cus, s) : launch_ms<G, 1, true>(d, cus, s);
    return wide ? launch_ms<G, 16, false>(d, cus, s) : launch_ms<G, 1, false>(d, cus, s);
}

// Few tokens whose operand fits, against few enough weight rows: with many the
// other kernel's 128-row tiles fill the card and move the tokens' codes less
// often, the earlier the more groups of 16 tokens there are.  Measured (this,
// tiles; us): 16 x 4096 x 5152 8.0, 16.8, x 64448 30.2, 31.5; 32 x 4096 x 32768
// 20.3, 21.8; 48 x 4096 x 20480 18.6, 18.9, x 32768 23.9, 23.1; 64 x 4096 x
// 8192 14.2, 18.5, x 12288 17.6, 18.9, x 16384 19.9, 19.0.
//
// More tokens, or more than fit, go in chunks that each stream the weights
// (again, from the caches): that fills the card where 128-row tiles are few and
// k is long.  The chunks' estimated time decides, with a margin: 6 us, and for
// each tile that a compute unit gets and each slice that a wave has of it the
// time below.
int mxfp4_stream_groups(int m, int k, int n, int cus, double tile_cost) {
    const int groups = (m + 15) / 16;
    auto fits = [&](int g) { return k <= kMsWaves * 512 || ms_lds(g, (int)(((int64_t)k + 511) / 512)) <= kMsLds; };
    if (groups <= kMsMaxGroups && fits(groups)) {
        const int rows = groups == 2 ? 128 : groups == 3 ? 80 : 48;   // of weights for a compute unit, at most
        return groups == 1 || n <= rows * cus ? groups : 0;
    }
    const double in_registers[kMsMaxGroups] = {1.55, 1.75, 1.8, 2.4}, in_lds[kMsMaxGroups] = {1.1, 1.75, 2.5, 3.2};
    const double *const item = k <= kMsWaves * 512 ? in_registers : in_lds;
    const int slices = (int)(((int64_t)k + 511) / 512), parts = slices < kMsWaves ? slices : kMsWaves;
    const int per_wave = (slices + parts - 1) / parts, subs = kMsWaves / parts;
    const int64_t units = ((n + 15) / 16 + subs - 1) / subs;
    int best = 0;
    for (int g = 1; g <= kMsMaxGroups && g <= groups && fits(g); g++) {
        const int chunks = (groups + g - 1) / g;
        if (chunks > kMsMaxChunks) continue;
        const int64_t all = units * chunks;
        const double cost = 1.15 * (6.0 + (double)((all + cus - 1) / cus) * per_wave * item[g - 1]);
        if (cost < tile_cost) {
            tile_cost = cost;
            best = g;
        }
    }
    return best;
}

int mxfp4_stream(const MgArgs &a, int groups, hipStream_t s) {
    switch (groups) {
        case 1: return launch_ms_g<1>(a, s);
        case 2: return launch_ms_g<2>(a, s);
        case 3: return launch_ms_g<3>(a, s);
        default: return launch_ms_g<4>(a, s);
    }
}

}  // namespace bqm
