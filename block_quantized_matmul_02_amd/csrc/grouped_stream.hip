// The grouped MXFP4 product for few slots a group, where the tiles of
// grouped_gemm.hip are too few to fill the card and each walks k alone.
//
// A workgroup takes up to 16 slots of one group against a strip of units of 32
// weight rows (with the gate: 16 of each half).  Its waves share k in slices of
// 512, or units where a row has few slices.  Weights go from memory straight
// into the operand registers of v_mfma_scale_f32_16x16x128 (lane: row l % 16,
// block 4 i + l / 16 of step i), an item (a slice of a unit) ahead; the slots'
// operand of a wave's slice stays in its registers where k <= 4096 and comes
// with each item beyond.  The waves' sums meet in LDS, added in wave order.
//
// In a graph, this and the tiles: 32 slots of 8 experts, 4096 x 1024 7.9 us and
// 13.8, 100 of 2, 8192 x 512 11.0 and 22.4, 200 of 8, 4096 x 1024 11.5 and 14.5;
// but 128 of 8, 2048 x 2816 14.4 and 11.0, 40 of 4, 768 x 512 7.1 and 6.0.  32
// slots a workgroup were no better (8.4, 13.3, 15.0).
#include <type_traits>

#include "grouped_gemm.h"

namespace bqm {

constexpr int kGsWaves = 8;

struct GsArgs {
    GgArgs a;
    int slices, parts, subs, per_wave;   // of k; waves along k; units at a time; slices of a wave
    int units, each, strips;             // of weight rows; of a workgroup; workgroups of 16 slots
};

template <int Q>
__device__ __forceinline__ v4f gs_mfma(u32x4 a, u32x4 b, v4f c, int sa, int sb) {
    const v8i va = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const v8i vb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, Q, sa, Q, sb);
}

// XREG: a wave has one slice (k <= 4096).
template <bool XREG, bool GLU>
__global__ __launch_bounds__(kGsWaves * 64) void grouped_stream_kernel(GsArgs d) {
    __shared__ v4f red[2][kGsWaves][2][64];
    __shared__ int slot_of[16];   // -1: not a row of y
    const GgArgs &a = d.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const GroupTile t = find_group(a.q, 16, d.strips, blockIdx.x);
    if (t.group > a.q.groups) return;
    const int chunk = t.local / d.strips, strip = t.local - chunk * d.strips;
    const int first = t.first + chunk * 16, rows = min(16, t.rows - chunk * 16);
    const int unit0 = strip * d.each, unit1 = min(unit0 + d.each, d.units);
    constexpr int COLS = GLU ? 16 : 32;   // columns of y of a unit
    if (tid < 16) {
        const unsigned s = tid < rows ? (unsigned)a.q.order[first + tid] : ~0u;
        slot_of[tid] = s < (unsigned)a.q.slots ? (int)s : -1;
    }
    if (t.group == a.q.groups) {   // slots of no group
        __syncthreads();
        const int lo = unit0 * COLS, cols = min(unit1 * COLS, a.outs) - lo;
        for (int i = 0; i < rows; i++)
            for (int j = tid; slot_of[i] >= 0 && j < cols; j += kGsWaves * 64) store_as(a.y, (int64_t)slot_of[i] * a.outs + lo + j, 0.0f, a.y_type);
        return;
    }

    const int nblk = a.k / 32;
    const int64_t rb = a.k / 2;
    const uint8_t *const w = a.w + (int64_t)t.group * a.n * rb, *const ws = a.ws + (int64_t)t.group * a.n * nblk;
    const int sub = wave / d.parts, wpart = wave % d.parts;   // sub == subs: a wave without work
    // this lane's four scales of a slice, one a byte: byte g4 of each dword
    auto pick = [&](const unsigned (&s)[4]) {
        const unsigned sel = 0x0C0C0400u + 0x0101u * (unsigned)g4;
        const unsigned lo = __builtin_amdgcn_perm(s[1], s[0], sel), hi = __builtin_amdgcn_perm(s[3], s[2], sel);
        return (int)(lo | hi << 16);
    };
    // slices past the last: the weights are zeros, and the scales those of a slice that there is
    auto block0 = [&](int slice) { return 16 * min(slice, d.slices - 1); };
    struct Tile {
        u32x4 c[4];
        unsigned s[4];
    };
    int next_unit = unit0 + sub, next_s = 0;
    auto load = [&](Tile (&q)[2]) {
        const int slice = wpart + d.parts * next_s, blk0 = 16 * slice;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int j0 = next_unit * COLS + (GLU ? 0 : 16 * h);
            const int64_t row0 = j0 + (GLU ? (int64_t)h * a.outs : 0);
            const int live = next_unit < unit1 && sub < d.subs ? min(a.outs - j0, 16) : 0;   // may be <= 0: nothing is read
            const __amdgpu_buffer_rsrc_t rw = mx_rsrc(w + row0 * rb, live * rb);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int b = blk0 + 4 * i + g4;
                q[h].c[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, b < nblk ? (uint32_t)(r16 * rb + 16 * b) : 0x80000000u, 0, 0));
            }
            const int64_t row = live > 0 ? row0 + min(r16, live - 1) : 0;
            scale_bytes(ws + row * nblk, block0(slice), nblk, q[h].s);
        }
        if (++next_s == d.per_wave) {
            next_s = 0;
            next_unit += d.subs;
        }
    };
    Tile it[2];
    load(it);
    __syncthreads();
    // the slots' rows of x: rows that are none read the last one, blocks past the end repeat the last one
    const int64_t xrow = max(slot_of[min(r16, rows - 1)], 0) / a.top;
    auto load_x = [&](Tile &x, int slice) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            x.c[i] = *reinterpret_cast<const u32x4 *>(a.xq + xrow * rb + 16 * min(16 * slice + 4 * i + g4, nblk - 1));
        scale_bytes(a.xs + xrow * nblk, block0(slice), nblk, x.s);
    };
    Tile x;
    if constexpr (XREG) load_x(x, wpart);

    v4f acc[2] = {};
    int s = 0, unit = unit0, set = 0;
    const int rounds = (unit1 - unit0 + d.subs - 1) / d.subs * d.per_wave;   // the same for all waves, which meet
#pragma unroll 1
    for (int j = 0; j < rounds; j++) {
        if constexpr (!XREG) load_x(x, wpart + d.parts * s);
        Tile now[2];
#pragma unroll
        for (int h = 0; h < 2; h++) now[h] = it[h];
        load(it);
        const int sa = pick(x.s);
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int sb = pick(now[h].s);
            acc[h] = gs_mfma<0>(x.c[0], now[h].c[0], acc[h], sa, sb);
            acc[h] = gs_mfma<1>(x.c[1], now[h].c[1], acc[h], sa, sb);
            acc[h] = gs_mfma<2>(x.c[2], now[h].c[2], acc[h], sa, sb);
            acc[h] = gs_mfma<3>(x.c[3], now[h].c[3], acc[h], sa, sb);
        }
        if (++s < d.per_wave) continue;
        s = 0;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            red[set][wave][h][lane] = acc[h];
            acc[h] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
        __syncthreads();
        // a lane's four results (weight row r16, slots 4 g4 .. + 3) of a unit's tile, all parts of k
        for (int p = wave; p < d.subs * (GLU ? 1 : 2); p += kGsWaves) {
            const int su = p % d.subs, h = p / d.subs;
            auto total = [&](int tile) {
                v4f sum = red[set][su * d.parts][tile][lane];
                for (int e = 1; e < d.parts; e++) sum += red[set][su * d.parts + e][tile][lane];
                return sum;
            };
            const int col = (unit + su) * COLS + (GLU ? 0 : 16 * h) + r16;
            v4f v = total(h);
            if (GLU) {
                const v4f up = total(1);
#pragma unroll
                for (int e = 0; e < 4; e++) v[e] = silu(v[e]) * up[e];
            }
            if (unit + su >= unit1 || col >= a.outs) continue;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int at = slot_of[4 * g4 + e];
                if (at >= 0) store_as(a.y, (int64_t)at * a.outs + col, v[e], a.y_type);
            }
        }
        unit += d.subs;
        set ^= 1;
    }
}

// Workgroups' chunks of 16 slots that an even spread over the groups makes.
static int64_t gs_chunks(const GgArgs &a) { return (a.q.groups < a.q.slots ? a.q.groups : a.q.slots) + a.q.slots / 16; }

template <bool GLU>
static int launch_gs(GsArgs d, int cus, hipStream_t s) {
    const GgArgs &a = d.a;
    d.slices = (a.k + 511) / 512;
    d.parts = d.slices < kGsWaves ? d.slices : kGsWaves;
    d.subs = kGsWaves / d.parts;
    d.per_wave = (d.slices + d.parts - 1) / d.parts;
    d.units = (a.outs + (GLU ? 15 : 31)) / (GLU ? 16 : 32);
    // about two workgroups a compute unit
    const int64_t turns = (d.units + d.subs - 1) / d.subs;
    int64_t strips = 2 * cus / gs_chunks(a);
    if (strips < 1) strips = 1;
    if (strips > turns) strips = turns;
    d.each = (int)((turns + strips - 1) / strips) * d.subs;
    d.strips = (d.units + d.each - 1) / d.each;
    const dim3 grid((unsigned)(most_tiles(a.q.slots, a.q.groups, 16) * d.strips)), b(kGsWaves * 64);
    if (d.per_wave == 1)
        hipLaunchKernelGGL((grouped_stream_kernel<true, GLU>), grid, b, 0, s, d);
    else
        hipLaunchKernelGGL((grouped_stream_kernel<false, GLU>), grid, b, 0, s, d);
    return launch_status();
}

// Estimated microseconds, of tiles that leave half of the card idle (0.6 a
// stage of 256 k and 4) and of this kernel (1.2 or, where the slots' operand
// comes with each, 2.7 a thousand items, and 5.5), with a margin.
bool grouped_stream_applies(const GgArgs &a, int64_t tiles, int cus) {
    if (2 * tiles > cus) return false;
    const double slices = (a.k + 511) / 512, items = (double)gs_chunks(a) * ((a.n + 31) / 32) * slices;
    return 1.15 * (5.5 + items * (slices > kGsWaves ? 0.0027 : 0.0012)) < 4.0 + 0.6 * ((a.k + 255) / 256);
}

int grouped_stream(const GgArgs &a, int cus, hipStream_t s) {
    const GsArgs d = {a, 0, 0, 0, 0, 0, 0, 0};
    return a.outs != a.n ? launch_gs<true>(d, cus, s) : launch_gs<false>(d, cus, s);
}

}  // namespace bqm
