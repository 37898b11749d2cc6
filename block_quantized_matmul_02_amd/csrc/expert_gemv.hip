// MXFP4 products of few slots with their experts' weights for gfx950: a decode
// or verify step of a sparse layer, f32 activations.
//
//   p[s][r] = sum_b 2^(ws - 127) sum_{i in b} x[s][i] e2m1(w[ids[s]][r][i])
//   y = p, or with the gate silu(p[s][j]) p[s][n/2 + j]
//
// HBM-bound: the chosen experts' weights, 17/32 byte each, are read once for
// up to T slots of an expert.  As in the decode GEMV an f32 is cut into three
// bf16 parts, exactly, which are three rows of the 16-row operand; five slots
// fit.
//  * A workgroup takes a strip of units of 32 weight rows (with the gate: 16
//    of each half) of one expert for up to T slots.  It finds them itself: a
//    slot's workgroup looks at all ids, and works if its slot is the first,
//    or the (T i)-th, of those with its id.
//  * The slots' rows are cut into LDS once.  A wave goes through a unit's k in
//    slices of 512 by itself, without a barrier; where there are few units,
//    several waves share its slices and their sums meet in LDS, added in wave
//    order.  Weights stream a slice of both tiles ahead and pass through a
//    wave's own LDS tile, 256 contiguous bytes a row from memory.
//  * Two workgroups of eight waves a compute unit, where their operands fit:
//    one starts (ids, x) while the other streams.  One a compute unit, with two
//    slices ahead, took 54 us instead of 35 at 54 slots of 64 experts, 1408 x
//    4096.
//
// In a graph: 8 slots of 64 experts, 4096 x 2816 with the gate, 15.4 us (49 MB:
// 9.6 at 5.1 TB/s; 176 workgroups, and ids, x and the first weights are three
// trips to memory that follow each other), 54 slots of 35 distinct of 64, 1408
// x 4096, 32.4 us (20.7; two units a wave), 48 of 32 distinct of 60, 5120 x
// 3328 with the gate, 85 us (57; two slots' operand is 113 KB of LDS, one
// workgroup a compute unit).
#include "groups.h"

namespace bqm {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kEvWaves = 8;
constexpr int kEvSlice = 512;
constexpr int kEvBlocks = kEvSlice / 32;
constexpr int kEvTileStride = kEvSlice / 2 + 16;
constexpr int kEvTileBytes = 16 * kEvTileStride;
constexpr int kEvSlots = 5;             // of a workgroup, at most
constexpr int kEvPlace = 32;            // bytes of the list of slots
constexpr int kEvLds = 160 * 1024;

struct EvArgs {
    const uint8_t *w, *ws;
    const float *x;
    const int *ids;
    float *y;
    int top;        // slots per row of x
    int slots, groups, k, n;
    int glu;
    int slices, parts, subs, per_wave;
    int take;       // T
    int each;       // units of a workgroup
};

// The three bf16 parts of eight f32 values.
__device__ __forceinline__ void ev_parts(const u32x4 (&v)[2], u32x4 (&p)[3]) {
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

template <int SEL>
__device__ __forceinline__ v2bf ev_two(unsigned q, float s) { return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, SEL); }

__device__ __forceinline__ v8bf ev_eight(unsigned q, float s) {
    const v2bf a = ev_two<0>(q, s), b = ev_two<1>(q, s), c = ev_two<2>(q, s), d = ev_two<3>(q, s);
    return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// WIDE: scale rows are whole, aligned dwords (k % 128 == 0); else bytes.
template <bool WIDE>
__global__ __launch_bounds__(kEvWaves * 64, 4) void expert_gemv_kernel(EvArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    int *const place = reinterpret_cast<int *>(lds);   // the slots that this workgroup takes
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const int slot0 = blockIdx.y;
    const int outs = a.glu ? a.n / 2 : a.n;
    const int per_unit = a.glu ? 16 : 32;                   // outputs of a unit
    const int units = (outs - 1) / per_unit + 1;            // n may be the most that 31 bits hold
    const int unit0 = blockIdx.x * a.each, unit1 = min(unit0 + a.each, units);
    if (unit0 >= unit1) return;

    // the slots with this slot's expert
    int all[BQM_EXPERT_GEMV_MAX_SLOTS / 64], expert = 0;
#pragma unroll
    for (int j = 0; j < BQM_EXPERT_GEMV_MAX_SLOTS / 64; j++) all[j] = 64 * j < a.slots ? a.ids[min(64 * j + lane, a.slots - 1)] : 0;
#pragma unroll
    for (int j = 0; j < BQM_EXPERT_GEMV_MAX_SLOTS / 64; j++)
        if (slot0 >> 6 == j) expert = __builtin_amdgcn_readlane(all[j], slot0 & 63);
    if ((unsigned)expert >= (unsigned)a.groups) {
        const int lo = unit0 * per_unit;
        const unsigned cols = (unsigned)min((int64_t)(unit1 - unit0) * per_unit, (int64_t)outs - lo);
        for (unsigned i = tid; i < cols; i += blockDim.x) a.y[(int64_t)slot0 * outs + lo + i] = 0.0f;
        return;
    }
    int count = 0, before = 0;
#pragma unroll
    for (int j = 0; j < BQM_EXPERT_GEMV_MAX_SLOTS / 64; j++) {
        const int s = 64 * j + lane;
        uint64_t same = __ballot(s < a.slots && all[j] == expert);
        const int up = slot0 - 64 * j;   // lanes below it are earlier slots
        const uint64_t earlier = up <= 0 ? 0 : up >= 64 ? ~(uint64_t)0 : ((uint64_t)1 << up) - 1;
        before += __builtin_popcountll(same & earlier);
        same &= ~earlier;
        while (same != 0 && count < a.take) {
            if (tid == 0) place[count] = 64 * j + __builtin_ctzll(same);
            count++;
            same &= same - 1;
        }
    }
    if (before % a.take != 0) return;
    __syncthreads();

    const int nblk = a.k / 32;
    const int64_t row_bytes = a.k / 2;
    const int xstride = a.slices * kEvSlice * 2 + 16;
    const int waves = a.parts * a.subs;
    uint8_t *const xs = lds + kEvPlace;
    uint8_t *const tile = xs + 3 * a.take * xstride + wave * kEvTileBytes;
    float2 *const red = reinterpret_cast<float2 *>(xs + 3 * a.take * xstride + waves * kEvTileBytes);   // [2][waves][2][64]
    const int sub = wave / a.parts, wpart = wave % a.parts;
    const uint8_t *const w = a.w + (int64_t)expert * a.n * row_bytes;
    const uint8_t *const ws = a.ws + (int64_t)expert * a.n * nblk;

    // item: slice wpart + parts * s of unit u; its two tiles of 16 rows
    struct Tile {
        u32x4 c[4];
        unsigned s;
    };
    int next_unit = unit0 + sub, next_s = 0;
    auto load = [&](Tile (&q)[2]) {
        const int blk0 = (wpart + a.parts * next_s) * kEvBlocks;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int j0 = (int)((unsigned)next_unit * per_unit) + (a.glu ? 0 : 16 * h);   // of units past the last, any
            const int64_t row0 = j0 + (a.glu ? (int64_t)h * outs : 0);
            const int rows = next_unit < unit1 ? min(outs - j0, 16) : 0;   // may be <= 0: nothing is read
            const __amdgpu_buffer_rsrc_t rw = mx_rsrc(w + row0 * row_bytes, rows * row_bytes);
            const __amdgpu_buffer_rsrc_t rs = mx_rsrc(ws + row0 * nblk, (int64_t)rows * nblk);
            const uint32_t off = blk0 + r16 < nblk ? (uint32_t)(g4 * row_bytes + 16 * (blk0 + r16)) : 0x80000000u;
#pragma unroll
            for (int i = 0; i < 4; i++)
                q[h].c[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, off + (uint32_t)(4 * i * row_bytes), 0, 0));
            const int b = blk0 + 4 * g4;
            if constexpr (WIDE) {
                q[h].s = __builtin_amdgcn_raw_buffer_load_b32(rs, b < nblk ? (uint32_t)(r16 * nblk + b) : 0x80000000u, 0, 0);
            } else {
                q[h].s = 0;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    q[h].s |= (unsigned)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                                  rs, b + e < nblk ? (uint32_t)(r16 * nblk + b + e) : 0x80000000u, 0, 0) << (8 * e);
            }
        }
        if (++next_s == a.per_wave) {
            next_s = 0;
            next_unit += a.subs;
        }
    };
    Tile it[2];
    load(it);

    // the slots' rows, eight values a thread and turn; zeros up to a whole slice
    const int per_row = a.slices * 64;
    for (int i = 0; i < count; i++) {
        const float *const x = a.x + (int64_t)(__builtin_amdgcn_readfirstlane(place[i]) / a.top) * a.k;
        for (int at = tid; at < per_row; at += blockDim.x) {
            u32x4 v[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}}, p[3];
            if (8 * at < a.k) {
                v[0] = *reinterpret_cast<const u32x4 *>(x + 8 * at);
                v[1] = *reinterpret_cast<const u32x4 *>(x + 8 * at + 4);
            }
            ev_parts(v, p);
#pragma unroll
            for (int h = 0; h < 3; h++) *reinterpret_cast<u32x4 *>(xs + (3 * i + h) * xstride + 16 * at) = p[h];
        }
    }
    __syncthreads();

    // this lane's operand row: part h of slots 0..3 has rows 4 i + h, of slot 4 rows 4 h + 3
    const int own = (r16 & 3) < 3 ? r16 >> 2 : 4, part = (r16 & 3) < 3 ? r16 & 3 : r16 >> 2;
    const bool used = own < count && r16 != 15;
    const uint8_t *const xrow = xs + (used ? 3 * own + part : 0) * xstride + 4 * g4 * 64;

    int s = 0, unit = unit0, set = 0;
    v4f acc[2] = {};
    auto item = [&](Tile (&q)[2]) {
        u32x4 c[2][4];
        unsigned sc[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                *reinterpret_cast<u32x4 *>(tile + (4 * i + g4) * kEvTileStride + 16 * r16) = q[h].c[i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int i = 0; i < 4; i++) c[h][i] = *reinterpret_cast<const u32x4 *>(tile + r16 * kEvTileStride + (4 * g4 + i) * 16);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            sc[h] = q[h].s;
        }
        load(q);
        const int slice = wpart + a.parts * s;
        const uint8_t *const xp = xrow + (slice < a.slices ? slice : 0) * (kEvSlice * 2);   // past the end: zero weights
#pragma unroll
        for (int qq = 0; qq < 4; qq++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                u32x4 xv = {0, 0, 0, 0};
                if (used && slice < a.slices) xv = *reinterpret_cast<const u32x4 *>(xp + qq * 64 + e * 16);
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float f = __builtin_bit_cast(float, ((sc[h] >> (8 * qq)) & 255u) << 23);
                    acc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, xv), ev_eight(c[h][qq][e], f), acc[h], 0, 0, 0);
                }
            }
        if (++s < a.per_wave) return;
        s = 0;
        // lane: weight row r16; its slot's sum, and a part of slot 4's, the smallest part first
        float mine_sum[2], fifth[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            mine_sum[h] = (acc[h][2] + acc[h][1]) + acc[h][0];
            fifth[h] = acc[h][3];
            acc[h] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
        if (a.parts == 1) {
            // the wave has its unit's sums: slot g4 of lanes r16, slot 4 of the first ones
            const int u = unit + sub;
            auto put = [&](int tok, float p0, float p1) {
                float *const to = a.y + (int64_t)place[tok] * outs;
                const int j = u * per_unit + r16;
                if (a.glu) {
                    if (j < outs) to[j] = silu(p0) * p1;
                } else {
                    if (j < outs) to[j] = p0;
                    if (j + 16 < outs) to[j + 16] = p1;
                }
            };
            if (u < unit1) {
                if (g4 < count) put(g4, mine_sum[0], mine_sum[1]);
                if (count > 4) {
                    float p[2];
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const float b = __shfl(fifth[h], r16 + 16), c = __shfl(fifth[h], r16 + 32);
                        p[h] = (c + b) + fifth[h];
                    }
                    if (g4 == 0) put(4, p[0], p[1]);
                }
            }
            unit += a.subs;
            return;
        }
        float2 *const out = red + set * (waves * 128);
#pragma unroll
        for (int h = 0; h < 2; h++) out[(wave * 2 + h) * 64 + lane] = make_float2(mine_sum[h], fifth[h]);
        __syncthreads();
        // an output a thread: slot, sub, column (of 32 weight rows, or 16 pairs)
        const int per = per_unit * count;
        for (int o = tid; o < per * a.subs; o += blockDim.x) {
            const int su = o / per, in = o - su * per, tok = in / per_unit, col = in - tok * per_unit;
            if (unit + su >= unit1) continue;
            const int j = (unit + su) * per_unit + col;
            if (j >= outs) continue;
            auto total = [&](int h, int c) {
                const float2 *const q0 = out + (su * a.parts * 2 + h) * 64;
                float sum = 0.0f;
                for (int p = 0; p < a.parts; p++) {
                    const float2 *const r = q0 + p * 128;
                    sum += tok < 4 ? r[16 * tok + c].x : (r[c + 32].y + r[c + 16].y) + r[c].y;
                }
                return sum;
            };
            float v;
            if (a.glu)
                v = silu(total(0, col)) * total(1, col);
            else
                v = total(col >> 4, col & 15);
            a.y[(int64_t)place[tok] * outs + j] = v;
        }
        unit += a.subs;
        set ^= 1;
    };
    const int rounds = (unit1 - unit0 + a.subs - 1) / a.subs * a.per_wave;   // the same for all waves, which meet
#pragma unroll 1
    for (int j = 0; j < rounds; j++) item(it);
}

static int64_t ev_lds(int take, int slices, int waves) {
    return kEvPlace + 3ll * take * (slices * kEvSlice * 2 + 16) + (int64_t)waves * (kEvTileBytes + 2 * 128 * (int)sizeof(float2));
}

}  // namespace bqm

extern "C" int bqm_mxfp4_expert_gemv(const uint8_t *w, const uint8_t *ws, const float *x, const int *ids, float *y,
                                     int glu, int rows, int slots, int groups, int k, int n, void *stream) {
    using namespace bqm;
    if (!w || !ws || !x || !ids || !y) return BQM_EINVAL;
    if (rows < 1 || slots < 1 || slots > BQM_EXPERT_GEMV_MAX_SLOTS || slots % rows != 0) return BQM_EINVAL;
    if (groups < 1 || groups > BQM_MAX_GROUPS || k < 32 || n < 1 || (glu && n % 2 != 0)) return BQM_EINVAL;
    if (k % 32 != 0 || k > BQM_EXPERT_GEMV_MAX_K) return BQM_EUNSUPPORTED;
    if (!aligned(w, 16) || !aligned(x, 16) || !aligned(ids, 4) || !aligned(y, 4)) return BQM_EUNSUPPORTED;
    const bool wide = k % 128 == 0 && aligned(ws, 4);
    static LaunchCache caches[2];
    const void *fn = wide ? reinterpret_cast<const void *>(&expert_gemv_kernel<true>) : reinterpret_cast<const void *>(&expert_gemv_kernel<false>);
    const int rc = raise_lds_limit(caches[wide], fn, kEvLds);
    if (rc) return rc;
    EvArgs a = {w, ws, x, ids, y, slots / rows, slots, groups, k, n, glu != 0, 0, 0, 0, 0, 0, 0};
    a.slices = (k + kEvSlice - 1) / kEvSlice;
    // As many distinct ids as slots choose by chance have work.
    const int per_unit = glu ? 16 : 32, cus = device_cus();
    const int units = ((glu ? n / 2 : n) - 1) / per_unit + 1;
    double distinct = slots;
    if (rows > 1) {
        double missed = 1.0;
        for (int i = 0; i < slots; i++) missed *= 1.0 - 1.0 / groups;
        distinct = groups * (1.0 - missed);
    }
    // Waves share k as far as there are fewer units than four a compute unit.
    // In a graph (us; one, two, four, eight waves a unit): 8 slots, 4096 x 2816
    // with the gate 22.2, 15.4 (taken), 16.2, 17.7; 4 of 4, 2048 x 1536 12.4,
    // 9.0, 7.4 (taken); 54 of 64, 1408 x 4096 32.9 (taken), 34.2, and 38.3 with
    // three; 48 of 60, 5120 x 3328 with the gate 83.8 (taken), 84.4, 91.9, 107.
    a.parts = 1;
    while (distinct * units * a.parts < 4.0 * cus && a.parts < kEvWaves && a.parts < a.slices) a.parts *= 2;
    if (a.parts > a.slices) a.parts = a.slices;
    a.subs = kEvWaves / a.parts;
    a.per_wave = (a.slices + a.parts - 1) / a.parts;
    const int waves = a.parts * a.subs;
    // Slots of an expert that a workgroup takes: about twice what an expert has
    // on average, since their operand costs LDS, and a second workgroup finds
    // the weights in the caches.
    a.take = rows == 1 ? 1 : 1 + 2 * slots / groups;   // one token's experts are different ones
    if (a.take > kEvSlots) a.take = kEvSlots;
    while (a.take > 1 && ev_lds(a.take, a.slices, waves) > kEvLds) a.take--;
    const int bytes = (int)ev_lds(a.take, a.slices, waves);
    // Units of a workgroup: one a wave (or group of waves), or as many more as
    // keep the workgroups that work to two a compute unit.
    const double most = 2.0 * cus / distinct;   // workgroups of an expert
    const int strips = most < 1.0 ? 1 : (int)most;
    const int rounds = (units + a.subs - 1) / a.subs;
    a.each = (rounds + strips - 1) / strips * a.subs;
    const dim3 grid((unsigned)((units + a.each - 1) / a.each), (unsigned)slots);
    hipStream_t s = as_stream(stream);
    if (wide)
        hipLaunchKernelGGL(expert_gemv_kernel<true>, grid, dim3(waves * 64), bytes, s, a);
    else
        hipLaunchKernelGGL(expert_gemv_kernel<false>, grid, dim3(waves * 64), bytes, s, a);
    return launch_status();
}
