// Low-rank adapters beside a projection, for gfx950: row t of adapter e,
//
//   h[t] = A[e] x[t],   y[t] = res[t] + scale[e] * B[e] h[t]
//
// HBM-bound: the adapters in use, x, res and y each move once; the products
// are small.  Two launches, h (f32, in the order of the grouped rows) between
// them.
//  * Every operand is exact on the bf16 matrix cores: an f32 is the sum of
//    three bf16 numbers (its significand cut into bytes), an fp16 of two, and
//    the products of the parts are exact, so only the f32 sums round.  x of
//    fp16 meets A in fp16 as it is.
//  * Shrink: the matrix cores' rows are ranks and their columns the rows of x,
//    so a lane ends with four consecutive ranks of a row.  A workgroup takes 16
//    rows of one adapter, or 64 of adapters with many, and a part of k, which
//    its waves share: one compute unit would draw a whole adapter too slowly
//    (one row, 4096 x 16: 7.5 us, and 3.9 with k in eight parts).  The parts'
//    results meet where h is read, added in order.
//  * Expand: rows are output columns, so a lane ends with four consecutive
//    values of a row of y; two tiles of 16 columns at a time, so that the lines
//    of res and y are used whole while they are near (4099 x 64 x 5152 62 us
//    with one, 50 with two).  Runs of 256 bytes a row through LDS were slower
//    (56), as were 64 rows a workgroup (55) and accesses past the caches (63).
//
// In a graph: 1 x 4096 x 16 x 4096 6.9 us, 64 rows of 40 adapters, 4096 x 16 x
// 20480 14.7 us (36 MB; 7.2 at 5.1 TB/s; some 1300 workgroups of the expand,
// each of 24 KB behind offsets, order, h and a barrier), 4099 rows of 6, 4096 x
// 64 x 5152 in fp16 16 + 54 us (33.6 and 169 MB; 40 in all), of f32 rows and
// bf16 adapters 25 + 52 (67 and 169 MB; 47).
#include "groups.h"

namespace bqm {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4fu __attribute__((ext_vector_type(4), aligned(4)));

struct LoraArgs {
    Grouping q;
    const void *x;
    int64_t ldx;
    const void *a, *b;
    const float *scale, *res;
    int64_t ldr;
    float *y;
    int64_t ldy;
    float *h;    // [splits][slots][rp]
    int k, n, r, rp;
    int splits, range;   // of k, and the k of each
};

// The bf16 parts of eight f32 values, by cutting: each part is the upper half
// of what the earlier ones left.
template <int P>
__device__ __forceinline__ void cut(const float (&v)[8], u32x4 (&p)[P]) {
    unsigned h[P][8];
#pragma unroll
    for (int e = 0; e < 8; e++) {
        float left = v[e];
#pragma unroll
        for (int i = 0; i < P; i++) {
            h[i][e] = __builtin_bit_cast(unsigned, left);
            left -= __builtin_bit_cast(float, h[i][e] & 0xFFFF0000u);
        }
    }
#pragma unroll
    for (int i = 0; i < P; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) p[i][e] = (h[i][2 * e] >> 16) | (h[i][2 * e + 1] & 0xFFFF0000u);
}

// Eight values of an adapter as bf16 parts: itself, or the two of an fp16.
template <bool F16>
struct AbParts {
    static constexpr int kParts = F16 ? 2 : 1;
    u32x4 p[kParts];
    __device__ __forceinline__ explicit AbParts(u32x4 raw) {
        if constexpr (F16) {
            const v8h f = __builtin_bit_cast(v8h, raw);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = (float)f[e];
            cut<2>(v, p);
        } else {
            p[0] = raw;
        }
    }
};

__device__ __forceinline__ v4f mfma_bf16(u32x4 a, u32x4 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// a += A operand . B operand over all pairs of parts, the smallest products first.
template <int PA, int PB>
__device__ __forceinline__ v4f mfma_parts(const u32x4 (&a)[PA], const u32x4 (&b)[PB], v4f c) {
#pragma unroll
    for (int i = PA - 1; i >= 0; i--)
#pragma unroll
        for (int j = PB - 1; j >= 0; j--) c = mfma_bf16(a[i], b[j], c);
    return c;
}

// RT: tiles of 16 ranks of a workgroup; G: its groups of 16 rows; W: waves,
// which share its range of k.
template <bool XF32, bool F16, int RT, int G, int W>
__global__ __launch_bounds__(W * 64) void lora_shrink_kernel(LoraArgs a) {
    constexpr int U = G > 1 ? (XF32 ? 1 : 2) : XF32 && RT > 1 ? 2 : 4;   // steps whose loads are on their way together
    __shared__ v4f red[RT][W][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const GroupTile t = find_group(a.q, 16 * G, 1, blockIdx.x);
    if (t.group >= a.q.groups) return;
    const int pos = t.first + t.local * 16 * G;
    const int rows = min(16 * G, t.rows - t.local * 16 * G);
    // a row past the last repeats it, an entry outside the rows reads row 0
    int64_t at[G];
#pragma unroll
    for (int g = 0; g < G; g++) {
        const unsigned row = (unsigned)a.q.order[pos + min(16 * g + r16, rows - 1)];
        at[g] = (int64_t)(row < (unsigned)a.q.slots ? row : 0) * a.ldx;
    }
    const int split = (int)blockIdx.y % a.splits, rank0 = (int)blockIdx.y / a.splits * 16 * RT;
    const int end = min(a.k, (split + 1) * a.range);
    // ranks past the last and k past the end are zeros
    const __amdgpu_buffer_rsrc_t ra = mx_rsrc(static_cast<const uint16_t *>(a.a) + (int64_t)t.group * a.r * a.k, 2ll * a.r * a.k);
    struct Step {
        u32x4 a[RT], x[G][XF32 ? 2 : 1];
    };
    auto load_a = [&](Step &s, int k0) {
        const int k = k0 + 8 * g4;   // eight values are in or out together: k % 8 == 0
        const uint32_t off = k < end ? (uint32_t)(((rank0 + r16) * (int64_t)a.k + k) * 2) : 0x80000000u;
#pragma unroll
        for (int i = 0; i < RT; i++)
            s.a[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, off + (uint32_t)(32 * i * a.k), 0, 0));
    };
    // past the end the row's last values, which meet zeros
    auto load_x = [&](Step &s, int k0) {
        const int k = min(k0 + 8 * g4, a.k - 8);
#pragma unroll
        for (int g = 0; g < G; g++) {
            if constexpr (XF32) {
                s.x[g][0] = *reinterpret_cast<const u32x4 *>(static_cast<const float *>(a.x) + at[g] + k);
                s.x[g][1] = *reinterpret_cast<const u32x4 *>(static_cast<const float *>(a.x) + at[g] + k + 4);
            } else {
                s.x[g][0] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.x) + at[g] + k);
            }
        }
    };
    v4f acc[G][RT] = {};
    auto multiply = [&](const Step &s) {
        if constexpr (XF32) {
            u32x4 px[G][3];
#pragma unroll
            for (int g = 0; g < G; g++) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const unsigned u = s.x[g][e >> 2][e & 3];
                    v[e] = __builtin_bit_cast(float, u);
                }
                cut<3>(v, px[g]);
            }
#pragma unroll
            for (int i = 0; i < RT; i++) {
                const AbParts<F16> parts(s.a[i]);
#pragma unroll
                for (int g = 0; g < G; g++) acc[g][i] = mfma_parts(parts.p, px[g], acc[g][i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < RT; i++)
#pragma unroll
                for (int g = 0; g < G; g++) {
                    if constexpr (F16)
                        acc[g][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, s.a[i]), __builtin_bit_cast(v8h, s.x[g][0]), acc[g][i], 0, 0, 0);
                    else
                        acc[g][i] = mfma_bf16(s.a[i], s.x[g][0], acc[g][i]);
                }
        }
    };
    // a wave takes U steps of 32 k at a time, whole lines of its rows
    for (int k0 = split * a.range + wave * (32 * U); k0 < end; k0 += W * 32 * U) {
        Step s[U];
#pragma unroll
        for (int u = 0; u < U; u++) load_a(s[u], k0 + 32 * u);
#pragma unroll
        for (int u = 0; u < U; u++) load_x(s[u], k0 + 32 * u);
        // left alone, the compiler keeps two to four loads on their way, to save registers
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; u++) multiply(s[u]);
    }
#pragma unroll
    for (int g = 0; g < G; g++) {
        if (16 * g >= rows) break;
        if (g > 0) __syncthreads();
#pragma unroll
        for (int i = 0; i < RT; i++) red[i][wave][lane] = acc[g][i];
        __syncthreads();
        for (int i = wave; i < RT; i += W) {
            v4f sum = red[i][0][lane];
#pragma unroll
            for (int w = 1; w < W; w++) sum += red[i][w][lane];
            // lane: row r16, ranks 4 g4 .. + 3
            const int r0 = rank0 + 16 * i + 4 * g4;
            if (16 * g + r16 < rows && r0 < a.rp)
                *reinterpret_cast<v4f *>(a.h + ((int64_t)split * a.q.slots + pos + 16 * g + r16) * a.rp + r0) = sum;
        }
    }
}

constexpr int kExpandWaves = 8;
constexpr int kExpandTiles = 4;                                       // of 16 columns, a wave
constexpr int kExpandStrip = kExpandWaves * kExpandTiles * 16;

// S: steps of 32 ranks; G: groups of 16 rows, which share an adapter's operand.
template <int S, int G, bool F16>
__global__ __launch_bounds__(kExpandWaves * 64, S == 8 ? 2 : 4) void lora_expand_kernel(LoraArgs a) {
    __shared__ u32x4 hp[G * S][3][64];   // the parts of h, as the matrix cores take them
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const GroupTile t = find_group(a.q, 16 * G, 1, blockIdx.y);
    if (t.group > a.q.groups) return;
    const bool none = t.group == a.q.groups;   // no adapter
    if (none && a.res == a.y) return;
    const int pos = t.first + t.local * 16 * G;
    const int rows = min(16 * G, t.rows - t.local * 16 * G);
    const int strip = (int)blockIdx.x * kExpandStrip + wave * kExpandTiles * 16;
    // columns past the last and ranks past the rank are zeros
    const __amdgpu_buffer_rsrc_t rb = mx_rsrc(static_cast<const uint16_t *>(a.b) + ((int64_t)t.group * a.n + strip) * a.r,
                                              none ? 0 : 2 * min((int64_t)kExpandTiles * 16, (int64_t)a.n - strip) * a.r);
    auto load_b = [&](u32x4 (&v)[S], int i) {
#pragma unroll
        for (int s = 0; s < S; s++)
            v[s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       rb, 32 * s + 8 * g4 < a.r ? (uint32_t)(((16 * i + r16) * a.r + 32 * s + 8 * g4) * 2) : 0x80000000u, 0, 0));
    };
    u32x4 b[2][S];
    load_b(b[0], 0);
    load_b(b[1], 1);
    unsigned row[G];   // of y; ~0: none
#pragma unroll
    for (int g = 0; g < G; g++) {
        row[g] = 16 * g + r16 < rows ? (unsigned)a.q.order[pos + 16 * g + r16] : ~0u;
        if (row[g] >= (unsigned)a.q.slots) row[g] = ~0u;
    }
    v4f old[G][2];
    auto load_res = [&](int i) {
        const int col = strip + 16 * i + 4 * g4;   // lane: row r16, columns col .. + 3, and 16 on
#pragma unroll
        for (int g = 0; g < G; g++)
#pragma unroll
            for (int c = 0; c < 2; c++) {
                old[g][c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
                if (!a.res || row[g] == ~0u) continue;
                const float *const res = a.res + (int64_t)row[g] * a.ldr + col + 16 * c;
                if (col + 16 * c + 4 <= a.n) {
                    old[g][c] = *reinterpret_cast<const v4fu *>(res);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (col + 16 * c + e < a.n) old[g][c][e] = res[e];
                }
            }
    };
    load_res(0);
    __builtin_amdgcn_sched_barrier(0);
    if (!none) {
        // a value a thread and piece (16 rows, 32 ranks): the sum of its parts of k, cut in three
        const int hr = tid >> 5, rank = tid & 31;
        auto stage = [&](auto splits) {
            constexpr int N = decltype(splits)::value;
#pragma unroll
            for (int p = 0; p < G * S; p++) {
                const int g = p / S, r0 = 32 * (p % S) + rank;
                const bool in = r0 < a.r && 16 * g + hr < rows;
                const float *const h = a.h + (int64_t)(pos + (in ? 16 * g + hr : 0)) * a.rp + (in ? r0 : 0);
                float part[N];
#pragma unroll
                for (int q = 0; q < N; q++) part[q] = h[(int64_t)q * a.q.slots * a.rp];
                float left = part[0];
#pragma unroll
                for (int q = 1; q < N; q++) left += part[q];
                if (!in) left = 0.0f;
#pragma unroll
                for (int i = 0; i < 3; i++) {
                    const unsigned u = __builtin_bit_cast(unsigned, left);
                    reinterpret_cast<uint16_t *>(&hp[p][i][(rank >> 3) * 16 + hr])[rank & 7] = (uint16_t)(u >> 16);
                    left -= __builtin_bit_cast(float, u & 0xFFFF0000u);
                }
            }
        };
        if (a.splits == 8)
            stage(std::integral_constant<int, 8>{});
        else if (a.splits == 4)
            stage(std::integral_constant<int, 4>{});
        else if (a.splits == 2)
            stage(std::integral_constant<int, 2>{});
        else
            stage(std::integral_constant<int, 1>{});
    }
    const float scale = none || !a.scale ? 1.0f : a.scale[t.group];
    __syncthreads();
    // two tiles of columns at a time, so that whole lines of res and y are in use together
#pragma unroll
    for (int i = 0; i < kExpandTiles; i += 2) {
        const int col = strip + 16 * i + 4 * g4;   // lane: row r16, columns col .. + 3, and 16 on
        if (i > 0) load_res(i);
        v4f acc[G][2] = {};
        if (!none) {
#pragma unroll
            for (int s = 0; s < S; s++) {
                const AbParts<F16> p0(b[0][s]), p1(b[1][s]);
#pragma unroll
                for (int g = 0; g < G; g++) {
                    const u32x4 ph[3] = {hp[g * S + s][0][lane], hp[g * S + s][1][lane], hp[g * S + s][2][lane]};
                    acc[g][0] = mfma_parts(p0.p, ph, acc[g][0]);
                    acc[g][1] = mfma_parts(p1.p, ph, acc[g][1]);
                }
            }
        }
        if (i + 2 < kExpandTiles) {
            load_b(b[0], i + 2);
            load_b(b[1], i + 3);
        }
#pragma unroll
        for (int g = 0; g < G; g++) {
            if (row[g] == ~0u) continue;
#pragma unroll
            for (int c = 0; c < 2; c++) {
                const v4f v = acc[g][c] * scale + old[g][c];
                float *const y = a.y + (int64_t)row[g] * a.ldy + col + 16 * c;
                if (col + 16 * c + 4 <= a.n) {
                    *reinterpret_cast<v4fu *>(y) = v;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (col + 16 * c + e < a.n) y[e] = v[e];
                }
            }
        }
    }
}

template <int S, int G>
static int launch_expand(const LoraArgs &a, bool f16, hipStream_t s) {
    const int64_t tiles = most_tiles(a.q.slots, a.q.groups, 16 * G);
    const dim3 grid((unsigned)((a.n + (int64_t)kExpandStrip - 1) / kExpandStrip), (unsigned)tiles), b(kExpandWaves * 64);
    if (f16)
        hipLaunchKernelGGL((lora_expand_kernel<S, G, true>), grid, b, 0, s, a);
    else
        hipLaunchKernelGGL((lora_expand_kernel<S, G, false>), grid, b, 0, s, a);
    return launch_status();
}

template <int RT, int G, int W>
static int launch_shrink(const LoraArgs &a, bool xf32, bool f16, hipStream_t s) {
    const dim3 grid((unsigned)most_tiles(a.q.slots, a.q.groups, 16 * G), (unsigned)((a.rp + 16 * RT - 1) / (16 * RT) * a.splits)), b(W * 64);
    if (xf32 && f16)
        hipLaunchKernelGGL((lora_shrink_kernel<true, true, RT, G, W>), grid, b, 0, s, a);
    else if (xf32)
        hipLaunchKernelGGL((lora_shrink_kernel<true, false, RT, G, W>), grid, b, 0, s, a);
    else if (f16)
        hipLaunchKernelGGL((lora_shrink_kernel<false, true, RT, G, W>), grid, b, 0, s, a);
    else
        hipLaunchKernelGGL((lora_shrink_kernel<false, false, RT, G, W>), grid, b, 0, s, a);
    return launch_status();
}

// Groups of 16 rows of a workgroup, and parts of k that have workgroups of
// their own and results of their own in the workspace: adapters of many rows
// are read once for 64 of them, and few workgroups share k.
static int lora_group(int m, int adapters) { return m >= 1024 && m >= 64 * (int64_t)adapters ? 4 : 1; }

static int lora_splits(int m, int group) {
    const int tiles = (m - 1) / (16 * group) + 1;
    return tiles <= 48 ? 8 : tiles <= 96 ? 4 : tiles <= 192 ? 2 : 1;
}

}  // namespace bqm

extern "C" int64_t bqm_lora_add_workspace(int m, int r) {
    if (m < 1 || r < 1 || r > BQM_LORA_MAX_RANK) return -1;
    // with the groups that some number of adapters leads to
    return (int64_t)bqm::lora_splits(m, m >= 1024 ? 4 : 1) * m * ((r + 15) / 16 * 16) * 4;
}

extern "C" int bqm_lora_add(const void *x, int64_t ldx, int x_type, const void *a, const void *b, int ab_type,
                            const float *scale, const int *offsets, const int *order, const float *res, int64_t ldr,
                            float *y, int64_t ldy, void *workspace, int m, int k, int n, int r, int adapters,
                            void *stream) {
    using namespace bqm;
    if (!x || !a || !b || !offsets || !order || !y || !workspace || !type_known(x_type) || !type_known(ab_type)) return BQM_EINVAL;
    if (m < 1 || k < 1 || n < 1 || r < 1 || r > BQM_LORA_MAX_RANK || adapters < 1 || adapters > BQM_MAX_GROUPS) return BQM_EINVAL;
    if (ab_type == BQM_F32 || (x_type != BQM_F32 && x_type != ab_type) || k % 8 != 0 || r % 8 != 0) return BQM_EUNSUPPORTED;
    if (m == 1) ldx = k, ldr = ldy = n;
    if (ldx < k || (res && ldr < n) || ldy < n) return BQM_EUNSUPPORTED;
    if (!aligned(x, 16) || ldx * type_bytes(x_type) % 16 != 0 || !aligned(a, 16) || !aligned(b, 16) || !aligned(workspace, 16)) return BQM_EUNSUPPORTED;
    if (!aligned(scale, 4) || !aligned(offsets, 4) || !aligned(order, 4) || !aligned(res, 4) || !aligned(y, 4)) return BQM_EUNSUPPORTED;
    if (res == y && ldr != ldy) return BQM_EUNSUPPORTED;
    const int group = lora_group(m, adapters);
    // The expand's grid, of tiles in y, in what a dispatch counts, and an adapter
    // in 31 bits.  The shrink's is smaller: 16 parts of the ranks times 8 of k
    // are for few rows, and many rows have one part of k.
    const int64_t tiles = most_tiles(m, adapters, group > 1 ? 32 : 16), strips = ((int64_t)n + kExpandStrip - 1) / kExpandStrip;
    if (tiles > 65535 || tiles * strips * 512 > 0x7FFFFFFFll || k > 1 << 21) return BQM_EUNSUPPORTED;
    LoraArgs q = {{offsets, order, adapters, m}, x, ldx, a, b, scale, res, ldr, y, ldy, static_cast<float *>(workspace),
                  k, n, r, (r + 15) / 16 * 16, lora_splits(m, group), 0};
    q.range = (((k + q.splits - 1) / q.splits) + 127) / 128 * 128;
    hipStream_t s = as_stream(stream);
    const bool xf32 = x_type == BQM_F32, f16 = ab_type == BQM_F16;
    // few rows: a workgroup for every 16 ranks
    const int rc = group == 1 ? launch_shrink<1, 1, 4>(q, xf32, f16, s)
                   : r <= 16  ? launch_shrink<1, 4, 8>(q, xf32, f16, s)
                              : launch_shrink<4, 4, 8>(q, xf32, f16, s);
    if (rc) return rc;
    if (r <= 32) return group > 1 ? launch_expand<1, 2>(q, f16, s) : launch_expand<1, 1>(q, f16, s);
    if (r <= 64) return group > 1 ? launch_expand<2, 2>(q, f16, s) : launch_expand<2, 1>(q, f16, s);
    if (r <= 128) return group > 1 ? launch_expand<4, 2>(q, f16, s) : launch_expand<4, 1>(q, f16, s);
    return group > 1 ? launch_expand<8, 2>(q, f16, s) : launch_expand<8, 1>(q, f16, s);
}
