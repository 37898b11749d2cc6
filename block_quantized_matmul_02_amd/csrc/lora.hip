// Low-rank adapters beside a projection, for gfx950: row t of adapter e,
//
//   h[t] = A[e] x[t],   y[t] = res[t] + scale[e] * B[e] h[t]
//
// HBM-bound: the adapters in use, x, res and y each move once; the products
// are small.  Two launches, h (f32, in the order of the grouped rows) between
// them.  A workgroup takes 16 rows of one adapter.
//  * Every operand is exact on the bf16 matrix cores: an f32 is the sum of
//    three bf16 numbers (its significand cut into bytes), an fp16 of two, and
//    the products of the parts are exact, so only the f32 sums round.  x of
//    fp16 meets A in fp16 as it is.
//  * Shrink: the matrix cores' rows are ranks and their columns the rows of x,
//    so a lane ends with four consecutive ranks of a row; the waves share k
//    and meet in LDS, added in wave order.
//  * Expand: rows are output columns, so a lane ends with four consecutive
//    values of a row of y.
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
    float *h;    // [slots][rp]
    int k, n, r, rp;
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

constexpr int kLoraRows = 16;
constexpr int kShrinkWaves = 8;

template <bool XF32, bool F16>
__global__ __launch_bounds__(kShrinkWaves * 64) void lora_shrink_kernel(LoraArgs a) {
    __shared__ v4f red[kShrinkWaves][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const GroupTile t = find_group(a.q, kLoraRows, 1, blockIdx.x);
    if (t.group >= a.q.groups) return;
    const int pos = t.first + t.local * kLoraRows;
    const int rows = min(kLoraRows, t.rows - t.local * kLoraRows);
    // a row past the last repeats it, an entry outside the rows reads row 0
    const unsigned row = (unsigned)a.q.order[pos + min(r16, rows - 1)];
    const int64_t at = (int64_t)(row < (unsigned)a.q.slots ? row : 0) * a.ldx;
    const int rank = min((int)blockIdx.y * 16 + r16, a.r - 1);
    const uint16_t *const pa = static_cast<const uint16_t *>(a.a) + ((int64_t)t.group * a.r + rank) * a.k;
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int k0 = wave * 32; k0 < a.k; k0 += kShrinkWaves * 32) {
        const int k = k0 + 8 * g4;
        const bool in = k < a.k;   // all eight: k % 8 == 0
        const u32x4 zero = {0, 0, 0, 0};
        u32x4 ra = zero;
        if (in) ra = *reinterpret_cast<const u32x4 *>(pa + k);
        if constexpr (XF32) {
            v4f lo = {0.0f, 0.0f, 0.0f, 0.0f}, hi = lo;
            if (in) {
                lo = *reinterpret_cast<const v4f *>(static_cast<const float *>(a.x) + at + k);
                hi = *reinterpret_cast<const v4f *>(static_cast<const float *>(a.x) + at + k + 4);
            }
            const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            u32x4 px[3];
            cut<3>(v, px);
            const AbParts<F16> parts(ra);
            acc = mfma_parts(parts.p, px, acc);
        } else {
            u32x4 rx = zero;
            if (in) rx = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.x) + at + k);
            if constexpr (F16)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, ra), __builtin_bit_cast(v8h, rx), acc, 0, 0, 0);
            else
                acc = mfma_bf16(ra, rx, acc);
        }
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int w = 1; w < kShrinkWaves; w++) acc += red[w][lane];
        // lane: row r16, ranks 4 g4 .. + 3
        const int r0 = (int)blockIdx.y * 16 + 4 * g4;
        if (r16 < rows) *reinterpret_cast<v4f *>(a.h + (int64_t)(pos + r16) * a.rp + r0) = acc;
    }
}

constexpr int kExpandWaves = 4;
constexpr int kExpandTiles = 4;                                       // of 16 columns, a wave
constexpr int kExpandStrip = kExpandWaves * kExpandTiles * 16;

// S: steps of 32 ranks.
template <int S, bool F16>
__global__ __launch_bounds__(kExpandWaves * 64) void lora_expand_kernel(LoraArgs a) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g4 = lane >> 4;
    const GroupTile t = find_group(a.q, kLoraRows, 1, blockIdx.y);
    if (t.group > a.q.groups) return;
    const int pos = t.first + t.local * kLoraRows;
    const int rows = min(kLoraRows, t.rows - t.local * kLoraRows);
    const unsigned row = (unsigned)a.q.order[pos + min(r16, rows - 1)];
    const bool live = r16 < rows && row < (unsigned)a.q.slots;
    const float *const res = a.res ? a.res + (int64_t)row * a.ldr : nullptr;
    float *const y = a.y + (int64_t)row * a.ldy;
    // four values of this lane's row, added to res and stored
    auto finish = [&](int col, v4f v) {
        if (!live || col >= a.n) return;
        if (col + 4 <= a.n) {
            if (res) v += *reinterpret_cast<const v4fu *>(res + col);
            *reinterpret_cast<v4fu *>(y + col) = v;
        } else {
            for (int i = 0; col + i < a.n; i++) y[col + i] = res ? v[i] + res[col + i] : v[i];
        }
    };
    const int strip = (int)blockIdx.x * kExpandStrip;
    if (t.group == a.q.groups) {   // no adapter
        if (a.res == a.y) return;
        for (int i = 0; i < kExpandTiles; i++) finish(strip + (i * kExpandWaves + wave) * 16 + 4 * g4, v4f{0.0f, 0.0f, 0.0f, 0.0f});
        return;
    }
    // this lane's row of h: ranks 32 s + 8 g4 .. + 7
    u32x4 ph[S][3];
    const float *const h = a.h + (int64_t)(pos + min(r16, rows - 1)) * a.rp;
#pragma unroll
    for (int s = 0; s < S; s++) {
        const int r0 = 32 * s + 8 * g4;
        float v[8] = {};
        if (r0 < a.r) {
            const v4f lo = *reinterpret_cast<const v4f *>(h + r0), hi = *reinterpret_cast<const v4f *>(h + r0 + 4);
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = lo[e], v[4 + e] = hi[e];
        }
        cut<3>(v, ph[s]);
    }
    const float scale = a.scale ? a.scale[t.group] : 1.0f;
#pragma unroll
    for (int i = 0; i < kExpandTiles; i++) {
        const int col0 = strip + (i * kExpandWaves + wave) * 16;
        if (col0 >= a.n) break;
        const uint16_t *const pb = static_cast<const uint16_t *>(a.b) + ((int64_t)t.group * a.n + min(col0 + r16, a.n - 1)) * a.r;
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < S; s++) {
            const int r0 = 32 * s + 8 * g4;
            u32x4 rb = {0, 0, 0, 0};
            if (r0 < a.r) rb = *reinterpret_cast<const u32x4 *>(pb + r0);
            const AbParts<F16> parts(rb);
            acc = mfma_parts(parts.p, ph[s], acc);
        }
        // lane: row r16, columns 4 g4 .. + 3
        finish(col0 + 4 * g4, acc * scale);
    }
}

template <bool F16>
static void launch_expand(const LoraArgs &a, dim3 grid, hipStream_t s) {
    const dim3 b(kExpandWaves * 64);
    if (a.r <= 32)
        hipLaunchKernelGGL((lora_expand_kernel<1, F16>), grid, b, 0, s, a);
    else if (a.r <= 64)
        hipLaunchKernelGGL((lora_expand_kernel<2, F16>), grid, b, 0, s, a);
    else if (a.r <= 128)
        hipLaunchKernelGGL((lora_expand_kernel<4, F16>), grid, b, 0, s, a);
    else
        hipLaunchKernelGGL((lora_expand_kernel<8, F16>), grid, b, 0, s, a);
}

}  // namespace bqm

extern "C" int64_t bqm_lora_add_workspace(int m, int r) {
    if (m < 1 || r < 1 || r > BQM_LORA_MAX_RANK) return -1;
    return (int64_t)m * ((r + 15) / 16 * 16) * 4;
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
    const int64_t tiles = most_tiles(m, adapters, kLoraRows);
    const int strips = (int)(((int64_t)n + kExpandStrip - 1) / kExpandStrip);
    if (tiles * strips * 256 > 0x7FFFFFFFll || tiles > 65535) return BQM_EUNSUPPORTED;   // what a dispatch counts
    LoraArgs q = {{offsets, order, adapters, m}, x, ldx, a, b, scale, res, ldr, y, ldy, static_cast<float *>(workspace),
                  k, n, r, (r + 15) / 16 * 16};
    hipStream_t s = as_stream(stream);
    const dim3 gs((unsigned)tiles, (unsigned)(q.rp / 16)), bs(kShrinkWaves * 64);
    const bool f16 = ab_type == BQM_F16;
    if (x_type == BQM_F32 && f16)
        hipLaunchKernelGGL((lora_shrink_kernel<true, true>), gs, bs, 0, s, q);
    else if (x_type == BQM_F32)
        hipLaunchKernelGGL((lora_shrink_kernel<true, false>), gs, bs, 0, s, q);
    else if (f16)
        hipLaunchKernelGGL((lora_shrink_kernel<false, true>), gs, bs, 0, s, q);
    else
        hipLaunchKernelGGL((lora_shrink_kernel<false, false>), gs, bs, 0, s, q);
    const int rc = launch_status();
    if (rc) return rc;
    const dim3 ge((unsigned)strips, (unsigned)tiles);
    if (f16)
        launch_expand<true>(q, ge, s);
    else
        launch_expand<false>(q, ge, s);
    return launch_status();
}
