// A router's choice of experts, and rows sorted by group, for gfx950.
//
//   ids[t] = the `top` largest logits' columns;  weights[t] = their softmax,
//   over all columns or over the chosen;
//   order = rows sorted by id, stable;  offsets = where each group begins.
//
// Both move a few bytes a row and are bound by latency.
//  * Choice: a wave a row, its logits in registers (column 64 j + lane); each
//    turn takes the wave's largest and, of equals, the first register with it
//    and there the first lane, which is the lowest column.
//  * Sort by counting: a workgroup counts 4096 rows, each wave its own 256 in
//    order, so that a row's place is (rows of lower groups) + (rows of its
//    group in earlier chunks, waves, batches and lanes): no atomics, the same
//    order every time.  Equal ids of a wave are found by a ballot for each bit
//    of the id.  More rows take two launches, the chunks' counts in between.
#include "groups.h"

namespace bqm {

__device__ __forceinline__ float wave_max(float v) {
    auto step = [&](auto ctrl) {
        const float o = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF, 0xF, false));
        v = fmaxf(v, o);
    };
    step(std::integral_constant<int, 0xB1>{});
    step(std::integral_constant<int, 0x4E>{});
    step(std::integral_constant<int, 0x141>{});
    step(std::integral_constant<int, 0x140>{});
    return swap32_max(swap16_max(v));
}

struct RouteArgs {
    const void *logits;
    int64_t ld;
    int *ids;
    float *weights;
    int type, top, renorm, m, e;
};

// J: registers of a lane, 64 J >= e.
template <int J>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.m) return;
    float v[J];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < J; j++) {
        const int c = 64 * j + lane;
        v[j] = c < a.e ? load_as(a.logits, t * a.ld + c, a.type) : -INFINITY;
        bad |= !(v[j] < INFINITY);   // NaN or +inf
        if (v[j] != v[j]) v[j] = -INFINITY;
    }
    const bool poison = __ballot(bad) != 0;
    float most = v[0];
#pragma unroll
    for (int j = 1; j < J; j++) most = fmaxf(most, v[j]);
    most = wave_max(most);
    float z = 0.0f;
    if (!a.renorm && most > -INFINITY) {
#pragma unroll
        for (int j = 0; j < J; j++) z += expf(v[j] - most);
        z = wave_sum(z);
    }
    // lane i keeps choice i
    int id = -1;
    float value = -INFINITY;
    for (int i = 0; i < a.top; i++) {
        float here = v[0];
#pragma unroll
        for (int j = 1; j < J; j++) here = fmaxf(here, v[j]);
        here = wave_max(here);
        if (here == -INFINITY) break;
        bool found = false;
#pragma unroll
        for (int j = 0; j < J; j++) {
            const uint64_t equal = __ballot(v[j] == here);
            if (!found && equal != 0) {
                found = true;
                const int at = __builtin_ctzll(equal);
                if (lane == at) v[j] = -INFINITY;
                if (lane == i) {
                    id = 64 * j + at;
                    value = here;
                }
            }
        }
    }
    float w = id >= 0 ? expf(value - most) : 0.0f;
    if (a.renorm) z = wave_sum(w);
    if (id >= 0) w = poison ? NAN : w / z;
    if (lane < a.top) {
        a.ids[t * a.top + lane] = id;
        a.weights[t * a.top + lane] = w;
    }
}

constexpr int kGrWaves = 16;
constexpr int kGrBatches = 4;                               // of 64 rows, a wave
constexpr int kGrChunk = kGrWaves * kGrBatches * 64;        // rows of a workgroup

struct GroupRowsArgs {
    const int *ids;
    int *offsets, *order, *counts;   // counts: [chunks][groups + 1]
    int count, groups, chunks, bits;
};

// MODE 0: all rows in one workgroup.  1: a chunk's counts.  2: a chunk's places.
template <int MODE>
__global__ __launch_bounds__(kGrWaves * 64) void group_rows_kernel(GroupRowsArgs a) {
    extern __shared__ int lds[];
    __shared__ int wave_total[kGrWaves];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int all = a.groups + 1;                 // the last one: rows of no group
    int *const hist = lds + wave * all;           // [waves][all]
    int *const base = lds + kGrWaves * all;       // [all]
    const int64_t row0 = (int64_t)blockIdx.x * kGrChunk + wave * (kGrBatches * 64) + lane;

    int id[kGrBatches];
    uint64_t same[kGrBatches];
#pragma unroll
    for (int b = 0; b < kGrBatches; b++) {
        const int64_t row = row0 + 64 * b;
        id[b] = row < a.count ? a.ids[row] : -1;
        if ((unsigned)id[b] >= (unsigned)a.groups) id[b] = a.groups;
        if (row >= a.count) id[b] = -1;
    }
    for (int i = tid; i < kGrWaves * all; i += kGrWaves * 64) lds[i] = 0;
    __syncthreads();
#pragma unroll
    for (int b = 0; b < kGrBatches; b++) {
        uint64_t s = __ballot(id[b] >= 0);
        for (int bit = 0; bit < a.bits; bit++) {
            const uint64_t one = __ballot((id[b] >> bit) & 1);
            s &= (id[b] >> bit) & 1 ? one : ~one;
        }
        same[b] = s;
        // the first of the lanes with this id counts them
        if (id[b] >= 0 && lane == __builtin_ctzll(s)) hist[id[b]] += __builtin_popcountll(s);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __syncthreads();
    // per group: the earlier waves' rows, and the chunk's
    int mine[2] = {0, 0};   // of groups tid and tid + 1024
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int g = tid + 1024 * h;
        if (g >= all) continue;
        int sum = 0;
        for (int w = 0; w < kGrWaves; w++) {
            const int c = lds[w * all + g];
            lds[w * all + g] = sum;
            sum += c;
        }
        mine[h] = sum;
        if (MODE == 1) a.counts[(int64_t)blockIdx.x * all + g] = sum;
    }
    if (MODE == 1) return;
    int earlier[2] = {0, 0};
    if (MODE == 2) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int g = tid + 1024 * h;
            if (g >= all) continue;
            int sum = 0;
            for (int c = 0; c < a.chunks; c++) {
                if (c == (int)blockIdx.x) earlier[h] = sum;
                sum += a.counts[(int64_t)c * all + g];
            }
            mine[h] = sum;
        }
    }
    // where each group begins: exclusive sums over the groups, group 1024 last
    const int upto = wave_upto(mine[0]);
    if (lane == 63) wave_total[wave] = upto;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < kGrWaves; w++) {
        if (w < wave) before += wave_total[w];
        total += wave_total[w];
    }
    const int begin = before + upto - mine[0];
    if (tid < all) {
        base[tid] = begin + earlier[0];
        if (blockIdx.x == 0) a.offsets[tid] = begin;
    }
    if (tid + 1024 < all) {
        base[tid + 1024] = total + earlier[1];
        if (blockIdx.x == 0) a.offsets[tid + 1024] = total;
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < kGrBatches; b++) {
        if (id[b] >= 0) {
            const uint64_t below = same[b] & (((uint64_t)1 << lane) - 1);
            const int at = base[id[b]] + hist[id[b]] + __builtin_popcountll(below);
            a.order[at] = (int)(row0 + 64 * b);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (id[b] >= 0 && lane == __builtin_ctzll(same[b])) hist[id[b]] += __builtin_popcountll(same[b]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

template <int MODE>
static int launch_group_rows(const GroupRowsArgs &a, hipStream_t s) {
    static LaunchCache cache;
    const int bytes = (kGrWaves + 1) * (a.groups + 1) * 4;
    const int rc = raise_lds_limit(cache, reinterpret_cast<const void *>(&group_rows_kernel<MODE>), (kGrWaves + 1) * (BQM_MAX_GROUPS + 1) * 4);
    if (rc) return rc;
    hipLaunchKernelGGL(group_rows_kernel<MODE>, dim3(a.chunks), dim3(kGrWaves * 64), bytes, s, a);
    return launch_status();
}

}  // namespace bqm

extern "C" int bqm_route(const void *logits, int64_t ld, int type, int top, int renorm, int *ids, float *weights, int m,
                         int e, void *stream) {
    using namespace bqm;
    if (!logits || !ids || !weights || !type_known(type)) return BQM_EINVAL;
    if (m < 1 || e < 1 || e > BQM_MAX_GROUPS || top < 1 || top > BQM_MAX_TOP || top > e) return BQM_EINVAL;
    if ((m > 1 && ld < e) || !aligned(logits, type_bytes(type)) || !aligned(ids, 4) || !aligned(weights, 4)) return BQM_EUNSUPPORTED;
    const int64_t grid = ((int64_t)m + 3) / 4;
    if (grid * 256 > 0x7FFFFFFFll) return BQM_EUNSUPPORTED;   // work items that a dispatch counts
    const RouteArgs a = {logits, m > 1 ? ld : 0, ids, weights, type, top, renorm, m, e};
    hipStream_t s = as_stream(stream);
    const dim3 g((unsigned)grid), b(256);
    if (e <= 64)
        hipLaunchKernelGGL(route_kernel<1>, g, b, 0, s, a);
    else if (e <= 128)
        hipLaunchKernelGGL(route_kernel<2>, g, b, 0, s, a);
    else if (e <= 256)
        hipLaunchKernelGGL(route_kernel<4>, g, b, 0, s, a);
    else if (e <= 512)
        hipLaunchKernelGGL(route_kernel<8>, g, b, 0, s, a);
    else
        hipLaunchKernelGGL(route_kernel<16>, g, b, 0, s, a);
    return launch_status();
}

extern "C" int64_t bqm_group_rows_workspace(int count, int groups) {
    using namespace bqm;
    if (count < 1 || count > 1 << 30 || groups < 1 || groups > BQM_MAX_GROUPS) return -1;
    const int64_t chunks = ((int64_t)count + kGrChunk - 1) / kGrChunk;
    return chunks == 1 ? 0 : chunks * (groups + 1) * 4;
}

extern "C" int bqm_group_rows(const int *ids, int count, int groups, int *offsets, int *order, void *workspace,
                              void *stream) {
    using namespace bqm;
    if (!ids || !offsets || !order) return BQM_EINVAL;
    const int64_t need = bqm_group_rows_workspace(count, groups);
    if (need < 0 || (need > 0 && !workspace)) return BQM_EINVAL;
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(order, 4) || (need > 0 && !aligned(workspace, 4))) return BQM_EUNSUPPORTED;
    GroupRowsArgs a = {ids, offsets, order, static_cast<int *>(workspace), count, groups, (count + kGrChunk - 1) / kGrChunk, 0};
    for (a.bits = 1; (groups >> a.bits) != 0;) a.bits++;   // ids 0..groups
    hipStream_t s = as_stream(stream);
    if (a.chunks == 1) return launch_group_rows<0>(a, s);
    const int rc = launch_group_rows<1>(a, s);
    return rc ? rc : launch_group_rows<2>(a, s);
}
