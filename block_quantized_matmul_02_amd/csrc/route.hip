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
//    The search is on whole numbers of the values' order.
//  * Sort by counting: a workgroup counts 2048 rows, each wave its own 256 in
//    order, so that a row's place is (rows of lower groups) + (rows of its
//    group in earlier chunks, waves, batches and lanes): no atomics, the same
//    order every time.  Equal ids of a wave are found by a ballot for each bit
//    of the id.  More rows take two launches, the chunks' counts in between,
//    of which each workgroup reads all: right up to 2^24 rows, but the time
//    grows with the square of the chunks (256 groups, 65536 rows 9.6 us, 2^20
//    56, 2^22 440; 2^24 of 1024 32 ms).  At most 64 take a wave that compares
//    them with each other.
//
// In a graph: 1 x 128, 8 of them, and their sort 4.6 us (two launches); 8192 x
// 256 and the sort of 65536 rows 16.5: 8 (the choice: 25 instructions a turn
// and wave), 2 and 7 us.
#include "groups.h"

namespace bqm {

// An f32 (no NaN) as a whole number of the same order, -0 as +0, and back.
__device__ __forceinline__ int order_of(float v) {
    const int b = __builtin_bit_cast(int, v + 0.0f);
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float value_of(int k) { return __builtin_bit_cast(float, k ^ ((k >> 31) & 0x7FFFFFFF)); }

constexpr int kOut = (int)0x807FFFFF;   // of -inf: not to be chosen

// The wave's largest, uniform: shifts within rows of 16 lanes, then the rows
// before, into the last lane.  Whole numbers: a step is one instruction, where
// floats have theirs made quiet first.
__device__ __forceinline__ int wave_max(int v) {
    constexpr int none = (int)0x80000000;
    v = max(v, __builtin_amdgcn_update_dpp(none, v, 0x111, 0xF, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(none, v, 0x112, 0xF, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(none, v, 0x114, 0xF, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(none, v, 0x118, 0xF, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(none, v, 0x142, 0xA, 0xF, false));
    v = max(v, __builtin_amdgcn_update_dpp(none, v, 0x143, 0xC, 0xF, false));
    return __builtin_amdgcn_readlane(v, 63);
}

struct RouteArgs {
    const void *logits;
    int64_t ld;
    int *ids;
    float *weights;
    int top, renorm, m, e;
};

// J: registers of a lane, 64 J >= e.
template <typename T, int J>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.m) return;
    // all loads at once, without branches: past the end the last column again
    const T *const logits = static_cast<const T *>(a.logits) + t * a.ld;
    float v[J];
    int key[J];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < J; j++) v[j] = (float)logits[min(64 * j + lane, a.e - 1)];
#pragma unroll
    for (int j = 0; j < J; j++) {
        bad |= !(v[j] < INFINITY);   // NaN or +inf
        key[j] = v[j] != v[j] || 64 * j + lane >= a.e ? kOut : order_of(v[j]);
    }
    const bool poison = __ballot(bad) != 0;
    // lane i keeps choice i
    int id = -1, chosen = kOut, most = kOut;
    for (int i = 0; i < a.top; i++) {
        int here = key[0];
#pragma unroll
        for (int j = 1; j < J; j++) here = max(here, key[j]);
        here = wave_max(here);
        if (here == kOut) break;
        if (i == 0) most = here;
        // of equals the first register, and there the first lane
        int at = -1;
#pragma unroll
        for (int j = J - 1; j >= 0; j--) {
            const uint64_t equal = __ballot(key[j] == here);
            at = equal != 0 ? 64 * j + __builtin_ctzll(equal) : at;
        }
#pragma unroll
        for (int j = 0; j < J; j++) key[j] = 64 * j + lane == at ? kOut : key[j];
        id = lane == i ? at : id;
        chosen = lane == i ? here : chosen;
    }
    const float top = value_of(most);
    float w = id >= 0 ? expf(value_of(chosen) - top) : 0.0f, z = w;
    if (!a.renorm && most != kOut) {
        z = 0.0f;
#pragma unroll
        for (int j = 0; j < J; j++) z += v[j] == v[j] && 64 * j + lane < a.e ? expf(v[j] - top) : 0.0f;
    }
    z = wave_sum(z);
    if (id >= 0) w = poison ? NAN : w / z;
    if (lane < a.top) {
        a.ids[t * a.top + lane] = id;
        a.weights[t * a.top + lane] = w;
    }
}

template <typename T>
static int launch_route(const RouteArgs &a, unsigned grid, hipStream_t s) {
    const dim3 g(grid), b(256);
    if (a.e <= 64)
        hipLaunchKernelGGL((route_kernel<T, 1>), g, b, 0, s, a);
    else if (a.e <= 128)
        hipLaunchKernelGGL((route_kernel<T, 2>), g, b, 0, s, a);
    else if (a.e <= 256)
        hipLaunchKernelGGL((route_kernel<T, 4>), g, b, 0, s, a);
    else if (a.e <= 512)
        hipLaunchKernelGGL((route_kernel<T, 8>), g, b, 0, s, a);
    else
        hipLaunchKernelGGL((route_kernel<T, 16>), g, b, 0, s, a);
    return launch_status();
}

constexpr int kGrWaves = 8;
constexpr int kGrThreads = kGrWaves * 64;
constexpr int kGrBatches = 4;                               // of 64 rows, a wave
constexpr int kGrChunk = kGrThreads * kGrBatches;        // rows of a workgroup

struct GroupRowsArgs {
    const int *ids;
    int *offsets, *order, *counts;   // counts: [chunks][groups + 1]
    int count, groups, chunks, bits;
};

// A chunk's counts.  Whole numbers: the order in which they are added is free.
__global__ __launch_bounds__(kGrThreads) void group_count_kernel(GroupRowsArgs a) {
    __shared__ int hist[BQM_MAX_GROUPS + 1];
    const int tid = threadIdx.x, all = a.groups + 1;
    const int64_t row0 = (int64_t)blockIdx.x * kGrChunk + tid;
    int id[kGrBatches];
#pragma unroll
    for (int b = 0; b < kGrBatches; b++) {
        const int64_t row = row0 + b * (kGrThreads);
        id[b] = a.ids[row < a.count ? row : a.count - 1];
    }
    for (int i = tid; i < all; i += kGrThreads) hist[i] = 0;
    __syncthreads();
#pragma unroll
    for (int b = 0; b < kGrBatches; b++)
        if (row0 + b * (kGrThreads) < a.count) atomicAdd(&hist[(unsigned)id[b] < (unsigned)a.groups ? id[b] : a.groups], 1);
    __syncthreads();
    for (int i = tid; i < all; i += kGrThreads) a.counts[(int64_t)blockIdx.x * all + i] = hist[i];
}

// CHUNKS: more than one workgroup, whose counts are known.
template <bool CHUNKS>
__global__ __launch_bounds__(kGrThreads) void group_rows_kernel(GroupRowsArgs a) {
    extern __shared__ int lds[];
    __shared__ int wave_total[BQM_MAX_GROUPS / kGrThreads + 1][kGrWaves];
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
        id[b] = a.ids[row < a.count ? row : a.count - 1];
    }
#pragma unroll
    for (int b = 0; b < kGrBatches; b++) {
        if ((unsigned)id[b] >= (unsigned)a.groups) id[b] = a.groups;
        if (row0 + 64 * b >= a.count) id[b] = -1;
    }
    for (int i = tid; i < kGrWaves * all; i += kGrThreads) lds[i] = 0;
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
    // per group: the earlier waves' rows, the chunk's, the earlier chunks' and all
    constexpr int H = BQM_MAX_GROUPS / kGrThreads + 1;   // groups of a thread: tid + kGrThreads h
    int mine[H] = {}, earlier[H] = {};
#pragma unroll
    for (int h = 0; h < H; h++) {
        const int g = tid + kGrThreads * h;
        if (g >= all) continue;
        int c[kGrWaves], sum = 0;
#pragma unroll
        for (int w = 0; w < kGrWaves; w++) c[w] = lds[w * all + g];
#pragma unroll
        for (int w = 0; w < kGrWaves; w++) {
            lds[w * all + g] = sum;
            sum += c[w];
        }
        mine[h] = sum;
    }
    if (CHUNKS) {
#pragma unroll
        for (int h = 0; h < H; h++) {
            const int g = tid + kGrThreads * h;
            if (g >= all) continue;
            int sum = 0, before = 0;
            for (int c0 = 0; c0 < a.chunks; c0 += 32) {
                int c[32];   // all on their way together
#pragma unroll
                for (int i = 0; i < 32; i++) c[i] = a.counts[(int64_t)min(c0 + i, a.chunks - 1) * all + g];
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < 32; i++) {
                    before += c0 + i < (int)blockIdx.x ? c[i] : 0;
                    sum += c0 + i < a.chunks ? c[i] : 0;
                }
            }
            earlier[h] = before;
            mine[h] = sum;
        }
    }
    // where each group begins: exclusive sums over the groups
    int done = 0;
#pragma unroll
    for (int h = 0; h < H; h++) {
        if (kGrThreads * h >= all) break;
        const int upto = wave_upto(mine[h]);
        if (lane == 63) wave_total[h][wave] = upto;
        __syncthreads();
        int before = done;
#pragma unroll
        for (int w = 0; w < kGrWaves; w++) {
            const int c = wave_total[h][w];
            before += w < wave ? c : 0;
            done += c;
        }
        const int g = tid + kGrThreads * h, begin = before + upto - mine[h];
        if (g < all) {
            base[g] = begin + earlier[h];
            if (blockIdx.x == 0) a.offsets[g] = begin;
        }
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

// At most 64 rows and 256 groups: one wave without LDS.  A row's place is the
// rows of lower groups and the earlier ones of its own.
__global__ __launch_bounds__(64) void group_few_kernel(GroupRowsArgs a) {
    constexpr int I = 5;   // groups of a lane: lane, lane + 64, ..
    const int lane = threadIdx.x;
    int id = a.ids[min(lane, a.count - 1)];
    if ((unsigned)id >= (unsigned)a.groups) id = a.groups;
    int place = 0, begin[I] = {};
    for (int j = 0; j < a.count; j++) {
        const int other = __builtin_amdgcn_readlane(id, j);
        place += other < id || (other == id && j < lane) ? 1 : 0;
#pragma unroll
        for (int i = 0; i < I; i++) begin[i] += other < 64 * i + lane ? 1 : 0;
    }
    if (lane < a.count) a.order[place] = lane;
#pragma unroll
    for (int i = 0; i < I; i++)
        if (64 * i + lane <= a.groups) a.offsets[64 * i + lane] = begin[i];
}

template <bool CHUNKS>
static int launch_group_rows(const GroupRowsArgs &a, hipStream_t s) {
    static LaunchCache cache;
    const int bytes = (kGrWaves + 1) * (a.groups + 1) * 4;
    const int rc = raise_lds_limit(cache, reinterpret_cast<const void *>(&group_rows_kernel<CHUNKS>), (kGrWaves + 1) * (BQM_MAX_GROUPS + 1) * 4);
    if (rc) return rc;
    hipLaunchKernelGGL(group_rows_kernel<CHUNKS>, dim3(a.chunks), dim3(kGrThreads), bytes, s, a);
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
    const RouteArgs a = {logits, m > 1 ? ld : 0, ids, weights, top, renorm, m, e};
    hipStream_t s = as_stream(stream);
    if (type == BQM_F32) return launch_route<float>(a, (unsigned)grid, s);
    return type == BQM_F16 ? launch_route<_Float16>(a, (unsigned)grid, s) : launch_route<__bf16>(a, (unsigned)grid, s);
}

extern "C" int64_t bqm_group_rows_workspace(int count, int groups) {
    using namespace bqm;
    if (count < 1 || count > BQM_MAX_ROWS || groups < 1 || groups > BQM_MAX_GROUPS) return -1;
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
    if (count <= 64 && groups <= 256) {
        hipLaunchKernelGGL(group_few_kernel, dim3(1), dim3(64), 0, s, a);
        return launch_status();
    }
    if (a.chunks == 1) return launch_group_rows<false>(a, s);
    hipLaunchKernelGGL(group_count_kernel, dim3(a.chunks), dim3(kGrThreads), 0, s, a);
    const int rc = launch_status();
    return rc ? rc : launch_group_rows<true>(a, s);
}
