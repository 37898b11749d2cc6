// Shared by the kernels whose rows are grouped by an index on the device.
#pragma once

#include "bqmm_groups.h"
#include "values.h"

namespace bqm {

// The arguments through which rows are found.
struct Grouping {
    const int *offsets, *order;
    int groups, slots;
};

// A workgroup's share of a group: `rows` sorted positions from `first` on, and
// which of the group's tiles (local) it is.
struct GroupTile {
    int group;   // == groups: rows of no group; > groups: no work
    int first, rows, local;
};

// Sum over this lane and the ones below it: within a row of 16 lanes by shifts,
// then the rows before it.
__device__ __forceinline__ int wave_upto(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast 15 to rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast 31 to rows 2 and 3
    return v;
}

// Item `id` of the list in which every group has ceil(rows / bm) * mult items,
// the rows of no group last.  A wave looks at 64 groups at a time; uniform.
// Offsets are taken into 0..slots, so positions are always inside order.
__device__ __forceinline__ GroupTile find_group(const Grouping &q, int bm, int mult, int id) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int base = 0; base <= q.groups; base += 64) {
        const int g = base + lane;
        // both at once, without a branch: a group past the last is empty, the last one ends with the slots
        const int from = q.offsets[min(g, q.groups)], to = q.offsets[min(g + 1, q.groups)];
        const int lo = g <= q.groups ? min(max(from, 0), q.slots) : q.slots;
        const int hi = g < q.groups ? min(max(to, 0), q.slots) : q.slots;
        const int rows = max(hi - lo, 0);
        const int items = (rows + bm - 1) / bm * mult;
        const int upto = wave_upto(items);
        const uint64_t past = __ballot(before + upto > id);
        if (past != 0) {
            const int at = __builtin_ctzll(past);
            GroupTile t;
            t.group = base + at;
            t.local = id - before - (__builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(items, at));
            // offsets that are none can make more items than 32 bits count
            if ((unsigned)t.local >= (unsigned)__builtin_amdgcn_readlane(items, at)) break;
            t.first = __builtin_amdgcn_readlane(lo, at);
            t.rows = __builtin_amdgcn_readlane(rows, at);
            return t;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return GroupTile{q.groups + 1, 0, 0, 0};
}

// The most tiles of bm rows that `slots` rows of `groups` groups (and of none) make.
inline int64_t most_tiles(int slots, int groups, int bm) {
    return (int64_t)slots / bm + (slots < groups + 1 ? slots : groups + 1);
}

// f32 -> type, stored.
__device__ __forceinline__ void store_as(void *p, int64_t i, float v, int type) {
    if (type == BQM_F32)
        static_cast<float *>(p)[i] = v;
    else if (type == BQM_F16)
        static_cast<_Float16 *>(p)[i] = (_Float16)v;
    else
        static_cast<__bf16 *>(p)[i] = (__bf16)v;
}

__device__ __forceinline__ float load_as(const void *p, int64_t i, int type) {
    if (type == BQM_F32) return static_cast<const float *>(p)[i];
    if (type == BQM_F16) return (float)static_cast<const _Float16 *>(p)[i];
    return (float)static_cast<const __bf16 *>(p)[i];
}

// x / (1 + exp(-x)) within 7 steps of 2^-24: the exponential of -|x|, which
// does not overflow, from the hardware's exponential of 2, the product with
// log2 e carried in two parts, and the hardware's reciprocal, refined once.
// The library's exponential and a division took 60 us of the 354 that a gated
// product of 32768 x 4096 x 2816 took.
__device__ __forceinline__ float silu(float x) {
    const float a = fminf(fabsf(x), 200.0f);        // from there on the result is 0, or x; NaN comes back with x
    const float t = a * -1.44269502f;               // log2 e, cut
    const float rest = fmaf(a, -1.44269502f, -t) - a * 1.92596303e-8f;
    const bool tiny = t < -100.0f;                  // below the normal numbers at -126: two factors
    float e = __builtin_amdgcn_exp2f(tiny ? t + 64.0f : t);
    e = fmaf(e, rest * 0.693147182f, e);
    const float d = 1.0f + (tiny ? 0.0f : e);
    float r = __builtin_amdgcn_rcpf(d);
    r = fmaf(r, fmaf(-d, r, 1.0f), r);
    const float y = x * (x < 0.0f ? e * r : r);
    return tiny && x < 0.0f ? y * 5.42101086e-20f : y;   // 2^-64
}

}  // namespace bqm
