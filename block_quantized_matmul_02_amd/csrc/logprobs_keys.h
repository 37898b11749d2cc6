// Keys that order logits, and the rule by which a wave passes over what a bound
// excludes.  Functions of values alone, for the kernels and for the host, where
// a model of the waves tries them in other orders.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bqmm_layer.h"

namespace bqm {

typedef unsigned long long u64;

constexpr int kLpVals = 16;   // logits per thread and step

// Whole numbers in the order of the values; -0 as +0, NaN below everything.
__host__ __device__ __forceinline__ unsigned order_of(float v) {
    const unsigned u = __builtin_bit_cast(unsigned, v + 0.0f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0;
    return (u >> 31) ? ~u : u | 0x80000000u;
}

__host__ __device__ __forceinline__ float value_of(unsigned order) {
    if (order == 0) return __builtin_nanf("");
    return __builtin_bit_cast(float, (order >> 31) ? order & 0x7FFFFFFFu : ~order);
}

__host__ __device__ __forceinline__ u64 key_of(float v, int column) { return ((u64)order_of(v) << 32) | (unsigned)~column; }

// Which lanes of a step may hold a key above a bound, from each lane's largest
// logit (NaN dropped; NaN where it has nothing else).  Every lane that holds one
// has to be among them: the waves share their bounds and nothing orders their
// steps, so a bound's column may be past the step's, at any value, -inf too.
// Compared as the keys are, in whole numbers: a bound just below +0 stands for
// -0 as a float, which is no less than +0.
struct LpGate {
    unsigned order;   // of the bound's value
    bool open;        // no bound, or one whose value is NaN: every lane may
    bool strict;      // the step's columns are past the bound's and lose ties against it

    __host__ __device__ __forceinline__ LpGate(u64 bound, int first_column)
        : order((unsigned)(bound >> 32)), open(order == 0), strict(first_column > (int)~(unsigned)bound) {}

    __host__ __device__ __forceinline__ bool admits(float big) const {
        const unsigned o = order_of(big);
        return open || o > order || (!strict && o == order);
    }
};

// Keys that can wait: fewer than a wave of them, and what a step appends before
// they are looked at: up to 16 of each lane that holds one above the bound.
// Those are at most K lanes or, where the bound is a value, K - 1 above it and 8
// equal to it; where a step has looked for no bound, fewer than K lanes passed
// the gate, and where it found none, fewer than K hold a key above the old one.
constexpr int kLpTies = 8;
constexpr int kLpWaiting = 64 + (BQM_LOGPROBS_MAX_TOP + kLpTies) * kLpVals;

}  // namespace bqm
