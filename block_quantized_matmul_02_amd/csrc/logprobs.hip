// Log probabilities of given tokens, log-sum-exp, entropy and the top
// alternatives of rows of logits, for gfx950.
//
// One pass over the logits: every thread keeps a running maximum m and the
// sums Z = sum e^(l-m), S = sum e^(l-m) (l-m), rescaled when m grows; then
//   lse = m + log Z,  log p_j = (l_j - m) - log Z,  H = log Z - S / Z.
// m starts at the lowest finite value, so a masked (-inf) logit gives e = 0
// and no inf - inf arises; Z stays 0 only where a mask leaves nothing.  A NaN
// or +inf reaches Z as NaN.
//
// Top alternatives: a logit and its column make one 64-bit key that orders
// them (value first, then the lower column), so equal logits need no care.
// A wave keeps its 64 best keys sorted, one per lane; the K-th of them is a
// bound, and only logits above it are appended to a short buffer in LDS that
// is sorted (bitonic, DPP exchanges) and merged when it holds a wave of them.
// A wave's first step has no bound yet: it takes the K-th of the lanes' own
// maxima, which at least K logits reach.  Random logits pass the bound about
// K (1 + log(length / 1024)) times in all; rising ones every time, where
// the lanes' maxima bound what a step of 1024 can append.
//
// HBM-bound (one read); with few rows the columns are split over workgroups
// and a second, one-wave launch joins their sums and lists.
#include "values.h"

namespace bqm {

constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / 64;
constexpr int kLpVals = 16;                         // logits per thread and step
constexpr int kLpStep = kLpThreads * kLpVals;       // logits per workgroup and step
constexpr int kLpMaxSplits = 64;                    // a lane for each in the joining launch
constexpr int kLpWantGroups = 2048;                 // workgroups that fill the card: 8 per compute unit
constexpr int kLpMaxN = 1 << 30;                    // 32-bit columns
constexpr float kLowest = -3.402823466e+38f;
constexpr float kLog2e = 1.44269504088896340736f;

struct LpArgs {
    const void *logits;
    int64_t ld;
    const int *tokens;
    float *logp, *lse, *entropy;
    int *top_ids;
    float *top_logp;
    float4 *stats;                 // [m][splits]: m, Z, S
    unsigned long long *keys;      // [m][splits][top]
    int n_tokens, top, m, n, splits;
};

typedef unsigned long long u64;

// ------------------------------------------------------------ keys and sorting

// Whole numbers in the order of the values; -0 as +0, NaN below everything.
__device__ __forceinline__ unsigned order_of(float v) {
    const unsigned u = __builtin_bit_cast(unsigned, v + 0.0f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0;
    return (u >> 31) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float value_of(unsigned order) {
    if (order == 0) return __builtin_nanf("");
    return __builtin_bit_cast(float, (order >> 31) ? order & 0x7FFFFFFFu : ~order);
}

__device__ __forceinline__ u64 key_of(float v, int column) { return ((u64)order_of(v) << 32) | (unsigned)~column; }

// The value of lane l ^ M.
template <int M>
__device__ __forceinline__ unsigned lane_xor(unsigned v) {
    if constexpr (M == 1) return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, false);
    else if constexpr (M == 2) return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, false);
    else if constexpr (M == 3) return __builtin_amdgcn_update_dpp(0, v, 0x1B, 0xF, 0xF, false);
    else if constexpr (M == 4) return lane_xor<3>(lane_xor<7>(v));
    else if constexpr (M == 7) return __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, false);
    else if constexpr (M == 8) return __builtin_amdgcn_update_dpp(0, v, 0x128, 0xF, 0xF, false);
    else if constexpr (M == 15) return __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, false);
    else if constexpr (M == 16) {
        auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        const unsigned even = s[0], odd = s[1];
        return (threadIdx.x & 16) ? even : odd;
    } else if constexpr (M == 31) return lane_xor<16>(lane_xor<15>(v));
    else if constexpr (M == 32) {
        auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        const unsigned low = s[0], high = s[1];
        return (threadIdx.x & 32) ? low : high;
    } else return lane_xor<32>(lane_xor<31>(v));
}

template <int M>
__device__ __forceinline__ u64 lane_xor64(u64 v) {
    return ((u64)lane_xor<M>((unsigned)(v >> 32)) << 32) | lane_xor<M>((unsigned)v);
}

// Of lanes l and l ^ M, the one without M's highest bit keeps the larger key.
template <int M>
__device__ __forceinline__ u64 keep(u64 v) {
    constexpr int H = M >= 32 ? 32 : M >= 16 ? 16 : M >= 8 ? 8 : M >= 4 ? 4 : M >= 2 ? 2 : 1;
    const u64 o = lane_xor64<M>(v);
    return ((threadIdx.x & H) != 0) == (v < o) ? v : o;
}

// 64 keys, one per lane, to descending order.
__device__ __forceinline__ u64 sort64(u64 v) {
    v = keep<1>(v);
    v = keep<1>(keep<3>(v));
    v = keep<1>(keep<2>(keep<7>(v)));
    v = keep<1>(keep<2>(keep<4>(keep<15>(v))));
    v = keep<1>(keep<2>(keep<4>(keep<8>(keep<31>(v)))));
    return keep<1>(keep<2>(keep<4>(keep<8>(keep<16>(keep<63>(v))))));
}

// The 64 largest of two descending lists, descending.
__device__ __forceinline__ u64 merge64(u64 a, u64 b) {
    b = lane_xor64<63>(b);
    const u64 v = a > b ? a : b;
    return keep<1>(keep<2>(keep<4>(keep<8>(keep<16>(keep<32>(v))))));
}

__device__ __forceinline__ u64 from_lane(u64 v, int lane) {
    return ((u64)(unsigned)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32) |
           (unsigned)__builtin_amdgcn_readlane((int)v, lane);
}

// One wave's best keys so far: 64 sorted in registers, and up to 127 more in
// LDS that are above the bound and wait to be merged.
struct WaveTop {
    u64 list;    // this lane's key of the sorted list
    u64 bound;   // a key must be above it; 0: no bound yet
    u64 *buf;    // 128 keys
    int waiting;
    int top;

    __device__ __forceinline__ void init(u64 *b, int k) {
        list = 0;
        bound = 0;
        buf = b;
        waiting = 0;
        top = k;
    }

    __device__ __forceinline__ void raise(u64 b) { bound = b > bound ? b : bound; }

    __device__ __forceinline__ void merge(int count) {
        const int lane = threadIdx.x & 63;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const u64 mine = lane < count ? buf[lane] : 0;
        list = merge64(list, sort64(mine));
        raise(from_lane(list, top - 1));
    }

    __device__ __forceinline__ void append(bool take, u64 key) {
        const u64 mask = __ballot(take);
        if (mask == 0) return;
        const int before = __builtin_amdgcn_mbcnt_hi((unsigned)(mask >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)mask, 0));
        if (take) buf[waiting + before] = key;
        waiting += __popcll(mask);
        if (waiting >= 64) {
            merge(64);
            const int lane = threadIdx.x & 63;
            const int rest = waiting - 64;
            const u64 moved = lane < rest ? buf[64 + lane] : 0;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (lane < rest) buf[lane] = moved;
            waiting = rest;
        }
    }

    __device__ __forceinline__ void finish() {
        if (waiting) merge(waiting);
        waiting = 0;
    }
};

// --------------------------------------------------------------- running sums

struct Sums {
    float m, z, s;
};

__device__ __forceinline__ Sums join(Sums a, Sums b) {
    Sums r;
    r.m = fmaxf(a.m, b.m);
    const float da = fmaxf(a.m - r.m, -200.0f), db = fmaxf(b.m - r.m, -200.0f);   // e^-200 is 0 in f32
    const float fa = __builtin_amdgcn_exp2f(da * kLog2e), fb = __builtin_amdgcn_exp2f(db * kLog2e);
    r.z = a.z * fa + b.z * fb;
    r.s = fa * (a.s + da * a.z) + fb * (b.s + db * b.z);
    return r;
}

template <int M>
__device__ __forceinline__ Sums join_lanes(Sums a) {
    Sums b;
    b.m = __builtin_bit_cast(float, lane_xor<M>(__builtin_bit_cast(unsigned, a.m)));
    b.z = __builtin_bit_cast(float, lane_xor<M>(__builtin_bit_cast(unsigned, a.z)));
    b.s = __builtin_bit_cast(float, lane_xor<M>(__builtin_bit_cast(unsigned, a.s)));
    return join(a, b);
}

__device__ __forceinline__ Sums join_wave(Sums a) {
    return join_lanes<32>(join_lanes<16>(join_lanes<8>(join_lanes<4>(join_lanes<2>(join_lanes<1>(a))))));
}

// ------------------------------------------------------------------- one pass

template <typename T>
__device__ __forceinline__ void write_row(const LpArgs &a, int64_t row, Sums r, u64 list) {
    const int lane = threadIdx.x & 63;
    const bool empty = r.z == 0.0f;   // nothing but -inf
    const float logz = logf(r.z);
    if (lane == 0) {
        a.lse[row] = empty ? -__builtin_inff() : r.m + logz;
        a.entropy[row] = empty ? 0.0f : logz - r.s / r.z;
    }
    const T *l = static_cast<const T *>(a.logits) + row * a.ld;
    for (int i = lane; i < a.n_tokens; i += 64) {
        const int tok = a.tokens[row * a.n_tokens + i];
        float v = __builtin_nanf("");
        if (tok >= 0 && tok < a.n) v = empty ? -__builtin_inff() : ((float)l[tok] - r.m) - logz;
        a.logp[row * a.n_tokens + i] = v;
    }
    if (lane < a.top) {
        a.top_ids[row * a.top + lane] = (int)~(unsigned)list;
        a.top_logp[row * a.top + lane] = empty ? -__builtin_inff() : (value_of((unsigned)(list >> 32)) - r.m) - logz;
    }
}

template <typename T, bool TOP>
__global__ __launch_bounds__(kLpThreads) void logprobs_kernel(LpArgs a) {
    constexpr int V = 16 / sizeof(T);      // logits of a 16-byte load
    constexpr int U = kLpVals / V;
    __shared__ u64 buf[kLpWaves][128];
    __shared__ Sums part[kLpWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = blockIdx.x / (unsigned)a.splits;
    const int split = blockIdx.x % (unsigned)a.splits;
    const T *l = static_cast<const T *>(a.logits) + row * a.ld;
    // loads are aligned to 16 bytes: the row starts `skip` logits into the first
    const int skip = (int)((reinterpret_cast<uintptr_t>(l) & 15) / sizeof(T));
    const int steps = (a.n + skip + kLpStep - 1) / kLpStep;
    const int each = (steps + a.splits - 1) / a.splits;
    const int last = min(steps, (split + 1) * each);

    Sums r = {kLowest, 0.0f, 0.0f};
    WaveTop best;
    best.init(buf[wave], a.top);
    for (int st = split * each; st < last; st++) {
        const int i0 = st * kLpStep + wave * (64 * kLpVals) + lane * V - skip;
        float v[kLpVals];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int i = i0 + u * 64 * V;
            if (i >= 0 && i + V <= a.n) {
                typedef T vec __attribute__((ext_vector_type(V)));
                const vec q = *reinterpret_cast<const vec *>(l + i);
#pragma unroll
                for (int e = 0; e < V; e++) v[u * V + e] = (float)q[e];
            } else {
#pragma unroll
                for (int e = 0; e < V; e++) v[u * V + e] = i + e >= 0 && i + e < a.n ? (float)l[i + e] : -__builtin_inff();
            }
        }
        float big = v[0];
#pragma unroll
        for (int e = 1; e < kLpVals; e++) big = fmaxf(big, v[e]);   // drops NaN

        const float m = fmaxf(r.m, big);
        const float dm = fmaxf(r.m - m, -200.0f);
        const float f = __builtin_amdgcn_exp2f(dm * kLog2e);
        r.s = f * (r.s + dm * r.z);
        r.z *= f;
        r.m = m;
#pragma unroll
        for (int e = 0; e < kLpVals; e++) {
            const float d = v[e] - m;
            const float p = __builtin_amdgcn_exp2f(d * kLog2e);
            r.z += p;
            r.s = __builtin_fmaf(p, fmaxf(d, -200.0f), r.s);   // 0 * -inf is left out
        }

        if constexpr (TOP) {
            auto column = [&](int e) { return i0 + (e / V) * 64 * V + e % V; };
            if ((best.bound >> 32) == 0) {
                // no bound, or one whose value is NaN: compare whole keys
                u64 mine = 0;
#pragma unroll
                for (int e = 0; e < kLpVals; e++) {
                    const int c = column(e);
                    const u64 key = c >= 0 && c < a.n ? key_of(v[e], c) : 0;
                    mine = key > mine ? key : mine;
                }
                if (__popcll(__ballot(mine > best.bound)) >= a.top) best.raise(from_lane(sort64(mine), a.top - 1) - 1);
#pragma unroll 1
                for (int e = 0; e < kLpVals; e++) {
                    float ve = v[0];
#pragma unroll
                    for (int q = 1; q < kLpVals; q++) ve = e == q ? v[q] : ve;
                    const int c = column(e);
                    const u64 key = c >= 0 && c < a.n ? key_of(ve, c) : 0;
                    best.append(key > best.bound, key);
                }
            } else {
                // later columns lose ties, so only a larger value passes
                float low = value_of((unsigned)(best.bound >> 32));
                const u64 above = __ballot(big > low);
                if (above != 0) {
                    if (__popcll(above) >= a.top) {
                        // rising logits: K lanes' maxima pass, so the K-th of them is a bound
                        u64 mine = 0;
#pragma unroll
                        for (int e = 0; e < kLpVals; e++) {
                            const int c = column(e);
                            const u64 key = c >= 0 && c < a.n ? key_of(v[e], c) : 0;
                            mine = key > mine ? key : mine;
                        }
                        best.raise(from_lane(sort64(mine), a.top - 1) - 1);
                        low = value_of((unsigned)(best.bound >> 32));
                    }
#pragma unroll
                    for (int e = 0; e < kLpVals; e++) {
                        if (__ballot(v[e] >= low) == 0) continue;
                        const int c = column(e);
                        const u64 key = c >= 0 && c < a.n ? key_of(v[e], c) : 0;
                        best.append(key > best.bound, key);
                    }
                }
            }
        }
    }

    r = join_wave(r);
    if constexpr (TOP) {
        best.finish();
        buf[wave][lane] = best.list;
    }
    if (lane == 0) part[wave] = r;
    __syncthreads();
    if (wave != 0) return;
    for (int w = 1; w < kLpWaves; w++) {
        r = join(r, part[w]);
        if constexpr (TOP) best.list = merge64(best.list, buf[w][lane]);
    }
    if (a.splits == 1) {
        write_row<T>(a, row, r, best.list);
    } else {
        const int64_t at = row * a.splits + split;
        if (lane == 0) a.stats[at] = make_float4(r.m, r.z, r.s, 0.0f);
        if (lane < a.top) a.keys[at * a.top + lane] = best.list;
    }
}

// Joins a row's splits: one wave.
template <typename T>
__global__ __launch_bounds__(64) void logprobs_join_kernel(LpArgs a) {
    __shared__ u64 buf[128];
    const int lane = threadIdx.x;
    const int64_t row = blockIdx.x;
    Sums r = {kLowest, 0.0f, 0.0f};
    if (lane < a.splits) {
        const float4 q = a.stats[row * a.splits + lane];
        r = {q.x, q.y, q.z};
    }
    r = join_wave(r);
    WaveTop best;
    best.init(buf, a.top);
    if (a.top > 0) {
        const u64 *keys = a.keys + row * a.splits * a.top;
        // the first ceil(top / splits) keys of each list hold at least `top`
        // keys, so the top-th of those is a bound; at most 64 of them
        const int heads = (a.top + a.splits - 1) / a.splits;
        const int mine = lane / heads;
        const u64 head = mine < a.splits ? keys[mine * a.top + lane % heads] : 0;
        const u64 bound = from_lane(sort64(head), a.top - 1);
        if (bound != 0) best.raise(bound - 1);
        const int all = a.splits * a.top;
        for (int i0 = 0; i0 < all; i0 += 512) {
            u64 k[8];
#pragma unroll
            for (int u = 0; u < 8; u++) k[u] = i0 + 64 * u + lane < all ? keys[i0 + 64 * u + lane] : 0;
#pragma unroll 1
            for (int u = 0; u < 8; u++) {
                u64 key = k[0];
#pragma unroll
                for (int q = 1; q < 8; q++) key = u == q ? k[q] : key;
                best.append(key > best.bound, key);
            }
        }
        best.finish();
    }
    write_row<T>(a, row, r, best.list);
}

// Splits of a row: enough workgroups to fill the card, each with at least one
// whole step.  A function of the sizes alone, so that the workspace is too.
static int lp_splits(int m, int n) {
    const int steps = (n + kLpStep - 1) / kLpStep;
    int s = kLpWantGroups / m;
    if (s > steps) s = steps;
    if (s > kLpMaxSplits) s = kLpMaxSplits;
    return s < 1 ? 1 : s;
}

static bool lp_sizes(int m, int n, int top) { return m >= 1 && n >= 1 && top >= 0 && top <= n && top <= BQM_LOGPROBS_MAX_TOP; }

template <typename T>
static int launch_logprobs(const LpArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.m * a.splits));
    if (a.top > 0)
        hipLaunchKernelGGL((logprobs_kernel<T, true>), grid, dim3(kLpThreads), 0, s, a);
    else
        hipLaunchKernelGGL((logprobs_kernel<T, false>), grid, dim3(kLpThreads), 0, s, a);
    if (a.splits == 1) return launch_status();
    const int rc = launch_status();
    if (rc) return rc;
    hipLaunchKernelGGL(logprobs_join_kernel<T>, dim3((unsigned)a.m), dim3(64), 0, s, a);
    return launch_status();
}

}  // namespace bqm

extern "C" int64_t bqm_logprobs_workspace(int m, int n, int top_k) {
    using namespace bqm;
    if (!lp_sizes(m, n, top_k)) return -1;
    const int64_t splits = lp_splits(m, n);
    return splits == 1 ? 0 : m * splits * (int64_t)(sizeof(float4) + 8 * top_k);
}

extern "C" int bqm_logprobs(const void *logits, int64_t ld, int type, const int *tokens, int n_tokens, float *logp,
                            float *lse, float *entropy, int *top_ids, float *top_logp, int top_k, void *workspace,
                            int m, int n, void *stream) {
    using namespace bqm;
    if (!logits || !lse || !entropy) return BQM_EINVAL;
    if (!lp_sizes(m, n, top_k) || n_tokens < 0 || !type_known(type)) return BQM_EINVAL;
    if (n_tokens > 0 && (!tokens || !logp)) return BQM_EINVAL;
    if (top_k > 0 && (!top_ids || !top_logp)) return BQM_EINVAL;
    const int splits = lp_splits(m, n);
    if (splits > 1 && !workspace) return BQM_EINVAL;
    if (m > 1 && ld < n) return BQM_EUNSUPPORTED;
    if (n > kLpMaxN || (int64_t)m * kLpThreads > 0xFFFFFFFFll) return BQM_EUNSUPPORTED;
    if (!aligned(logits, type_bytes(type)) || !aligned(tokens, 4) || !aligned(logp, 4) || !aligned(lse, 4) ||
        !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logp, 4) || !aligned(workspace, 16))
        return BQM_EUNSUPPORTED;
    LpArgs a = {};
    a.logits = logits;
    a.ld = m > 1 ? ld : 0;
    a.tokens = tokens;
    a.logp = logp;
    a.lse = lse;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logp = top_logp;
    a.n_tokens = n_tokens;
    a.top = top_k;
    a.m = m;
    a.n = n;
    a.splits = splits;
    a.stats = static_cast<float4 *>(workspace);
    a.keys = reinterpret_cast<u64 *>(static_cast<char *>(workspace) + (int64_t)m * splits * sizeof(float4));
    hipStream_t s = as_stream(stream);
    if (type == BQM_F16) return launch_logprobs<_Float16>(a, s);
    if (type == BQM_BF16) return launch_logprobs<__bf16>(a, s);
    return launch_logprobs<float>(a, s);
}
