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
// A wave keeps a bound that the K-th best is known to reach; logits above it
// are appended to a short buffer in LDS, and once that holds a wave of them it
// is sorted (bitonic, DPP exchanges) and merged into the 64 best, one per lane,
// whose K-th raises the bound.  So does the K-th of the lanes' running maxima (a
// sort of 64 floats), from the first step on and whenever a logit passes, and a
// workgroup's waves share their bounds.  Random logits pass about
// K (1 + log(length / 1024)) times in all; rising ones every time, where the
// lanes' maxima limit what a step of 1024 can append.  What waits at the end is
// sorted once for the whole workgroup.
//
// HBM-bound (one read, the next two steps' loads in flight); with few rows the
// columns are split over workgroups and a second, one-wave launch joins their
// sums and lists.  512 x 131071 f32 with 5 alternatives: 52 us (5.2 TB/s); 300
// rows of them 40 to 42 (3.8 TB/s: one workgroup a row); one row of 64448 with
// 20: 7.3 us and 4.4 for the join, latency and sorting.
#include "logprobs_keys.h"
#include "values.h"

namespace bqm {

constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / 64;
constexpr int kLpStep = kLpThreads * kLpVals;       // logits per workgroup and step
constexpr int kLpMaxSplits = 64;                    // a lane for each in the joining launch
constexpr int kLpWantGroups = 512;                  // workgroups that fill the card: 2 per compute unit
constexpr int kLpMaxN = 1 << 28;                    // a row's bytes in 31 bits
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

// ------------------------------------------------------------ keys and sorting

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

template <int M>
__device__ __forceinline__ float keepf(float v) {
    constexpr int H = M >= 32 ? 32 : M >= 16 ? 16 : M >= 8 ? 8 : M >= 4 ? 4 : M >= 2 ? 2 : 1;
    const float o = __builtin_bit_cast(float, lane_xor<M>(__builtin_bit_cast(unsigned, v)));
    return (threadIdx.x & H) ? fminf(v, o) : fmaxf(v, o);
}

// 64 values (no NaN), one per lane, to descending order.
__device__ __forceinline__ float sort64f(float v) {
    v = keepf<1>(v);
    v = keepf<1>(keepf<3>(v));
    v = keepf<1>(keepf<2>(keepf<7>(v)));
    v = keepf<1>(keepf<2>(keepf<4>(keepf<15>(v))));
    v = keepf<1>(keepf<2>(keepf<4>(keepf<8>(keepf<31>(v)))));
    return keepf<1>(keepf<2>(keepf<4>(keepf<8>(keepf<16>(keepf<63>(v))))));
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

// One wave's best keys so far: 64 sorted in registers (none before the first
// merge), and more in LDS that are above the bound and wait.
struct WaveTop {
    u64 list;    // this lane's key of the sorted list
    u64 bound;   // a key must be above it; 0: no bound yet
    u64 *buf;    // kLpWaiting keys
    int waiting;
    int top;
    bool merged;

    __device__ __forceinline__ void init(u64 *b, int k) {
        list = 0;
        bound = 0;
        buf = b;
        waiting = 0;
        top = k;
        merged = false;
    }

    __device__ __forceinline__ void raise(u64 b) { bound = b > bound ? b : bound; }

    // Takes in one key per lane (0: none).
    __device__ __forceinline__ void take(u64 mine) {
        mine = sort64(mine);
        list = merged ? merge64(list, mine) : mine;
        merged = true;
        raise(from_lane(list, top - 1));
    }

    // Appends a key of each lane that has one to append.
    __device__ __forceinline__ void append(bool pass, u64 key) {
        const u64 mask = __ballot(pass);
        if (mask == 0) return;
        const int before = __builtin_amdgcn_mbcnt_hi((unsigned)(mask >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)mask, 0));
        if (pass) buf[waiting + before] = key;
        waiting += __popcll(mask);
    }

    // Appends those of a lane's N keys that are above the bound: the lanes'
    // counts are summed up across the wave, and each lane writes its own behind
    // the lanes before it, without a branch.
    template <int N>
    __device__ __forceinline__ void append(const u64 (&k)[N]) {
        int n = 0;
#pragma unroll
        for (int e = 0; e < N; e++) n += k[e] > bound ? 1 : 0;
        int sum = n;   // over lanes 0 .. this one
        sum += __builtin_amdgcn_update_dpp(0, sum, 0x111, 0xF, 0xF, false);   // 1, 2, 4, 8 lanes of a row of 16 back
        sum += __builtin_amdgcn_update_dpp(0, sum, 0x112, 0xF, 0xF, false);
        sum += __builtin_amdgcn_update_dpp(0, sum, 0x114, 0xF, 0xF, false);
        sum += __builtin_amdgcn_update_dpp(0, sum, 0x118, 0xF, 0xF, false);
        sum += __builtin_amdgcn_update_dpp(0, sum, 0x142, 0xA, 0xF, false);   // row 0 to 1, row 2 to 3
        sum += __builtin_amdgcn_update_dpp(0, sum, 0x143, 0xC, 0xF, false);   // rows 0, 1 to 2, 3
        u64 *to = buf + waiting + sum - n;
#pragma unroll
        for (int e = 0; e < N; e++)
            if (k[e] > bound) *to++ = k[e];
        waiting += __builtin_amdgcn_readlane(sum, 63);
    }

    // Merges whole waves of waiting keys.
    __device__ __forceinline__ void drain() {
        while (waiting >= 64) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            waiting -= 64;
            take(buf[waiting + (threadIdx.x & 63)]);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    }

    __device__ __forceinline__ void finish() {
        const int lane = threadIdx.x & 63;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (waiting) take(lane < waiting ? buf[lane] : 0);
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
    __shared__ u64 buf[kLpWaves][kLpWaiting];
    __shared__ u64 lists[kLpWaves][64];
    __shared__ Sums part[kLpWaves];
    __shared__ u64 shared_bound;           // the highest of the waves' bounds
    __shared__ int counts[kLpWaves];       // keys that wait (under 64), + 64 if the wave has a list
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = blockIdx.x / (unsigned)a.splits;
    const int split = blockIdx.x % (unsigned)a.splits;
    const T *l = static_cast<const T *>(a.logits) + row * a.ld;
    // loads are aligned to 16 bytes: the row starts `skip` logits into the
    // first; past its last dword they give zeros
    const int skip = (int)((reinterpret_cast<uintptr_t>(l) & 15) / sizeof(T));
    const __amdgpu_buffer_rsrc_t rl = mx_rsrc(l - skip, ((int64_t)(a.n + skip) * sizeof(T) + 3) & ~3ll);
    const int steps = (a.n + skip + kLpStep - 1) / kLpStep;
    const int each = (steps + a.splits - 1) / a.splits;
    const int last = min(steps, (split + 1) * each);

    struct Raw {
        u32x4 q[U];
    };
    auto load = [&](Raw &w, int st) {
        const uint32_t off = (uint32_t)(st * kLpStep + wave * (64 * kLpVals) + lane * V) * (uint32_t)sizeof(T);
#pragma unroll
        for (int u = 0; u < U; u++) w.q[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rl, off + u * 1024, 0, 0));
    };

    Sums r = {kLowest, 0.0f, 0.0f};
    WaveTop best;
    best.init(buf[wave], a.top);
    float most = -__builtin_inff();   // this lane's largest logit so far
    int passed = 0;                   // lanes that passed since the bound was last looked for
    auto step = [&](const Raw &w, int st) {
        // an atomic load, as other waves raise it meanwhile; on the LDS variable
        // itself, so that it does not wait for the logits in flight (300 x
        // 131071 f32 40 us; 49 where it does)
        u64 others = 0;
        if constexpr (TOP) others = __hip_atomic_load(&shared_bound, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        const int i0 = st * kLpStep + wave * (64 * kLpVals) + lane * V - skip;
        auto column = [&](int e) { return i0 + (e / V) * 64 * V + e % V; };
        float v[kLpVals];
#pragma unroll
        for (int u = 0; u < U; u++) {
            typedef T vec __attribute__((ext_vector_type(V)));
            const vec q = __builtin_bit_cast(vec, w.q[u]);
#pragma unroll
            for (int e = 0; e < V; e++) v[u * V + e] = (float)q[e];
        }
        // columns outside the row: only in its first and last step
        if (st == 0 || (st + 1) * kLpStep > a.n + skip) {
#pragma unroll
            for (int e = 0; e < kLpVals; e++) v[e] = column(e) >= 0 && column(e) < a.n ? v[e] : -__builtin_inff();
        }
        float four[kLpVals / 4];   // fmaxf drops NaN
#pragma unroll
        for (int g = 0; g < kLpVals / 4; g++) four[g] = fmaxf(fmaxf(v[4 * g], v[4 * g + 1]), fmaxf(v[4 * g + 2], v[4 * g + 3]));
        float big = four[0];
#pragma unroll
        for (int g = 1; g < kLpVals / 4; g++) big = fmaxf(big, four[g]);

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
            auto key = [&](int e) {
                const int c = column(e);
                return c >= 0 && c < a.n ? key_of(v[e], c) : 0;
            };
            // the K-th of the lanes' best keys: at least K keys reach it
            auto raise_by_keys = [&]() {
                u64 mine = 0;
#pragma unroll
                for (int e = 0; e < kLpVals; e++) {
                    const u64 k = key(e);
                    mine = k > mine ? k : mine;
                }
                if (__popcll(__ballot(mine > best.bound)) >= a.top) best.raise(from_lane(sort64(mine), a.top - 1) - 1);
            };
            best.raise(others);
            const u64 before = best.bound;
            const LpGate gate(before, st * kLpStep + wave * (64 * kLpVals) - skip);
            const u64 above = __ballot(gate.admits(big));
            most = fmaxf(most, big);
            if (above == 0) return;   // whatever the order of the waves
            // The K-th of the lanes' running maxima is a bound, which all of its
            // value pass; keys decide where many lanes are equal to it.  Looked
            // for when K lanes pass at once and after every 8 + K / 2 that pass:
            // the sort costs as much as appending a few keys.
            const int lanes = __popcll(above);
            passed += lanes;
            if (gate.open || lanes >= a.top || passed >= 8 + a.top / 2) {
                passed = 0;
                const float kth = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sort64f(most)), a.top - 1));
                if (kth >= kLowest && __popcll(__ballot(most == kth)) <= kLpTies)
                    best.raise(((u64)order_of(kth) << 32) - 1);
                else if (gate.open || lanes >= a.top)
                    raise_by_keys();
            }
            // Append what passes: in one go where many lanes have something, else
            // by looking for the few.  (Without a bound on the values fewer than K
            // lanes have keys at all.)
            if ((best.bound >> 32) == 0 || lanes > 8) {
                u64 k[kLpVals];
#pragma unroll
                for (int e = 0; e < kLpVals; e++) k[e] = key(e);
                best.append(k);
            } else {
                const float low = value_of((unsigned)(best.bound >> 32));
#pragma unroll
                for (int g = 0; g < kLpVals / 4; g++) {
                    if (__ballot(four[g] >= low) == 0) continue;
#pragma unroll
                    for (int e = 4 * g; e < 4 * g + 4; e++) {
                        if (__ballot(v[e] >= low) == 0) continue;
                        const u64 k = key(e);
                        best.append(k > best.bound, k);
                    }
                }
            }
            best.drain();
            if (best.bound > before && lane == 0) atomicMax(&shared_bound, best.bound);
        }
    };

    Raw w0, w1;
    load(w0, split * each);
    load(w1, split * each + 1);
    if constexpr (TOP) {
        if (threadIdx.x == 0) shared_bound = 0;
        __syncthreads();
    }
#pragma unroll 1
    for (int st = split * each; st < last; st += 2) {
        step(w0, st);
        load(w0, st + 2);
        if (st + 1 < last) step(w1, st + 1);
        load(w1, st + 3);
    }

    r = join_wave(r);
    if constexpr (TOP) {
        lists[wave][lane] = best.list;
        if (lane == 0) counts[wave] = best.waiting + (best.merged ? 64 : 0);
    }
    if (lane == 0) part[wave] = r;
    __syncthreads();
    if (wave != 0) return;
    for (int w = 1; w < kLpWaves; w++) r = join(r, part[w]);
    if constexpr (TOP) {
        // the waves' lists are sorted; what waits is taken a wave of keys at a time
        int first[kLpWaves + 1];
        first[0] = 0;
#pragma unroll
        for (int w = 0; w < kLpWaves; w++) {
            const int c = __builtin_amdgcn_readfirstlane(counts[w]);
            first[w + 1] = first[w] + (c & 63);
            if (w > 0 && c >= 64) {
                best.list = best.merged ? merge64(best.list, lists[w][lane]) : lists[w][lane];
                best.merged = true;
            }
        }
        for (int j0 = 0; j0 < first[kLpWaves]; j0 += 64) {
            const int j = j0 + lane;
            u64 k = 0;
#pragma unroll
            for (int w = 0; w < kLpWaves; w++)
                if (j >= first[w] && j < first[w + 1]) k = buf[w][j - first[w]];
            best.take(k);
        }
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
    __shared__ u64 buf[64 + 512];   // fewer than 64 waiting and eight waves' worth
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
            best.append(k);
            best.drain();
        }
        best.finish();
    }
    write_row<T>(a, row, r, best.list);
}

// Splits of a row: enough workgroups to fill the card, each with at least one
// whole step.  A function of the sizes alone, so that the workspace is too.
static int lp_splits(int m, int n) {
    const int64_t steps = ((int64_t)n + kLpStep - 1) / kLpStep;
    int s = kLpWantGroups / m;
    if (s > steps) s = (int)steps;
    if (s > kLpMaxSplits) s = kLpMaxSplits;
    return s < 1 ? 1 : s;
}

static bool lp_sizes(int m, int n, int top) { return m >= 1 && n >= 1 && top >= 0 && top <= n && top <= BQM_LOGPROBS_MAX_TOP; }

// A row's bytes in 31 bits, and the work items that a dispatch counts.
static bool lp_fits(int m, int n) { return n <= kLpMaxN && (int64_t)m * kLpThreads <= 0xFFFFFFFFll; }

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
    if (!lp_sizes(m, n, top_k) || !lp_fits(m, n)) return -1;
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
    if (!lp_fits(m, n)) return BQM_EUNSUPPORTED;
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
