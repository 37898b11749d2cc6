// The weighted sum of each token's slots, for gfx950:
//
//   out[t][i] = (res[t][i] +) sum_j weights[t][j] * y[t * top + j][i]
//
// HBM-bound: every slot's row is read once.  A thread takes 16 bytes of each
// of a token's slots, eight slots' loads at a time.
#include "groups.h"

namespace bqm {

struct CombineArgs {
    const void *y;
    const float *weights;
    const void *res;
    void *out;
    int64_t items;   // of V values, all tokens
    int per, n, top;
};

// V values of a thread at a time, 1 where rows are not aligned.
template <typename T, typename O, int V>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
    typedef T VT __attribute__((ext_vector_type(V), aligned(V == 1 ? sizeof(T) : 16)));
    typedef O VO __attribute__((ext_vector_type(V), aligned(V == 1 ? sizeof(O) : 16)));
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (item >= a.items) return;
    const int64_t t = item / a.per, at = (item - t * a.per) * V;
    const float *const w = a.weights + t * a.top;
    const T *const y = static_cast<const T *>(a.y) + t * a.top * a.n + at;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; i++) sum[i] = 0.0f;
    for (int j0 = 0; j0 < a.top; j0 += 8) {
        VT v[8];
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int q = min(j0 + j, a.top - 1);
            v[j] = *reinterpret_cast<const VT *>(y + (int64_t)q * a.n);
            f[j] = j0 + j < a.top ? w[q] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; j++)
#pragma unroll
            for (int i = 0; i < V; i++) sum[i] = f[j] != 0.0f ? fmaf(f[j], (float)v[j][i], sum[i]) : sum[i];
    }
    VO o;
    const int64_t to = t * a.n + at;
    if (a.res) {
        const VO r = *reinterpret_cast<const VO *>(static_cast<const O *>(a.res) + to);
#pragma unroll
        for (int i = 0; i < V; i++) o[i] = (O)(sum[i] + (float)r[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) o[i] = (O)sum[i];
    }
    *reinterpret_cast<VO *>(static_cast<O *>(a.out) + to) = o;
}

template <typename T, typename O>
static int launch_combine(CombineArgs a, int m, hipStream_t s) {
    constexpr int W = 16 / (int)sizeof(T);
    const bool wide = a.n % W == 0 && aligned(a.y, 16) && aligned(a.out, 16) && aligned(a.res, 16);
    a.per = wide ? a.n / W : a.n;
    a.items = (int64_t)m * a.per;
    if (a.items > 0x7FFFFFFFll - 255) return BQM_EUNSUPPORTED;   // work items that a dispatch counts
    const dim3 grid((unsigned)((a.items + 255) / 256));
    if (wide)
        hipLaunchKernelGGL((combine_kernel<T, O, W>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((combine_kernel<T, O, 1>), grid, dim3(256), 0, s, a);
    return launch_status();
}

}  // namespace bqm

extern "C" int bqm_combine(const void *y, int y_type, const float *weights, const void *res, void *out, int out_type,
                           int m, int top, int n, void *stream) {
    using namespace bqm;
    if (!y || !weights || !out || !type_known(y_type) || !type_known(out_type)) return BQM_EINVAL;
    if (m < 1 || n < 1 || top < 1 || top > BQM_MAX_TOP) return BQM_EINVAL;
    if (out_type != BQM_F32 && out_type != y_type) return BQM_EUNSUPPORTED;
    if (!aligned(y, type_bytes(y_type)) || !aligned(weights, 4) || !aligned(res, type_bytes(out_type)) || !aligned(out, type_bytes(out_type)))
        return BQM_EUNSUPPORTED;
    const CombineArgs a = {y, weights, res, out, 0, 0, n, top};
    hipStream_t s = as_stream(stream);
    if (y_type == BQM_F32) return launch_combine<float, float>(a, m, s);
    if (y_type == BQM_F16)
        return out_type == BQM_F32 ? launch_combine<_Float16, float>(a, m, s) : launch_combine<_Float16, _Float16>(a, m, s);
    return out_type == BQM_F32 ? launch_combine<__bf16, float>(a, m, s) : launch_combine<__bf16, __bf16>(a, m, s);
}
