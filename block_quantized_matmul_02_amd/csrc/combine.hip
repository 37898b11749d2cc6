// The weighted sum of each token's slots, for gfx950:
//
//   out[t][i] = (res[t][i] +) sum_j weights[t][j] * y[t * top + j][i]
//
// HBM-bound: every slot's row is read once.  A thread takes 16 bytes of each
// of a token's slots, J slots' loads at a time, whatever the rows' alignment;
// where n is no multiple of that, a row's last thread reads the row's last 16
// bytes and stores the values that are its own (res may be out, so the others'
// are neither read nor stored).
//
// Measured, in a graph: 4001 x 8 x 5120 bf16 69 to 72 us (5.3 TB/s, what a
// large copy reaches), x 10, whose second turn loads its last slot again, 86
// (88 at the copy's rate); 4001 x 8 x 5121 75.1 (95.1 value by value), 5068 x 1 x 2529
// f32 21.2 (44.6 value by value and with eight loads of the one slot, so J is
// 1, 4 or 8), 3000 x 2 x 4100 f16 to f32 31.0 (52.8); 8 x 8 x 4097 f32, all
// latency, 2.7 (2.4).
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

template <typename T, typename O, int J>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
    constexpr int V = 16 / (int)sizeof(T);
    typedef T VT __attribute__((ext_vector_type(V), aligned(sizeof(T))));
    typedef O VO __attribute__((ext_vector_type(V), aligned(sizeof(O))));
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (item >= a.items) return;
    const int64_t t = item / a.per, at = (item - t * a.per) * V;
    const float *const w = a.weights + t * a.top;
    const T *y = static_cast<const T *>(a.y) + t * a.top * a.n;
    const O *res = static_cast<const O *>(a.res) + t * a.n;
    O *out = static_cast<O *>(a.out) + t * a.n;
    if (a.n < V) {
        for (int i = 0; i < a.n; i++) {
            float sum = 0.0f;
            for (int j = 0; j < a.top; j++) sum = w[j] != 0.0f ? fmaf(w[j], (float)y[(int64_t)j * a.n + i], sum) : sum;
            out[i] = (O)(a.res ? sum + (float)res[i] : sum);
        }
        return;
    }
    const int64_t from = min(at, (int64_t)a.n - V);
    const int others = (int)(at - from);   // values before this thread's own
    y += from, res += from, out += from;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; i++) sum[i] = 0.0f;
    for (int j0 = 0; j0 < a.top; j0 += J) {
        VT v[J];
        float f[J];
#pragma unroll
        for (int j = 0; j < J; j++) {
            const int q = min(j0 + j, a.top - 1);
            v[j] = *reinterpret_cast<const VT *>(y + (int64_t)q * a.n);
            f[j] = j0 + j < a.top ? w[q] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < J; j++)
#pragma unroll
            for (int i = 0; i < V; i++) sum[i] = f[j] != 0.0f ? fmaf(f[j], (float)v[j][i], sum[i]) : sum[i];
    }
    if (others) {
        float r[V];
#pragma unroll
        for (int i = 1; i < V; i++) r[i] = a.res && i >= others ? (float)res[i] : 0.0f;
#pragma unroll
        for (int i = 1; i < V; i++)
            if (i >= others) out[i] = (O)(a.res ? sum[i] + r[i] : sum[i]);
        return;
    }
    VO o;
    if (a.res) {
        const VO r = *reinterpret_cast<const VO *>(res);
#pragma unroll
        for (int i = 0; i < V; i++) o[i] = (O)(sum[i] + (float)r[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) o[i] = (O)sum[i];
    }
    *reinterpret_cast<VO *>(out) = o;
}

template <typename T, typename O>
static int launch_combine(CombineArgs a, int m, hipStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    a.per = (int)(((int64_t)a.n + V - 1) / V);
    a.items = (int64_t)m * a.per;
    if (a.items > 0x7FFFFFFFll - 255) return BQM_EUNSUPPORTED;   // work items that a dispatch counts
    const dim3 grid((unsigned)((a.items + 255) / 256));
    if (a.top == 1)
        hipLaunchKernelGGL((combine_kernel<T, O, 1>), grid, dim3(256), 0, s, a);
    else if (a.top <= 4)
        hipLaunchKernelGGL((combine_kernel<T, O, 4>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((combine_kernel<T, O, 8>), grid, dim3(256), 0, s, a);
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
