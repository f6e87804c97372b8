// Backward kernels of the stored-row consumers (include/tp_logits.h): the row is read again, its probabilities
// come from the forward's statistics, and each gradient element is written once.
#include <cuda_runtime.h>

#include "tp_launch.h"
#include "tp_logits.cuh"

namespace tp {
namespace rows {
namespace {

constexpr int kThreads = 256;

template <class T>
__device__ __forceinline__ void zero_row(const View& g, int64_t row) {
    T* o = row_at<T>(g, row);
    for (int i = threadIdx.x; i < g.M; i += kThreads) o[i] = Elem<T>::put(0.f);
}

template <class T>
__global__ void __launch_bounds__(kThreads) logprobs_bwd_kernel(const LogprobArgs a) {
    const int64_t row = blockIdx.x;
    const int64_t tok = a.tokens ? a.tokens[row] : 0;
    const float* st = a.stats + row * kStats;
    const float m = st[0], ls = st[1], H = st[2];
    if (tok < 0 || tok >= a.x.M || m == neg_inf()) return zero_row<T>(a.g, row);
    const T* x = row_at<const T>(a.x, row);
    T* o = row_at<T>(a.g, row);
    const float g1 = a.g_logprob && a.tokens ? a.g_logprob[row] : 0.f, g2 = a.g_entropy ? a.g_entropy[row] : 0.f;
    const float ls2 = ls * kLog2e;
    for (int i = threadIdx.x; i < a.x.M; i += kThreads) {
        const float t = max_nan(fmaf(Elem<T>::get(x[i]) - m, a.sc.c, -ls2), -1e30f);  // log2 p
        const float p = ex2(t);
        float g = -p * fmaf(g2, fmaf(t, (float)kLn2, H), g1);
        if (i == tok) g += g1;
        o[i] = Elem<T>::put(g * a.sc.inv);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) distill_bwd_kernel(const DistillArgs a) {
    __shared__ ListBuf list;
    __shared__ float q[kMaxList];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const T* x = row_at<const T>(a.x, row);
    const float* st = a.stats + row * kStats;
    const float m = st[0], ls = st[1], gm = st[2], gls = st[3], Z = st[4];
    if (!load_list<T, kThreads>(a, row, x, list) || m == neg_inf()) return zero_row<T>(a.g, row);
    const float w = (a.weights ? a.weights[row] : 1.f) * a.sc.inv;
    // the teacher's shares
    float ym = neg_inf(), sum = 0.f;
    if (!a.rest) {
        for (int k = 0; k < a.K; ++k)
            if (list.ok[k]) ym = max_nan(ym, list.y[k]);
        for (int k = 0; k < a.K; ++k)
            if (list.ok[k]) sum += expf((list.y[k] - ym) * a.sc.inv);
    } else {
        for (int k = 0; k < a.K; ++k)
            if (list.ok[k]) sum += expf(list.y[k]);
    }
    for (int k = tid; k < a.K; k += kThreads)
        q[k] = !list.ok[k] ? 0.f : a.rest ? expf(list.y[k]) : expf((list.y[k] - ym) * a.sc.inv) / sum;
    float coef = Z;
    if (a.rest) {  // Z - sum is q_r: at least kLeastRest, or 0 and what rounding makes of it
        const float q_r = Z - sum > 0.5f * (float)kLeastRest ? Z - sum : 0.f;
        coef = Z * expf((gm - m) * a.sc.inv + gls - ls) - q_r;
    }
    coef *= w;
    const float gls2 = gls * kLog2e;
    T* o = row_at<T>(a.g, row);
    for (int i = tid; i < a.x.M; i += kThreads)
        o[i] = Elem<T>::put(coef * ex2(fmaf(Elem<T>::get(x[i]) - gm, a.sc.c, -gls2)));
    __syncthreads();
    for (int k = tid; k < a.K; k += kThreads)
        if (list.ok[k] && list.first[k]) {
            float qs = 0.f;
            for (int j = k; j < a.K; ++j)
                if (list.id[j] == list.id[k]) qs += q[j];
            o[list.id[k]] = Elem<T>::put(w * (Z * expf((list.x[k] - m) * a.sc.inv - ls) - qs));
        }
}

template <class T>
void run_logprobs(const LogprobArgs& a, cudaStream_t s) {
    HookScope h("token_logprobs_backward", s);
    logprobs_bwd_kernel<T><<<(unsigned)a.N, kThreads, 0, s>>>(a);
}
template <class T>
void run_distill(const DistillArgs& a, cudaStream_t s) {
    HookScope h("topk_distillation_backward", s);
    distill_bwd_kernel<T><<<(unsigned)a.N, kThreads, 0, s>>>(a);
}

}  // namespace

void launch_logprobs_backward(tp_rows_dtype t, const LogprobArgs& a, cudaStream_t s) {
    if (t == TP_ROWS_F32) run_logprobs<float>(a, s);
    else if (t == TP_ROWS_F16) run_logprobs<__half>(a, s);
    else run_logprobs<__nv_bfloat16>(a, s);
}
void launch_distill_backward(tp_rows_dtype t, const DistillArgs& a, cudaStream_t s) {
    if (t == TP_ROWS_F32) run_distill<float>(a, s);
    else if (t == TP_ROWS_F16) run_distill<__half>(a, s);
    else run_distill<__nv_bfloat16>(a, s);
}

}  // namespace rows
}  // namespace tp
