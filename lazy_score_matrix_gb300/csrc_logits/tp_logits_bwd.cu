// Backward kernels of the stored-row consumers (include/tp_logits.h): the row is read again, its probabilities
// come from the forward's statistics, and each gradient element is written once. Memory bounds them: 4096 x 131072
// bf16 303 us, the measured copy rate; rows whose alignment differs from their gradient's (1021 x 50001 fp32 of rows of
// 50048) 73 us, 0.82 of it.
#include <cuda_runtime.h>

#include "tp_launch.h"
#include "tp_logits.cuh"
#include "tp_logits_out.cuh"

namespace tp {
namespace rows {
namespace {

// Rows are visited from the last to the first: the forward has read the last ones most recently, and what of
// them is left in the cache need not come from memory again.
template <int TEAM>
__device__ __forceinline__ int64_t row_of(int64_t N, int parts) {
    const int64_t r = TEAM == 32 ? (int64_t)blockIdx.x * Team<TEAM>::kPerCta + Team<TEAM>::id() : blockIdx.x / parts;
    return N - 1 - r;
}

template <class T, int TEAM, bool ENTROPY>
__global__ void __launch_bounds__(kThreads) logprobs_bwd_kernel(const LogprobArgs a, int parts) {
    const int64_t row = row_of<TEAM>(a.N, parts);
    if (row < 0) return;
    T* o = row_at<T>(a.g, row);
    const Range r = range_of(o, a.x.M, TEAM == 32 ? 0 : blockIdx.x % parts, parts);
    const int64_t tok = a.tokens ? a.tokens[row] : 0;
    const float* st = a.stats + row * kStats;
    const float m = st[0], ls = st[1], H = st[2];
    if (tok < 0 || tok >= a.x.M || m == neg_inf()) return zero_range<T, TEAM>(o, r.e0, r.e1);
    const float g1 = a.g_logprob ? a.g_logprob[row] * a.sc.inv : 0.f;
    const float g2 = ENTROPY ? a.g_entropy[row] * a.sc.inv : 0.f;
    const float ls2 = ls * kLog2e, c = a.sc.c, gt = a.g_logprob ? g1 : 0.f;
    const float b1 = fmaf(g2, H, g1), b2 = g2 * kLn2;
    const Source<T> x = from_row<T>(row_at<const T>(a.x, row), a.x.M, o);
    Fetch<T, TEAM, false> scores(o, r.e0, r.e1, x);
    map_range<T, TEAM>(o, r.e0, r.e1, scores, [&](float* f, int e) {
#pragma unroll
        for (int i = 0; i < Elem<T>::kVec; ++i) {
            float t = fmaf(f[i] - m, c, -ls2);  // log2 p
            // p = 0 from -126 on: times a small number, so that the weights' product with it stays finite up to 2^120
            if (ENTROPY) t = max_nan(t, -128.f);
            f[i] = -ex2(t) * (ENTROPY ? fmaf(b2, t, b1) : g1);
        }
        if (tok >= e && tok < e + Elem<T>::kVec) {
#pragma unroll
            for (int i = 0; i < Elem<T>::kVec; ++i)
                if (tok == e + i) f[i] += gt;
        }
    });
}

template <class T, int TEAM>
__global__ void __launch_bounds__(kThreads, 4) distill_bwd_kernel(const DistillArgs a, int parts) {
    using Tm = Team<TEAM>;
    __shared__ ListBuf lists[Tm::kPerCta];
    const int64_t row = row_of<TEAM>(a.N, parts);
    if (row < 0) return;
    T* o = row_at<T>(a.g, row);
    const Range r = range_of(o, a.x.M, TEAM == 32 ? 0 : blockIdx.x % parts, parts);
    const T* p = row_at<const T>(a.x, row);
    ListBuf& list = lists[Tm::id()];
    const float* st = a.stats + row * kStats;
    if (!load_list<TEAM>(a, row, list) || st[0] == neg_inf()) return zero_range<T, TEAM>(o, r.e0, r.e1);
    const Source<T> from = from_row<T>(p, a.x.M, o);
    Fetch<T, TEAM, true> scores(o, r.e0, r.e1, from);
    const bool twice = look_up<T, TEAM>(a, p, list, r.e0, r.e1);
    if (TEAM == 32 || threadIdx.x < 32) shares(a, list);
    Tm::sync();
    RowStats s;
    s.m = st[0], s.ls = st[1], s.gm = st[2], s.gls = st[3], s.Z = st[4], s.coef = st[5];
    const float w = (a.weights ? a.weights[row] : 1.f) * a.sc.inv;
    distill_row_grad<T, TEAM>(a, s, w, o, r.e0, r.e1, scores);
    Tm::sync();
    distill_list_grad<T, TEAM>(a, s, w, o, r.e0, r.e1, list, twice);
}

template <class T>
void run_logprobs(const LogprobArgs& a, cudaStream_t s) {
    HookScope h("token_logprobs_backward", s);
    const Shape sh = shape_of(a.N, (int64_t)a.x.M * (int64_t)sizeof(T), kWarpBytes, kResident);
    const int parts = sh.cluster;
    if (sh.warp) {
        if (a.g_entropy) logprobs_bwd_kernel<T, 32, true><<<sh.grid, kThreads, 0, s>>>(a, 1);
        else logprobs_bwd_kernel<T, 32, false><<<sh.grid, kThreads, 0, s>>>(a, 1);
    } else {
        if (a.g_entropy) logprobs_bwd_kernel<T, kThreads, true><<<sh.grid, kThreads, 0, s>>>(a, parts);
        else logprobs_bwd_kernel<T, kThreads, false><<<sh.grid, kThreads, 0, s>>>(a, parts);
    }
}
template <class T>
void run_distill(const DistillArgs& a, cudaStream_t s) {
    HookScope h("topk_distillation_backward", s);
    const Shape sh = shape_of(a.N, (int64_t)a.x.M * (int64_t)sizeof(T), kWarpBytes, kResident);
    if (sh.warp) distill_bwd_kernel<T, 32><<<sh.grid, kThreads, 0, s>>>(a, 1);
    else distill_bwd_kernel<T, kThreads><<<sh.grid, kThreads, 0, s>>>(a, sh.cluster);
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
