// Kernel arguments of the stored-row consumers (include/tp_logits.h), shared by the C entries and the
// kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "tp_logits.h"

namespace tp {
namespace rows {

constexpr int kMaxList = 128;  // longest list of alternatives, and of a teacher's columns
// The unlisted columns' share 1 - sum q counts as 0 below this: log probabilities rounded to fp32, and a common
// error of their normaliser of a few 2^-24, leave up to about 1e-6 of a full list, and a student that masks
// everything else by a large negative score would turn such a remainder into any loss at all.
constexpr float kLeastRest = 1.f / (1 << 20);
constexpr int kStats = 8;      // floats per row that a forward leaves for its backward

struct View {
    void* data;
    int64_t row_stride, group_stride;
    int M, group;
    bool grouped;  // more than one group
};

// The temperature as the kernels use it. c = log2(e)/T rounded to fp32 (exponents are 2^(c d)); its rounding is a
// slightly other temperature for the whole row, which a loss near zero shows. Two ways out: delta = 1/T - c ln 2
// corrects a sum s of exponentials with first moment h to s + delta h; or exponents are formed with c_hi + c_lo =
// log2(e)/T, c_lo > 0.
struct Scale {
    float c, delta, c_hi, c_lo;
    float inv, inv_lo;  // inv + inv_lo = 1/T
};

struct LogprobArgs {
    View x;
    int64_t N, under_way;  // under_way: rows that the card works on at a time
    const int64_t* tokens;
    Scale sc;
    int top;
    float *logprobs, *entropy, *stats, *top_logprobs;
    int64_t* top_ids;
    // backward
    const float *g_logprob, *g_entropy;
    View g;
};

struct DistillArgs {
    View x;
    int64_t N, under_way;
    const int64_t* ids;
    const float* values;
    int K, rest;
    Scale sc;
    float *loss, *stats;
    // backward
    const float* weights;
    View g;
};

// How a kernel's threads are laid over the rows: one warp a row, one CTA, or a cluster of CTAs.
struct Shape {
    bool warp;
    int cluster;
    unsigned grid;
    unsigned threads = 256;
    size_t smem = 0;
};
constexpr int64_t kSms = 152;
constexpr int64_t kWarpCols = 4096, kWarpRows = kSms * 8;
constexpr int64_t kFewRows = kSms * 4;

// Many rows: one CTA a row, or, where a row is short, one warp a row. Few rows: up to 8 CTAs a row, as long as a
// CTA keeps a chunk of `chunk` columns of its own.
inline Shape shape_of(int64_t N, int64_t M, bool warps, int64_t chunk) {
    Shape s;
    s.warp = warps && M <= kWarpCols && N >= kWarpRows;
    s.cluster = 1;
    while (!s.warp && s.cluster < 8 && N * s.cluster < kFewRows && M >= 2 * s.cluster * chunk) s.cluster *= 2;
    s.grid = (unsigned)(s.warp ? (N + 7) / 8 : N * s.cluster);
    return s;
}

// Lets a kernel use so many bytes of dynamic shared memory; `ready` remembers the devices where it may, bit by bit.
// An error is left for the launch check.
template <class K>
inline bool raise_smem(K kernel, size_t bytes, std::atomic<uint64_t>& ready) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (ready.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) return false;
    ready.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Kernels that read a row twice want it in the L2 cache (129 MB) the second time: the rows under way on the whole
// card may take so much of it. Where the CTAs that an SM's registers admit would have more, one is kept alone
// on its SM by shared memory that it does not use.
constexpr int64_t kCacheBytes = (int64_t)110 << 20;
constexpr size_t kAlone = 120 * 1024;

template <class... KArgs, class... Args>
inline void launch(void (*kernel)(KArgs...), const Shape& sh, cudaStream_t s, const Args&... a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sh.grid);
    cfg.blockDim = dim3(sh.threads);
    cfg.dynamicSmemBytes = sh.smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)sh.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = sh.cluster > 1 ? 1 : 0;
    cudaLaunchKernelEx(&cfg, kernel, a...);
}

void launch_logprobs(tp_rows_dtype t, const LogprobArgs& a, cudaStream_t s);
void launch_logprobs_backward(tp_rows_dtype t, const LogprobArgs& a, cudaStream_t s);
void launch_distill(tp_rows_dtype t, const DistillArgs& a, cudaStream_t s);
void launch_distill_grad(tp_rows_dtype t, const DistillArgs& a, cudaStream_t s);
void launch_distill_backward(tp_rows_dtype t, const DistillArgs& a, cudaStream_t s);

}  // namespace rows
}  // namespace tp
