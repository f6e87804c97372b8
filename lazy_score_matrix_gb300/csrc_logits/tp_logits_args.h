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
// A warp a row from so many rows on, up to so many bytes a row (a kernel that reads the row twice: half, so that the
// 4864 rows under way fit the L2 cache). 12000 x 5000 bf16: forward 77 us with a CTA a row, 38 with a warp; 12000
// x 12000: 91 and 68 us; 8192 x 32000: 97 and 110 us.
constexpr int64_t kWarpRows = kSms * 8, kWarpBytes = 32 << 10;
constexpr int64_t kResident = kSms * 4, kResidentLong = kSms * 2;  // CTAs of kThreads and of kLongThreads on the card

// Many rows of at most warp_bytes: one warp a row. Few rows: a cluster of up to 8 CTAs a row, as long as all of them
// are resident at once (`resident` CTAs on the card) and each keeps 8 KB of the row or more. Else one CTA a row.
inline Shape shape_of(int64_t N, int64_t row_bytes, int64_t warp_bytes, int64_t resident) {
    Shape s;
    s.warp = row_bytes <= warp_bytes && N >= kWarpRows;
    s.cluster = 1;
    while (!s.warp && s.cluster < 8 && 2 * N * s.cluster <= resident && row_bytes >= 2 * s.cluster * (8 << 10)) s.cluster *= 2;
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
