// topk_distillation_grad: loss and gradient of a row by one kernel. The row is read twice, and the second time it
// comes from the L2 cache: traffic to memory is one read of the scores and one write of the gradient, all that the
// operator has to move, while the forward and backward kernels one after the other read the scores twice.
//
// What bounds it is memory, as long as the rows under way on the whole card fit the cache (kCacheBytes) and are
// enough to cover the time between a row's last load and its first store. Measured on 8192 x 131072 bf16 (floor
// 618 us at the measured copy rate): two CTAs of 512 an SM 715 us; one of 1024 957 us (nothing covers the
// reduction); four CTAs an SM with the row's slices in the shared memory of a cluster of four 1100 us (the
// start of a cluster waits for four free places at once), and with slices half as long 2218 us.
#include <cuda_runtime.h>

#include <atomic>

#include "tp_launch.h"
#include "tp_logits.cuh"
#include "tp_logits_out.cuh"

namespace tp {
namespace rows {
namespace {

template <class T, int TEAM, bool REST>
__global__ void __launch_bounds__(TEAM == 32 ? kThreads : TEAM, TEAM == kLongThreads ? 2 : 4) distill_grad_kernel(const DistillArgs a) {
    using Tm = Team<TEAM>;
    constexpr bool kCluster = TEAM == kLongThreads;
    __shared__ ReduceBuf red;
    __shared__ ClusterBuf parts;
    __shared__ ListBuf lists[Tm::kPerCta];
    __shared__ Marks<TEAM> marks[REST ? Tm::kPerCta : 1];
    __shared__ RowStats shared_stats;
    const int rank = kCluster ? cluster_rank() : 0, size = kCluster ? cluster_size() : 1;
    const int64_t row = TEAM == 32 ? (int64_t)blockIdx.x * Tm::kPerCta + Tm::id() : blockIdx.x / size;
    if (row >= a.N) return;
    const int t = Tm::tid(), M = a.x.M;
    const T* p = row_at<const T>(a.x, row);
    T* o = row_at<T>(a.g, row);
    ListBuf& list = lists[Tm::id()];
    const RowVecs<T> x(p, M);
    const Slice sl = slice_of(x.n, rank, size);
    const int e0 = max(x.first(sl.begin), 0), e1 = min(x.first(sl.end), M);  // the slice's elements
    if (!load_list<TEAM>(a, row, list)) {
        if (rank == 0 && t == 0) {
            a.loss[row] = 0.f;
            for (int i = 0; i < kStats; ++i) a.stats[row * kStats + i] = 0.f;
        }
        return zero_range<T, TEAM>(o, e0, e1);
    }
    if (size > 1) cluster_arrive();
    uint4 next[kUnroll];
    x.load(next, sl.begin + t, TEAM, sl.end);
    if (TEAM != 32 && t == 0) x.ahead(sl.begin + TEAM * kUnroll, TEAM * kUnroll, sl.end, true);
    const bool twice = look_up<T, TEAM>(a, p, list, 0, M);
    sum_list<TEAM>(a, list);
    State st = read_slice<T, TEAM, REST>(a, x, sl, list, marks[REST ? Tm::id() : 0], next);
    const Source<T> from = from_row<T>(p, M, o);
    Fetch<T, TEAM, false> scores(o, e0, e1, from);  // the second reading begins while the states meet
    st = team_state<TEAM>(st, a.sc.c, red);
    if (size > 1) {
        cluster_wait();  // every CTA of the cluster runs
        cluster_share(st, parts, rank, size);
        cluster_arrive();
        cluster_wait();  // every CTA has looked the listed scores up: from here on the row may be overwritten
        st = cluster_merge(parts, size, a.sc.c);
    }
    RowStats s;
    if (TEAM == 32 || threadIdx.x < 32) s = close_row(a, st, list);
    if (t == 0) {
        if (TEAM != 32) shared_stats = s;
        if (rank == 0) {
            a.loss[row] = s.loss;
            float* q = a.stats + row * kStats;
            q[0] = s.m, q[1] = s.ls, q[2] = s.gm, q[3] = s.gls, q[4] = s.Z, q[5] = s.coef;
            q[6] = q[7] = 0.f;
        }
    }
    if (TEAM != 32) {
        __syncthreads();
        s = shared_stats;
    }
    if (s.m == neg_inf()) return zero_range<T, TEAM>(o, e0, e1);  // a row of -inf alone
    const float w = (a.weights ? a.weights[row] : 1.f) * a.sc.inv;
    distill_row_grad<T, TEAM>(a, s, w, o, e0, e1, scores);
    if (TEAM != 32 && size == 1 && t == 0) begin_row<T>(a.x, a.N, row + a.under_way, TEAM * kUnroll);
    Tm::sync();
    distill_list_grad<T, TEAM>(a, s, w, o, e0, e1, list, twice);
}

// CTAs of 256 have 608 rows under way, of 512 304; where those would be more than the cache keeps, one of 512 is kept alone
// on its SM by shared memory that it does not use. 3000 rows bf16, 33 entries, CTAs of 256 and of 512: 65536 columns 146 and 170 us,
// 90112 (608 rows are 110 MB) 216 and 211, 131072 341 and 285. 1000 rows, 64 entries, two on an SM and one alone: bf16
// 180224 columns (304 rows are 110 MB) 162 and 169 us, 262144 242 and 234, 700000 669 and 683; fp32 200000 374 and 357, 524288 986
// and 980. Alone gains from 304 rows on; with fewer the second place on an SM is worth more (200 x 262144: 56 and 67).
constexpr int64_t kCacheBytes = (int64_t)110 << 20;
constexpr size_t kAlone = 120 * 1024;

template <class T, int TEAM, bool REST>
void go(DistillArgs a, Shape sh, bool alone, cudaStream_t s) {
    auto kernel = distill_grad_kernel<T, TEAM, REST>;
    if (alone) {
        static std::atomic<uint64_t> ready{0};
        if (!raise_smem(kernel, kAlone, ready)) return;
        sh.smem = kAlone;
    }
    a.under_way = TEAM != kLongThreads ? kResident : alone ? kSms : kResidentLong;
    HookScope h("topk_distillation_grad", s);
    launch(kernel, sh, s, a);
}

template <class T, bool REST>
void run(const DistillArgs& a, cudaStream_t s) {
    const int64_t row = (int64_t)a.x.M * (int64_t)sizeof(T);
    Shape sh = shape_of(a.N, row, kWarpBytes / 2, kResidentLong);
    if (sh.warp) return go<T, 32, REST>(a, sh, false, s);
    if (a.N >= kResident && kResident * row <= kCacheBytes) return go<T, kThreads, REST>(a, sh, false, s);
    sh.threads = kLongThreads;
    go<T, kLongThreads, REST>(a, sh, sh.cluster == 1 && a.N > kSms && kResidentLong * row > kCacheBytes, s);
}

}  // namespace

void launch_distill_grad(tp_rows_dtype t, const DistillArgs& a, cudaStream_t s) {
    const auto by_rest = [&](auto z) {
        using T = decltype(z);
        if (a.rest) run<T, true>(a, s);
        else run<T, false>(a, s);
    };
    if (t == TP_ROWS_F32) by_rest(float{});
    else if (t == TP_ROWS_F16) by_rest(__half{});
    else by_rest(__nv_bfloat16{});
}

}  // namespace rows
}  // namespace tp
