// topk_distillation_grad: loss and gradient of a row from one reading of it. The row's scores stay on chip between
// the two: each CTA of a cluster copies a slice of the row into its shared memory, the softmax states meet
// through distributed shared memory, and the gradient is written from the slices.
//
// Traffic is one read of the scores and one write of the gradient, which is all the operator has to move; the
// forward and backward kernels in a row read the scores twice. What bounds it is memory, as long as enough
// slices are resident to cover the time between a slice's last load and its first store (reduction, cluster
// barrier, the list's arithmetic).
#include <cuda_runtime.h>

#include <atomic>

#include "tp_launch.h"
#include "tp_logits.cuh"
#include "tp_logits_out.cuh"

namespace tp {
namespace rows {
namespace {

__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// wait until at most `left` of the thread's groups of copies are under way
__device__ __forceinline__ void copies_wait(int left) {
    if (left >= 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (left == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (left == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The scores of a slice in shared memory: n vectors from element e0 on (of the scores' own alignment).
template <class T>
__device__ __forceinline__ Source<T> from_slice(const uint4* buf, int e0, int n, const T* o) {
    constexpr int V = Elem<T>::kVec;
    Source<T> s;
    const int at = -off_of(o) - e0;                    // where the gradient's vector 0 begins, in elements of buf
    const int r = ((at % V) + V) % V, j = (at - r) / V;
    s.p = reinterpret_cast<const T*>(buf) - e0;
    s.q = buf + j;
    s.shift = r * (int)sizeof(T);
    s.lo = -j, s.hi = n - j - (r ? 1 : 0);
    return s;
}

template <class T, int TEAM, bool REST>
__global__ void __launch_bounds__(kThreads) distill_grad_kernel(const DistillArgs a, int room) {
    constexpr int V = Elem<T>::kVec;
    using Tm = Team<TEAM>;
    extern __shared__ uint4 dyn[];  // per team: room vectors, then (rest) one bit per element of them
    __shared__ ReduceBuf red;
    __shared__ ClusterBuf parts;
    __shared__ ListBuf lists[Tm::kPerCta];
    __shared__ RowStats shared_stats;
    const int words = REST ? room * V / 32 : 0;  // room is a multiple of 32
    uint4* buf = dyn + (size_t)Tm::id() * (room + words / 4);
    uint32_t* marks = reinterpret_cast<uint32_t*>(buf + room);
    const int rank = TEAM == 32 ? 0 : cluster_rank(), size = TEAM == 32 ? 1 : cluster_size();
    const int64_t row = TEAM == 32 ? (int64_t)blockIdx.x * Tm::kPerCta + Tm::id() : blockIdx.x / size;
    if (row >= a.N) return;
    const int t = Tm::tid();
    const T* p = row_at<const T>(a.x, row);
    T* o = row_at<T>(a.g, row);
    ListBuf& list = lists[Tm::id()];
    const RowVecs<T> x(p, a.x.M);
    const Slice sl = slice_of(x.n, rank, size);
    const int n = sl.end - sl.begin;
    // the slice's elements, and the gradient's vectors that hold them (the first and the last may be shared with
    // a neighbouring slice and are then written element by element)
    const int s0 = x.first(sl.begin), e0 = max(s0, 0), e1 = min(x.first(sl.end), a.x.M);
    if (!load_list<TEAM>(a, row, list)) {
        if (rank == 0 && t == 0) {
            a.loss[row] = 0.f;
            for (int i = 0; i < kStats; ++i) a.stats[row * kStats + i] = 0.f;
        }
        return zero_range<T, TEAM>(o, e0, e1);
    }
    if (size > 1) cluster_arrive();
    // every thread copies the vectors that it will reduce: no barrier stands between the two
    for (int i = t; i < n; i += TEAM * kUnroll) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int j = i + u * TEAM;
            if (j < n && x.inside(sl.begin + j)) copy_async(buf + j, x.base + sl.begin + j);
            else if (j < n) buf[j] = x.edge(sl.begin + j);
        }
        copies_end();
    }
    // what the list alone decides, while the copies are under way
    const bool twice = look_up<T, TEAM>(a, p, list, 0, a.x.M);
    if (REST) {
        for (int i = t; i < words; i += TEAM) marks[i] = 0;
        Tm::sync();
        for (int k = t; k < a.K; k += TEAM)
            if (list.ok(k) && list.id[k] >= e0 && list.id[k] < e1) {
                const int at = list.id[k] - s0;
                atomicOr(&marks[at >> 5], 1u << (at & 31));
            }
        Tm::sync();
    }
        if (TEAM == 32 || threadIdx.x < 32) sum_list(a, list);
    State st;
    int left = (n - t + TEAM * kUnroll - 1) / (TEAM * kUnroll);  // groups of this thread
    for (int i = t; i < n; i += TEAM * kUnroll) {
        copies_wait(--left);
        uint4 r[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int j = i + u * TEAM;
            r[u] = j < n ? buf[j] : Elem<T>::none();
            if (REST && j < n) r[u] = without<T>(r[u], marks[j * V >> 5] >> (j * V & 31));
        }
        add_scores<T, false>(st, r, a.sc);
    }
    st = team_state<TEAM>(st, a.sc.c, red);
    if (size > 1) {
        cluster_wait();  // every CTA of the cluster runs
        cluster_share(st, parts, rank, size);
        cluster_arrive();
        cluster_wait();
        st = cluster_merge(parts, size, a.sc.c);
    }
    RowStats s;
    if (TEAM == 32 || threadIdx.x < 32) s = close_row(a, st, list);
    if (rank == 0 && t == 0) {
        a.loss[row] = s.loss;
        float* q = a.stats + row * kStats;
        q[0] = s.m, q[1] = s.ls, q[2] = s.gm, q[3] = s.gls, q[4] = s.Z, q[5] = s.coef;
        q[6] = q[7] = 0.f;
    }
    if (TEAM != 32) {
        if (t == 0) shared_stats = s;
        __syncthreads();
        s = shared_stats;
    } else {
        __syncwarp();
    }
    const float w = (a.weights ? a.weights[row] : 1.f) * a.sc.inv;
    if (s.m == neg_inf()) {  // a row of -inf alone
        zero_range<T, TEAM>(o, e0, e1);
        return;
    }
    const Source<T> from = from_slice<T>(buf, s0, n, o);
    Fetch<T, TEAM, false> scores(o, e0, e1, from);
    distill_row_grad<T, TEAM, false>(a, s, w, o, e0, e1, scores);
    Tm::sync();
    distill_list_grad<T, TEAM>(a, s, w, o, e0, e1, list, twice);
}

constexpr size_t kSmemMost = 200 * 1024;     // a CTA's slice at most
constexpr size_t kSmemThree = 68 * 1024;     // three CTAs an SM
constexpr int64_t kManyRows = 2 * kSms;
constexpr int64_t kWarpBytes = 4096;         // rows up to this long: one warp a row

// Rows too long for that, or for enough of them on an SM: one CTA a row reads it twice, and the second time it comes
// from the L2 cache, as long as the rows under way on the whole card fit there (go_long).

template <class T, bool REST>
__global__ void __launch_bounds__(kLongThreads, 2) distill_grad_long_kernel(const DistillArgs a) {
    constexpr int TEAM = kLongThreads;
    __shared__ ReduceBuf red;
    __shared__ ListBuf list;
    __shared__ RowStats shared_stats;
    __shared__ Marks<TEAM> marks[1];
    const int64_t row = blockIdx.x;
    const T* p = row_at<const T>(a.x, row);
    T* o = row_at<T>(a.g, row);
    const int M = a.x.M;
    if (!load_list<TEAM>(a, row, list)) {
        if (threadIdx.x == 0) {
            a.loss[row] = 0.f;
            for (int i = 0; i < kStats; ++i) a.stats[row * kStats + i] = 0.f;
        }
        return zero_range<T, TEAM>(o, 0, M);
    }
    const RowVecs<T> x(p, M);
    uint4 next[kUnroll];
    x.load(next, threadIdx.x, TEAM, x.n);
    if (threadIdx.x == 0) x.ahead(TEAM * kUnroll, TEAM * kUnroll, x.n, true);
    const bool twice = look_up<T, TEAM>(a, p, list, 0, M);
    if (threadIdx.x < 32) sum_list(a, list);
    State st = read_slice<T, TEAM, REST>(a, x, Slice{0, x.n}, list, marks[0], next);
    const Source<T> from = from_row<T>(p, M, o);
    Fetch<T, TEAM, true> scores(o, 0, M, from);  // the second reading begins while the states meet
    st = team_state<TEAM>(st, a.sc.c, red);
    if (threadIdx.x < 32) {
        const RowStats s = close_row(a, st, list);
        if (threadIdx.x == 0) {
            shared_stats = s;
            a.loss[row] = s.loss;
            float* q = a.stats + row * kStats;
            q[0] = s.m, q[1] = s.ls, q[2] = s.gm, q[3] = s.gls, q[4] = s.Z, q[5] = s.coef;
            q[6] = q[7] = 0.f;
        }
    }
    __syncthreads();
    const RowStats s = shared_stats;
    if (s.m == neg_inf()) return zero_range<T, TEAM>(o, 0, M);  // a row of -inf alone
    const float w = (a.weights ? a.weights[row] : 1.f) * a.sc.inv;
    distill_row_grad<T, TEAM, true>(a, s, w, o, 0, M, scores);
    if (threadIdx.x == 0) begin_row<T>(a.x, a.N, row + a.under_way, TEAM * kUnroll);
    __syncthreads();
    distill_list_grad<T, TEAM>(a, s, w, o, 0, M, list, twice);
}

template <class T, bool REST>
void go_long(DistillArgs a, cudaStream_t s) {
    auto kernel = distill_grad_long_kernel<T, REST>;
    static std::atomic<uint64_t> ready{0};
    if (!raise_smem(kernel, kAlone, ready)) return;
    Shape sh;
    sh.warp = false;
    sh.cluster = 1;
    sh.threads = kLongThreads;
    sh.grid = (unsigned)a.N;
    // two CTAs an SM by their registers, or one by its shared memory
    sh.smem = 2 * kSms * (int64_t)a.x.M * (int64_t)sizeof(T) <= kCacheBytes ? 0 : kAlone;
    a.under_way = kSms * (sh.smem ? 1 : 2);
    HookScope h("topk_distillation_grad", s);
    launch(kernel, sh, s, a);
}

// Shared memory for slices of n vectors; room receives the vectors per team.
inline size_t smem_of(int64_t n, int teams, int V, bool rest, int& room) {
    const int64_t r = (n + 31) / 32 * 32;
    room = (int)r;
    return (size_t)teams * (size_t)(r * 16 + (rest ? r * V / 8 : 0));
}

template <class T, int TEAM, bool REST>
void go(const DistillArgs& a, const Shape& sh, int room, cudaStream_t s) {
    auto kernel = distill_grad_kernel<T, TEAM, REST>;
    static std::atomic<uint64_t> ready{0};
    if (!raise_smem(kernel, kSmemMost, ready)) return;
    HookScope h("topk_distillation_grad", s);
    launch(kernel, sh, s, a, room);
}

template <class T>
void run(const DistillArgs& a, cudaStream_t s) {
    constexpr int V = Elem<T>::kVec;
    const int64_t n = ((int64_t)a.x.M + 2 * V - 2) / V + 1;  // vectors of a row at any alignment, at most
    Shape sh;
    int room = 0;
    sh.warp = n * 16 <= kWarpBytes && a.N >= kWarpRows;
    sh.cluster = 1;
    if (sh.warp) {
        sh.smem = smem_of(n, 8, V, a.rest, room);
        sh.grid = (unsigned)((a.N + 7) / 8);
        if (a.rest) go<T, 32, true>(a, sh, room, s);
        else go<T, 32, false>(a, sh, room, s);
        return;
    }
    const auto smem = [&](int c) { return smem_of((n + c - 1) / c, 1, V, a.rest, room); };
    if (a.N >= kManyRows && smem(1) > kSmemThree) {
        if (a.rest) go_long<T, true>(a, s);
        else go_long<T, false>(a, s);
        return;
    }
    while (sh.cluster < kMaxCluster && (smem(sh.cluster) > kSmemThree || (a.N * sh.cluster < kFewRows && n >= (int64_t)(sh.cluster + 1) * kThreads)))
        ++sh.cluster;
    sh.smem = smem(sh.cluster);
    if (sh.smem > kSmemMost) {
        if (a.rest) go_long<T, true>(a, s);
        else go_long<T, false>(a, s);
        return;
    }
    sh.grid = (unsigned)(a.N * sh.cluster);
    if (a.rest) go<T, kThreads, true>(a, sh, room, s);
    else go<T, kThreads, false>(a, sh, room, s);
}

}  // namespace

void launch_distill_grad(tp_rows_dtype t, const DistillArgs& a, cudaStream_t s) {
    if (t == TP_ROWS_F32) run<float>(a, s);
    else if (t == TP_ROWS_F16) run<__half>(a, s);
    else run<__nv_bfloat16>(a, s);
}

}  // namespace rows
}  // namespace tp
