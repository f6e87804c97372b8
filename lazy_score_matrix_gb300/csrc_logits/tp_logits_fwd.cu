// Forward kernels of the stored-row consumers (include/tp_logits.h): one pass over each row with the running
// softmax state in registers; the alternatives are filtered in the same pass.
#include <cuda_runtime.h>

#include "tp_launch.h"
#include "tp_logits.cuh"

namespace tp {
namespace rows {
namespace {

// Alternatives. Candidates (keys) collect in shared memory; keys at or below `thr` cannot be among the best
// `top` and are dropped. When the buffer is full it is cut back to at most kSlack keys more than `top`.
constexpr int kSlack = 16;
template <int TEAM>
struct TopBuf {
    static constexpr int kCap = TEAM == 32 ? 256 : kMaxCluster * (kMaxList + kSlack);
    unsigned long long key[kCap];
    unsigned long long thr;
    int cnt;
    uint32_t slot[3];  // reductions of a CTA, in turn: one in use, one read, one cleared
};

template <int TEAM>
struct Tops {
    using Buf = TopBuf<TEAM>;
    static constexpr int kPer = (Buf::kCap + TEAM - 1) / TEAM;  // keys a thread looks at
    Buf& b;
    const int top;
    int turn = 0;

    __device__ __forceinline__ Tops(Buf& b_, int top_) : b(b_), top(top_) {}
    __device__ __forceinline__ void clear() {
        if (Team<TEAM>::tid() == 0) b.cnt = 0, b.thr = 0, b.slot[0] = b.slot[1] = b.slot[2] = 0;
        Team<TEAM>::sync();
    }
    template <class Op, class Warp>
    __device__ __forceinline__ uint32_t reduce(uint32_t v, Op op, Warp warp) {
        v = warp(v);
        if (TEAM == 32) return v;
        uint32_t* s = &b.slot[turn];
        if ((threadIdx.x & 31) == 0) op(s, v);
        __syncthreads();
        v = *s;
        turn = turn == 2 ? 0 : turn + 1;  // the slot after it was cleared a barrier ago
        if (threadIdx.x == 0) b.slot[turn == 2 ? 0 : turn + 1] = 0;
        return v;
    }
    __device__ __forceinline__ uint32_t sum(uint32_t v) {
        return reduce(v, [](uint32_t* s, uint32_t x) { atomicAdd(s, x); }, [](uint32_t x) { return __reduce_add_sync(~0u, x); });
    }
    __device__ __forceinline__ uint32_t max(uint32_t v) {
        return reduce(v, [](uint32_t* s, uint32_t x) { atomicMax(s, x); }, [](uint32_t x) { return __reduce_max_sync(~0u, x); });
    }

    // A key that at least k of the team's cnt keys (all above `above`) reach, by bisection, until at most `limit`
    // do or the bounds are `grain` apart. `key` are the thread's own of them (0: none).
    __device__ __forceinline__ unsigned long long bound(const unsigned long long (&key)[kPer], int cnt, int k, int limit,
                                                        unsigned long long above, unsigned long long grain) {
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < kPer; ++r) m = ::max(m, (uint32_t)(key[r] >> 32));
        unsigned long long lo = above + 1, hi = ((unsigned long long)max(m) + 1) << 32;
        int n = cnt;
        while (n > limit && hi - lo > grain) {
            const unsigned long long mid = lo + (hi - lo) / 2;
            uint32_t c = 0;
#pragma unroll
            for (int r = 0; r < kPer; ++r) c += key[r] >= mid;
            c = sum(c);
            if ((int)c >= k) lo = mid, n = (int)c;
            else hi = mid;
        }
        return lo;
    }
    // Cuts the buffer back to at most top + kSlack keys, the best `top` among them. Barriers on both sides.
    __device__ __forceinline__ void cut() {
        Team<TEAM>::sync();
        const int t = Team<TEAM>::tid(), cnt = min(b.cnt, Buf::kCap);
        if (cnt <= top + kSlack) return;
        unsigned long long key[kPer];
#pragma unroll
        for (int r = 0; r < kPer; ++r) key[r] = t + r * TEAM < cnt ? b.key[t + r * TEAM] : 0;
        const unsigned long long lo = bound(key, cnt, top, top + kSlack, b.thr, 1);
        Team<TEAM>::sync();
        if (t == 0) b.cnt = 0, b.thr = lo - 1;
        Team<TEAM>::sync();
#pragma unroll
        for (int r = 0; r < kPer; ++r)
            if (key[r] >= lo) b.key[atomicAdd(&b.cnt, 1)] = key[r];
        Team<TEAM>::sync();
    }
    // A first threshold, from every thread's best value so far: `top` threads that reach it are as many columns.
    // `grain`: the step of the scores' type in a key (fp16 and bf16 leave the low bits of an fp32 value alone).
    __device__ __forceinline__ void start(float best, unsigned long long grain) {
        unsigned long long key[kPer];
#pragma unroll
        for (int r = 0; r < kPer; ++r) key[r] = 0;
        if (best > neg_inf()) key[0] = (unsigned long long)ord_of(best) << 32;
        const int have = (int)sum(key[0] != 0);
        if (have < top) return;
        const unsigned long long lo = bound(key, have, top, top + top / 8, 0, grain);
        if (Team<TEAM>::tid() == 0) b.thr = lo - 1;
        Team<TEAM>::sync();
    }
    // The value that a column from `col` on has to reach. A key at the threshold's value but of a later column
    // is below the threshold, so the bar is then one step higher.
    __device__ __forceinline__ float bar(int64_t col) const {
        const unsigned long long thr = b.thr;
        if (thr == 0) return __uint_as_float(0xff7fffffu);  // anything above -inf
        const uint32_t o = ::max((uint32_t)(thr >> 32), 0x00800000u);  // a bound may lie below every finite value
        return of_ord((int64_t)(uint32_t)~(uint32_t)thr < col ? o + 1 : o);
    }
    // Offer this thread's elements of a chunk: bit i of `mask` stands for column col(i), value val(i).
    template <class Col, class Val>
    __device__ __forceinline__ void offer(uint32_t mask, Col col, Val val) {
        while (true) {
            uint32_t left = 0;
            const unsigned long long thr = b.thr;
            for (uint32_t m = mask; m; m &= m - 1) {
                const int i = __ffs(m) - 1;
                const unsigned long long k = key_of(val(i), col(i));
                if (k <= thr) continue;
                const int at = atomicAdd(&b.cnt, 1);
                if (at < Buf::kCap) b.key[at] = k;
                else left |= 1u << i;
            }
            mask = left;
            if (!Team<TEAM>::any(mask != 0)) return;
            cut();
        }
    }
};

// What a row that does not count gives.
__device__ __forceinline__ void leave_out(const LogprobArgs& a, int64_t row, int t, int team) {
    if (t == 0) {
        a.logprobs[row] = 0.f, a.entropy[row] = 0.f;
        if (a.stats)
            for (int i = 0; i < kStats; ++i) a.stats[row * kStats + i] = 0.f;
    }
    for (int i = t; i < a.top; i += team) a.top_logprobs[row * a.top + i] = neg_inf(), a.top_ids[row * a.top + i] = -1;
}

struct Gather {  // the candidates of a cluster's other CTAs
    unsigned long long key[kMaxCluster][kMaxList + kSlack];
    int n[kMaxCluster];
};

template <class T, int TEAM, bool TOP>
__global__ void __launch_bounds__(kThreads, TOP && TEAM != 32 ? 6 : 4) logprobs_kernel(const LogprobArgs a) {
    constexpr int V = Elem<T>::kVec;
    using Tm = Team<TEAM>;
    __shared__ ReduceBuf red;
    __shared__ ClusterBuf parts;
    __shared__ TopBuf<TEAM> tops[TOP ? Tm::kPerCta : 1];
    __shared__ Gather others[1];
    const int rank = TEAM == 32 ? 0 : cluster_rank(), size = TEAM == 32 ? 1 : cluster_size();
    const int64_t row = TEAM == 32 ? (int64_t)blockIdx.x * Tm::kPerCta + Tm::id() : blockIdx.x / size;
    if (row >= a.N) return;
    const int t = Tm::tid();
    const int64_t tok = a.tokens ? a.tokens[row] : 0;
    if (tok < 0 || tok >= a.x.M) {
        if (rank == 0) leave_out(a, row, t, TEAM);
        return;
    }
    if (size > 1) cluster_arrive();
    const RowVecs<T> x(row_at<const T>(a.x, row), a.x.M);
    const Slice sl = slice_of(x.n, rank, size);
    Tops<TEAM> best(tops[TOP ? Tm::id() : 0], a.top);
    if (TOP) best.clear();
    State st;
    uint4 next[kUnroll];  // without alternatives, a chunk is under way while the one before it is reduced
    if (!TOP) x.load(next, sl.begin + t, TEAM, sl.end);
    for (int base = sl.begin; base < sl.end; base += TEAM * kUnroll) {
        uint4 r[kUnroll];
        if (TOP) {
            x.load(r, base + t, TEAM, sl.end);
        } else {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) r[u] = next[u];
            x.load(next, base + TEAM * kUnroll + t, TEAM, sl.end);
        }
        add_scores<T, true>(st, r, a.sc);
        if (TOP) {
            if (base == sl.begin) best.start(st.m, sizeof(T) == 2 ? 1ull << 44 : 1ull << 32);
            const float bar = best.bar(x.first(base));
            uint32_t mask = 0;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                float f[V];
                Elem<T>::unpack(r[u], f);
#pragma unroll
                for (int i = 0; i < V; ++i) mask |= f[i] >= bar ? 1u << (u * V + i) : 0u;
            }
            const auto col = [&](int i) { return x.first(base + (i / V) * TEAM + t) + i % V; };
            best.offer(mask, col, [&](int i) { return Elem<T>::get(x.p[col(i)]); });
        }
    }
    st = team_state<TEAM>(st, a.sc.c, red);
    if (size > 1) {
        if (TOP) best.cut();
        cluster_wait();  // every CTA of the cluster runs
        cluster_share(st, parts, rank, size);
        if (TOP) {
            Gather* g = of_rank(&others[0], 0);
            const int n = min(best.b.cnt, a.top + kSlack);
            for (int i = t; i < n; i += TEAM) g->key[rank][i] = best.b.key[i];
            if (t == 0) g->n[rank] = n;
        }
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
        st = cluster_merge(parts, size, a.sc.c);
        if (TOP) {
            int at = 0;
            for (int r = 0; r < size; ++r) {
                const int n = others[0].n[r];
                for (int i = t; i < n; i += TEAM) best.b.key[at + i] = others[0].key[r][i];
                at += n;
            }
            if (t == 0) best.b.cnt = at, best.b.thr = 0;
        }
    }
    const bool some = st.m != neg_inf();
    const float z = st.s + (st.lo + a.sc.delta * st.h);
    const float ls = some ? logf(z) : 0.f;
    if (t == 0) {
        const float H = some ? ls - st.h / z * a.sc.inv : 0.f;
        a.entropy[row] = H;
        if (a.logprobs) a.logprobs[row] = some ? (Elem<T>::get(x.p[tok]) - st.m) * a.sc.inv - ls : neg_inf();
        if (a.stats) {
            float* o = a.stats + row * kStats;
            o[0] = st.m, o[1] = ls, o[2] = H;
            for (int i = 3; i < kStats; ++i) o[i] = 0.f;
        }
    }
    if (TOP) {
        best.cut();
        const int n = min(best.b.cnt, a.top + kSlack);
        for (int i = t; i < n; i += TEAM) {  // the keys differ: a key's place is the number of larger ones
            const unsigned long long k = best.b.key[i];
            int place = 0;
            for (int j = 0; j < n; ++j) place += best.b.key[j] > k;
            if (place < a.top) {
                a.top_logprobs[row * a.top + place] = (of_ord((uint32_t)(k >> 32)) - st.m) * a.sc.inv - ls;
                a.top_ids[row * a.top + place] = (int64_t)(~(uint32_t)k);
            }
        }
        for (int i = n + t; i < a.top; i += TEAM) a.top_logprobs[row * a.top + i] = neg_inf(), a.top_ids[row * a.top + i] = -1;
    }
}

template <class T, int TEAM, bool REST>
__global__ void __launch_bounds__(kThreads, 4) distill_kernel(const DistillArgs a) {
    using Tm = Team<TEAM>;
    __shared__ ReduceBuf red;
    __shared__ ClusterBuf parts;
    __shared__ ListBuf lists[Tm::kPerCta];
    __shared__ Marks<TEAM> marks[REST ? Tm::kPerCta : 1];
    const int rank = TEAM == 32 ? 0 : cluster_rank(), size = TEAM == 32 ? 1 : cluster_size();
    const int64_t row = TEAM == 32 ? (int64_t)blockIdx.x * Tm::kPerCta + Tm::id() : blockIdx.x / size;
    if (row >= a.N) return;
    const int t = Tm::tid();
    const T* p = row_at<const T>(a.x, row);
    ListBuf& list = lists[Tm::id()];
    if (!load_list<TEAM>(a, row, list)) {
        if (rank == 0 && t == 0) {
            a.loss[row] = 0.f;
            if (a.stats)
                for (int i = 0; i < kStats; ++i) a.stats[row * kStats + i] = 0.f;
        }
        return;
    }
    if (size > 1) cluster_arrive();
    const RowVecs<T> x(p, a.x.M);
    const Slice sl = slice_of(x.n, rank, size);
    look_up<T, TEAM>(a, p, list, 0, a.x.M);
    if (rank == 0 && (TEAM == 32 || threadIdx.x < 32)) sum_list(a, list);
    State st = read_slice<T, TEAM, REST>(a, x, sl, list, marks[REST ? Tm::id() : 0]);
    st = team_state<TEAM>(st, a.sc.c, red);
    if (size > 1) {
        cluster_wait();  // every CTA of the cluster runs
        cluster_share(st, parts, rank, size);
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
        st = cluster_merge(parts, size, a.sc.c);
    }
    if (TEAM == 32 || threadIdx.x < 32) {
        const RowStats s = close_row(a, st, list);
        if (t == 0) {
            a.loss[row] = s.loss;
            if (a.stats) {
                float* o = a.stats + row * kStats;
                o[0] = s.m, o[1] = s.ls, o[2] = s.gm, o[3] = s.gls, o[4] = s.Z, o[5] = s.coef;
                o[6] = o[7] = 0.f;
            }
        }
    }
}

template <class T>
constexpr int64_t kChunk = kThreads * kUnroll * Elem<T>::kVec;

template <class T>
void run_logprobs(const LogprobArgs& a, cudaStream_t s) {
    HookScope h("token_logprobs", s);
    const Shape sh = shape_of(a.N, a.x.M, a.top <= 32, kChunk<T>);
    if (sh.warp) {
        if (a.top) launch(logprobs_kernel<T, 32, true>, sh, s, a);
        else launch(logprobs_kernel<T, 32, false>, sh, s, a);
    } else {
        if (a.top) launch(logprobs_kernel<T, kThreads, true>, sh, s, a);
        else launch(logprobs_kernel<T, kThreads, false>, sh, s, a);
    }
}
template <class T>
void run_distill(const DistillArgs& a, cudaStream_t s) {
    HookScope h("topk_distillation", s);
    const Shape sh = shape_of(a.N, a.x.M, true, kChunk<T>);
    if (sh.warp) {
        if (a.rest) launch(distill_kernel<T, 32, true>, sh, s, a);
        else launch(distill_kernel<T, 32, false>, sh, s, a);
    } else {
        if (a.rest) launch(distill_kernel<T, kThreads, true>, sh, s, a);
        else launch(distill_kernel<T, kThreads, false>, sh, s, a);
    }
}

}  // namespace

void launch_logprobs(tp_rows_dtype t, const LogprobArgs& a, cudaStream_t s) {
    if (t == TP_ROWS_F32) run_logprobs<float>(a, s);
    else if (t == TP_ROWS_F16) run_logprobs<__half>(a, s);
    else run_logprobs<__nv_bfloat16>(a, s);
}
void launch_distill(tp_rows_dtype t, const DistillArgs& a, cudaStream_t s) {
    if (t == TP_ROWS_F32) run_distill<float>(a, s);
    else if (t == TP_ROWS_F16) run_distill<__half>(a, s);
    else run_distill<__nv_bfloat16>(a, s);
}

}  // namespace rows
}  // namespace tp
