// Forward kernels of the stored-row consumers (include/tp_logits.h): one pass over each row with the running
// softmax state in registers; the alternatives are filtered in the same pass.
#include <cuda_runtime.h>

#include "tp_launch.h"
#include "tp_logits.cuh"

namespace tp {
namespace rows {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // 16-byte vectors in flight per thread
constexpr int kCap = 1024;  // candidates kept before they are cut back to the best `top`

// Alternatives. Candidates (keys) collect in shared memory; `thr` is the key of the top-th best known so far
// and candidates at or below it are dropped. When the buffer is full it is sorted and cut to its best `top`.
struct TopBuf {
    unsigned long long key[kCap];
    unsigned long long thr;
    int cnt;
};

// key[0..n) sorted descending, n a power of two (bitonic network). Ends with a barrier.
template <int TPB>
__device__ __forceinline__ void block_sort(unsigned long long* key, int n) {
    for (int size = 2; size <= n; size <<= 1)
        for (int stride = size >> 1; stride; stride >>= 1) {
            __syncthreads();
            for (int i = threadIdx.x; i < n / 2; i += TPB) {
                const int a = 2 * i - (i & (stride - 1)), b = a + stride;
                const unsigned long long x = key[a], y = key[b];
                const bool down = (a & size) == 0;
                if ((x < y) == down) key[a] = y, key[b] = x;
            }
        }
    __syncthreads();
}

// The candidates sorted, best first, in key[0..min(cnt, top)); returns that count. Barriers on both sides.
template <int TPB>
__device__ __forceinline__ int top_sorted(TopBuf& b, int top) {
    __syncthreads();
    const int cnt = min(b.cnt, kCap);
    int n = 2;
    while (n < cnt) n <<= 1;
    for (int i = cnt + threadIdx.x; i < n; i += TPB) b.key[i] = 0;
    block_sort<TPB>(b.key, n);
    return min(cnt, top);
}

// Offer this thread's elements of a chunk: bit i of `mask` stands for column col(i), value val(i).
template <int TPB, class Col, class Val>
__device__ __forceinline__ void top_offer(TopBuf& b, int top, uint32_t mask, Col col, Val val) {
    while (true) {
        uint32_t left = 0;
        const unsigned long long thr = b.thr;
        for (uint32_t m = mask; m; m &= m - 1) {
            const int i = __ffs(m) - 1;
            const unsigned long long k = key_of(val(i), col(i));
            if (k <= thr) continue;
            const int at = atomicAdd(&b.cnt, 1);
            if (at < kCap) b.key[at] = k;
            else left |= 1u << i;
        }
        mask = left;
        if (!__syncthreads_or(mask != 0)) return;
        const int have = top_sorted<TPB>(b, top);  // the buffer was full: have == top
        if (threadIdx.x == 0) b.cnt = have, b.thr = b.key[have - 1];
        __syncthreads();
    }
}

template <class T, bool TOP>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a) {
    constexpr int V = Elem<T>::kVec;
    __shared__ ReduceBuf red;
    __shared__ TopBuf tops;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const int64_t tok = a.tokens ? a.tokens[row] : 0;
    if (tok < 0 || tok >= a.x.M) {  // left out: nothing is read
        if (tid == 0) {
            a.logprobs[row] = 0.f, a.entropy[row] = 0.f;
            if (a.stats)
                for (int i = 0; i < kStats; ++i) a.stats[row * kStats + i] = 0.f;
        }
        for (int i = tid; i < a.top; i += kThreads) a.top_logprobs[row * a.top + i] = neg_inf(), a.top_ids[row * a.top + i] = -1;
        return;
    }
    const RowVecs<T> x(row_at<const T>(a.x, row), a.x.M);
    if (TOP) {
        if (tid == 0) tops.cnt = 0, tops.thr = 0;
        __syncthreads();
    }
    State st;
    for (int base = 0; base < x.n; base += kThreads * kUnroll) {
        float f[kUnroll * V];
        if (x.inside(base, base + kThreads * kUnroll)) {
            uint4 r[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) r[u] = x.raw(base + u * kThreads + tid);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) Elem<T>::unpack(r[u], f + u * V);
        } else {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) x.edge(base + u * kThreads + tid, f + u * V);
        }
        add_scores(st, f, a.sc.c);
        if (TOP) {
            const float bar = tops.thr ? of_ord((uint32_t)(tops.thr >> 32)) : neg_inf();
            uint32_t mask = 0;
#pragma unroll
            for (int i = 0; i < kUnroll * V; ++i) mask |= (f[i] > neg_inf() && f[i] >= bar) ? 1u << i : 0u;
            const auto col = [&](int i) { return (int)(x.first(base + (i / V) * kThreads + tid) + i % V); };
            top_offer<kThreads>(tops, a.top, mask, col, [&](int i) { return Elem<T>::get(x.p[col(i)]); });
        }
    }
    st = block_state<kThreads>(st, a.sc.c, red);
    const bool some = st.m != neg_inf();
    const float z = st.s + (st.lo + a.sc.delta * st.h);
    const float ls = some ? logf(z) : 0.f;
    if (tid == 0) {
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
        const int have = top_sorted<kThreads>(tops, a.top);
        for (int i = tid; i < a.top; i += kThreads) {
            const unsigned long long k = tops.key[i < have ? i : 0];
            a.top_logprobs[row * a.top + i] = i < have ? (of_ord((uint32_t)(k >> 32)) - st.m) * a.sc.inv - ls : neg_inf();
            a.top_ids[row * a.top + i] = i < have ? (int64_t)(~(uint32_t)k) : -1;
        }
    }
}

constexpr int kMarkCols = 1 << 16;  // unlisted columns are told by a bit map of this many columns at a time

// The list's part of a row, by one warp: teacher's shares q, the loss, and the row's statistics. `st` is the
// state of all columns (plain) or of the unlisted ones (rest). In fp64: what is left of a loss near zero is
// the difference of logarithms that agree to several digits.
__device__ __forceinline__ void distill_row(const DistillArgs& a, int64_t row, const State& st, const ListBuf& l) {
    const int lane = threadIdx.x & 31;
    const double inv = a.sc.inv64;
    const double zs = exact_sum(st, a.sc);
    float m = st.m;       // maximum over all columns
    double z = zs;        // sum over all columns, relative to m
    double q[4], lq[4];
    if (a.rest) {
        float lm = neg_inf();
        for (int j = 0; j < 4; ++j) {
            const int k = lane + 32 * j;
            if (k < a.K && l.ok[k]) lm = max_nan(lm, l.x[k]);
        }
        m = max_nan(st.m, warp_max(lm));
        double sum = 0;
        for (int j = 0; j < 4; ++j) {
            const int k = lane + 32 * j;
            if (k < a.K && l.ok[k] && l.first[k] && l.x[k] > neg_inf()) sum += exp_table(((double)l.x[k] - m) * inv);
        }
        z = warp_sum64(sum);
        if (st.m > neg_inf()) z += zs * exp_table(((double)st.m - m) * inv);
        if (m != m) z = m;  // NaN
        for (int j = 0; j < 4; ++j) {
            const int k = lane + 32 * j;
            const bool ok = k < a.K && l.ok[k];
            lq[j] = ok ? l.y[k] : 0.0;
            q[j] = ok ? exp_table(lq[j]) : 0.0;
        }
    } else {
        float ym = neg_inf();
        for (int j = 0; j < 4; ++j) {
            const int k = lane + 32 * j;
            if (k < a.K && l.ok[k]) ym = max_nan(ym, l.y[k]);
        }
        ym = warp_max(ym);
        double sum = 0;
        for (int j = 0; j < 4; ++j) {
            const int k = lane + 32 * j;
            const bool ok = k < a.K && l.ok[k];
            lq[j] = ok ? ((double)l.y[k] - ym) * inv : 0.0;
            q[j] = ok ? exp_table(lq[j]) : 0.0;
            sum += q[j];
        }
        sum = warp_sum64(sum);
        const double ln = ln64(sum), r = 1.0 / sum;
        for (int j = 0; j < 4; ++j) q[j] *= r, lq[j] -= ln;
    }
    const double m0 = m == neg_inf() ? 0.0 : (double)m, ls = m == neg_inf() ? 0.0 : ln64(z);
    double loss = 0, Z = 0;
    for (int j = 0; j < 4; ++j) {
        const int k = lane + 32 * j;
        if (q[j] > 0) loss += q[j] * (lq[j] - (((double)l.x[k] - m0) * inv - ls));
        Z += q[j];
    }
    loss = warp_sum64(loss), Z = warp_sum64(Z);
    float gm = m, gls = (float)ls;
    if (a.rest && st.m != neg_inf()) {
        const double q_r = 1.0 - Z >= kLeastRest ? 1.0 - Z : 0.0, lr = ln64(zs), lp = ((double)st.m - m0) * inv + lr - ls;
        if (q_r > 0) loss += q_r * (ln64(q_r) - lp);
        Z += q_r;
        gm = st.m, gls = (float)lr;
    }
    if (lane == 0) {
        a.loss[row] = (float)loss;
        if (a.stats) {
            float* o = a.stats + row * kStats;
            o[0] = m, o[1] = (float)ls, o[2] = gm, o[3] = gls, o[4] = (float)Z;
            o[5] = o[6] = o[7] = 0.f;
        }
    }
}

template <class T, bool REST>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillArgs a) {
    constexpr int V = Elem<T>::kVec;
    __shared__ ReduceBuf red;
    __shared__ ListBuf list;
    __shared__ uint32_t marks[REST ? kMarkCols / 32 + 2 : 1];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const T* p = row_at<const T>(a.x, row);
    if (!load_list<T, kThreads>(a, row, p, list)) {
        if (tid == 0) {
            a.loss[row] = 0.f;
            if (a.stats)
                for (int i = 0; i < kStats; ++i) a.stats[row * kStats + i] = 0.f;
        }
        return;
    }
    const RowVecs<T> x(p, a.x.M);
    constexpr int kMarkVecs = kMarkCols / V;
    State st;
    for (int part = 0; part < x.n; part += kMarkVecs) {
        if (REST) {  // bit i of the map is element first(part) + i
            __syncthreads();
            for (int i = tid; i < kMarkCols / 32 + 2; i += kThreads) marks[i] = 0;
            __syncthreads();
            for (int k = tid; k < a.K; k += kThreads) {
                const int64_t at = list.ok[k] ? list.id[k] - x.first(part) : -1;
                if (at >= 0 && at < kMarkCols) atomicOr(&marks[at >> 5], 1u << (at & 31));
            }
            __syncthreads();
        }
        const int end = min(x.n, part + kMarkVecs);
        for (int base = part; base < end; base += kThreads * kUnroll) {
            float f[kUnroll * V];
            if (base + kThreads * kUnroll <= end && x.inside(base, base + kThreads * kUnroll)) {
                uint4 r[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) r[u] = x.raw(base + u * kThreads + tid);
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) Elem<T>::unpack(r[u], f + u * V);
            } else {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int j = base + u * kThreads + tid;
                    x.edge(j < end ? j : x.n, f + u * V);
                }
            }
            if (REST) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int bit = (base - part + u * kThreads + tid) * V;
                    if (bit >= kMarkCols) continue;
                    const uint32_t w = marks[bit >> 5] >> (bit & 31);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (w & (1u << i)) f[u * V + i] = neg_inf();
                }
            }
            add_scores(st, f, a.sc.c);
        }
    }
    st = block_state<kThreads>(st, a.sc.c, red);
    if (tid < 32) distill_row(a, row, st, list);
}

template <class T>
void run_logprobs(const LogprobArgs& a, cudaStream_t s) {
    HookScope h("token_logprobs", s);
    if (a.top) logprobs_kernel<T, true><<<(unsigned)a.N, kThreads, 0, s>>>(a);
    else logprobs_kernel<T, false><<<(unsigned)a.N, kThreads, 0, s>>>(a);
}
template <class T>
void run_distill(const DistillArgs& a, cudaStream_t s) {
    HookScope h("topk_distillation", s);
    if (a.rest) distill_kernel<T, true><<<(unsigned)a.N, kThreads, 0, s>>>(a);
    else distill_kernel<T, false><<<(unsigned)a.N, kThreads, 0, s>>>(a);
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
