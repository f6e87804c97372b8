// Forward kernels of the stored-row consumers (include/tp_logits.h): one pass over each row with the running softmax
// state in registers.
//
// What bounds them is memory on long rows without alternatives or a list (4096 x 131072 bf16: 165 us cold, 0.91 of the
// measured copy rate), instructions and a row's fixed part elsewhere (2048 x 65536 bf16 with 64 alternatives: 76 us, half
// the copy rate; 32768 x 261 fp32 with 8: 31 us for 34 MB).
#include <cuda_runtime.h>

#include "tp_launch.h"
#include "tp_logits.cuh"

namespace tp {
namespace rows {
namespace {

// Alternatives. While a row is read, every thread notes the largest score of each of its chunks. When it has been
// read, the top-th largest of the threads' own maxima bounds the top-th largest score from below: that many
// threads hold a column that reaches it. Only the chunks whose maximum reaches the bound are looked at again, about
// 1.2 times `top` of the 2048 of a row of 64K columns, spread evenly over the threads, and their columns
// that reach it are ranked by counting, each against all others. Where ties let through more chunks or columns
// than there is room for, the whole row is read again and the columns cut back to the best ones by bisection; the
// bound then becomes a key (value and column).
template <int TEAM>
struct TopBuf {
    static constexpr int kKeep = TEAM == 32 ? 96 : kMaxList + 32;       // keys after a cut, at most
    static constexpr int kCap = TEAM == 32 ? 256 : kMaxCluster * kKeep;  // room for what a cluster's CTAs keep
    static constexpr int kSlots = TEAM == kLongThreads ? 8 : 16, kWork = TEAM == 32 ? 128 : 1024;
    alignas(16) unsigned long long key[kCap];
    unsigned long long thr;  // keys at or below it cannot be among the best
    float chunk[kSlots][TEAM];      // largest score of the thread's chunks, `each` of them to a slot
    unsigned short work[kWork];     // slots to look at again: slot * TEAM + thread
    int cnt, todo;
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
        if (Team<TEAM>::tid() == 0) b.cnt = b.todo = 0, b.thr = 0, b.slot[0] = b.slot[1] = b.slot[2] = 0;
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

    // The bound from every thread's largest score (-inf: none): an order (ord_of) that at least `top` of them reach,
    // or 0. `grain`: the step of the scores' type in it.
    __device__ __forceinline__ uint32_t bound(float best, uint32_t grain) {
        const uint32_t o = best > neg_inf() ? ord_of(best) : 0;
        int n = Team<TEAM>::count(o != 0);
        if (n < top) return 0;
        uint32_t lo = ~max(o ? ~o : 0), hi = max(o) + 1;  // smallest and largest
        while (n > top + top / 8 && hi - lo > grain) {
            const uint32_t mid = lo + (hi - lo) / 2;
            const int c = Team<TEAM>::count(o >= mid);
            if (c >= top) lo = mid, n = c;
            else hi = mid;
        }
        return lo;
    }
    // Cuts the buffer back to at most kKeep keys, the best `top` among them. Barriers on both sides.
    __device__ __noinline__ void cut() {
        Team<TEAM>::sync();
        const int t = Team<TEAM>::tid();
        int n = min(b.cnt, Buf::kCap);
        if (n <= Buf::kKeep) return;
        unsigned long long key[kPer];
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
            key[r] = t + r * TEAM < n ? b.key[t + r * TEAM] : 0;
            m = ::max(m, (uint32_t)(key[r] >> 32));
        }
        unsigned long long lo = b.thr + 1, hi = ((unsigned long long)max(m) + 1) << 32;
        while (n > Buf::kKeep) {  // keys differ: this ends at the latest when lo and hi are neighbours
            const unsigned long long mid = lo + (hi - lo) / 2;
            uint32_t c = 0;
#pragma unroll
            for (int r = 0; r < kPer; ++r) c += key[r] >= mid;
            c = sum(c);
            if ((int)c >= top) lo = mid, n = (int)c;
            else hi = mid;
        }
        Team<TEAM>::sync();
        if (t == 0) b.cnt = 0, b.thr = lo - 1;
        Team<TEAM>::sync();
#pragma unroll
        for (int r = 0; r < kPer; ++r)
            if (key[r] >= lo) b.key[atomicAdd(&b.cnt, 1)] = key[r];
        Team<TEAM>::sync();
    }
    // The value that a column from `col` on has to reach. A key at the threshold's value but of a later column
    // is below the threshold, so the bar is then one step higher.
    __device__ __forceinline__ float bar(int col) const {
        const unsigned long long thr = b.thr;
        if (thr == 0) return lowest();
        const uint32_t o = ::max((uint32_t)(thr >> 32), ord_of(lowest()));  // a bound may lie below every finite value
        return of_ord(~(uint32_t)thr < (uint32_t)col ? o + 1 : o);
    }
    // The columns that reach the bar, to the buffer, by way of the chunks that do. false: there was not room for all.
    // Slots hold `each` chunks; the slice begins at vector `begin`.
    template <class T>
    __device__ __forceinline__ bool collect(const RowVecs<T>& x, int begin, int end, int slots, int each, float bar) {
        constexpr int V = Elem<T>::kVec;
        const int t = Team<TEAM>::tid(), chunk = TEAM * kUnroll;
        for (int i = 0; i < slots; ++i)
            if (b.chunk[i][t] >= bar) {
                const int at = atomicAdd(&b.todo, 1);
                if (at < Buf::kWork) b.work[at] = (unsigned short)(i * TEAM + t);
            }
        Team<TEAM>::sync();
        const int n = min(b.todo, Buf::kWork), lane = t % kUnroll * TEAM;
        for (int i = t / kUnroll; i < n; i += TEAM / kUnroll) {
            const int w = b.work[i];
            int j = begin + w / TEAM * each * chunk + w % TEAM + lane;
            for (int c = 0; c < each && j < end; ++c, j += chunk) {
                float f[V];
                Elem<T>::unpack(x.inside(j) ? __ldcg(x.base + j) : x.edge(j), f);
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (f[k] >= bar) {
                        const int at = atomicAdd(&b.cnt, 1);
                        if (at < Buf::kCap) b.key[at] = key_of(f[k], x.first(j) + k);
                    }
            }
        }
        Team<TEAM>::sync();
        return b.todo <= Buf::kWork && b.cnt <= Buf::kCap;
    }
    // The columns of this thread's vectors (vector u at column col0 + u step of the row p) that reach the bar, to the
    // buffer, which is cut back whenever it is full. The whole team calls it.
    template <class T, int N>
    __device__ __forceinline__ void offer(const uint4 (&r)[N], const T* p, int col0, int step, float bar) {
        constexpr int V = Elem<T>::kVec;
        const auto top_bar = Elem<T>::bar(bar);
        uint32_t mask = 0;
#pragma unroll
        for (int u = 0; u < N; ++u)
            if (Elem<T>::reaches(r[u], top_bar)) {  // few do
                float f[V];
                Elem<T>::unpack(r[u], f);
#pragma unroll
                for (int i = 0; i < V; ++i) mask |= f[i] >= bar ? 1u << (u * V + i) : 0u;
            }
        while (true) {
            const unsigned long long thr = b.thr;
            uint32_t left = 0;  // what finds no room
            for (; mask; mask &= mask - 1) {
                const int i = __ffs(mask) - 1, col = col0 + i / V * step + i % V;
                const unsigned long long k = key_of(Elem<T>::get(p[col]), col);
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

// (x - m)/T where the difference itself may leave fp32's range; the bits of (x - m) inv elsewhere
__device__ __forceinline__ float scaled_distance(float x, float m, float inv) { return (0.5f * x - 0.5f * m) * (2.f * inv); }

// The row's results from its state, the token's score xt (thread 0) and the keys of its best columns; `shared`: a word
// for the CTA.
template <int TEAM, bool TOP>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t row, const State& st, float xt, Tops<TEAM>& best, float* shared) {
    const int t = Team<TEAM>::tid();
    const bool some = st.m != neg_inf();
    const float z = st.s + (st.lo + a.sc.delta * st.h);
    float ls = some ? logf(z) : 0.f;
    if (t == 0) {
        if (TOP && TEAM != 32) *shared = ls;  // to the other warps
        const float H = some ? ls - st.h / z * a.sc.inv : 0.f;
        a.entropy[row] = H;
        if (a.logprobs) a.logprobs[row] = some ? scaled_distance(xt, st.m, a.sc.inv) - ls : neg_inf();
        if (a.stats) {
            float* o = a.stats + row * kStats;
            o[0] = st.m, o[1] = ls, o[2] = H;
            for (int i = 3; i < kStats; ++i) o[i] = 0.f;
        }
    }
    if (TOP) {
        Team<TEAM>::sync();
        if (best.b.cnt > TopBuf<TEAM>::kKeep) best.cut();
        if (TEAM != 32) ls = *shared;
        const int n = best.b.cnt;
        for (int i = t; i < n; i += TEAM) {  // the keys differ: a key's place is the number of larger ones
            const unsigned long long k = best.b.key[i];
            int place = n & 1 ? best.b.key[n - 1] > k : 0;
            const ulonglong2* pair = reinterpret_cast<const ulonglong2*>(best.b.key);
#pragma unroll 4
            for (int j = 0; j < n / 2; ++j) {
                const ulonglong2 p = pair[j];
                place += (p.x > k) + (p.y > k);
            }
            if (place < a.top) {
                a.top_logprobs[row * a.top + place] = scaled_distance(of_ord((uint32_t)(k >> 32)), st.m, a.sc.inv) - ls;
                a.top_ids[row * a.top + place] = (int64_t)(~(uint32_t)k);
            }
        }
        for (int i = n + t; i < a.top; i += TEAM) a.top_logprobs[row * a.top + i] = neg_inf(), a.top_ids[row * a.top + i] = -1;
    }
}

struct Gather {  // the candidates of a cluster's CTAs, in the first of them
    static constexpr int kMost = TopBuf<kLongThreads>::kKeep;
    unsigned long long key[kMaxCluster][kMost];
    int n[kMaxCluster];
};

template <class T, int TEAM, bool TOP>
__global__ void __launch_bounds__(TEAM == 32 ? kThreads : TEAM, TEAM == kLongThreads ? 2 : 4) logprobs_kernel(const LogprobArgs a) {
    constexpr int V = Elem<T>::kVec;
    using Tm = Team<TEAM>;
    __shared__ ReduceBuf red;
    __shared__ ClusterBuf parts;
    __shared__ TopBuf<TEAM> tops[TOP ? Tm::kPerCta : 1];
    __shared__ Gather others[1];
    __shared__ uint32_t bounds[kMaxCluster];
    // clusters: the kernels of kLongThreads with alternatives, all of a CTA a row without
    constexpr bool kCluster = TEAM == kLongThreads || (TEAM != 32 && !TOP);
    const int rank = kCluster ? cluster_rank() : 0, size = kCluster ? cluster_size() : 1;
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
    State st;
    const int chunks = (sl.end - sl.begin + TEAM * kUnroll - 1) / (TEAM * kUnroll);
    const int each = max(1, (chunks + TopBuf<TEAM>::kSlots - 1) / TopBuf<TEAM>::kSlots);  // chunks to a slot
    int slot = 0, in_slot = 0;
    float noted = neg_inf();
    uint4 next[kUnroll];  // a chunk is under way while the one before it is reduced
    x.load(next, sl.begin + t, TEAM, sl.end);
    if (TEAM != 32 && t == 0) x.ahead(sl.begin + TEAM * kUnroll, TEAM * kUnroll, sl.end, true);
    for (int base = sl.begin; base < sl.end; base += TEAM * kUnroll) {
        uint4 r[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) r[u] = next[u];
        if (base + TEAM * kUnroll < sl.end) x.load(next, base + TEAM * kUnroll + t, TEAM, sl.end);
        if (TEAM != 32 && t == 0) x.ahead(base + TEAM * kUnroll, TEAM * kUnroll, sl.end);
        const float here = add_scores<T, true>(st, r, a.sc);
        if (TOP) {
            noted = max_nan(noted, here);
            if (++in_slot == each || base + TEAM * kUnroll >= sl.end) tops[Tm::id()].chunk[slot++][t] = noted, noted = neg_inf(), in_slot = 0;
        }
    }
    if (!TOP && TEAM != 32 && t == 0) begin_row<T>(a.x, a.N, row + a.under_way, TEAM * kUnroll);
    const float own = st.m;
    st = team_state<TEAM>(st, a.sc.c, red);
    Tops<TEAM> best(tops[TOP ? Tm::id() : 0], a.top);
    uint32_t bound = 0;
    if (TOP) {
        best.clear();
        bound = best.bound(own, sizeof(T) == 2 ? 1u << 12 : 1u);
    }
    if (size > 1) {
        cluster_wait();  // every CTA of the cluster runs
        cluster_share(st, parts, rank, size);
        if (TOP && t < size) of_rank(bounds, t)[rank] = bound;
        cluster_arrive();
        cluster_wait();
        if (!TOP && rank != 0) return;
        st = cluster_merge(parts, size, a.sc.c);
        if (TOP)
            for (int r = 0; r < size; ++r) bound = max(bound, bounds[r]);  // each holds for the whole row
    }
    if (TOP) {
        if (!best.template collect<T>(x, sl.begin, sl.end, slot, each, bound ? of_ord(bound) : lowest())) {
            Tm::sync();
            if (t == 0) best.b.cnt = 0, best.b.thr = bound ? ((unsigned long long)bound << 32) - 1 : 0;
            Tm::sync();
            for (int base = sl.begin; base < sl.end; base += TEAM * kUnroll) {
                uint4 r[kUnroll];
                x.load(r, base + t, TEAM, sl.end);
                best.template offer<T>(r, x.p, x.first(base + t), TEAM * V, best.bar(max(x.first(base), 0)));
            }
        }
        if (size > 1) {
            best.cut();
            Gather* g = of_rank(&others[0], 0);
            const int n = best.b.cnt;
            for (int i = t; i < n; i += TEAM) g->key[rank][i] = best.b.key[i];
            if (t == 0) g->n[rank] = n;
            cluster_arrive();
            cluster_wait();
            if (rank != 0) return;
            int at = 0;
            for (int r = 0; r < size; ++r) {
                const int m = others[0].n[r];
                for (int i = t; i < m; i += TEAM) best.b.key[at + i] = others[0].key[r][i];
                at += m;
            }
            Tm::sync();
            if (t == 0) best.b.cnt = at, best.b.thr = 0;
        }
    }
    write_row<TEAM, TOP>(a, row, st, t == 0 ? Elem<T>::get(x.p[tok]) : 0.f, best, red.s);
}

// Short rows, a warp each, one score a register: no vectors, so no edges of any, and the maximum before the first
// exponential. 32768 x 261 fp32 with 8 alternatives: 31 us, 42 by logprobs_kernel; without any 17 and 24. At 500 columns
// 36 and 43 us, bf16 41 and 48; with PER = 16 for all lengths 100 columns took 33 us instead of 25. Fewer registers for
// more rows under way: 39 us with five CTAs an SM, 44 with six, 50 with eight. Few rows too: 600 x 261 bf16 with 8 alternatives
// 9 us, 19 with a CTA a row; one row of 32 columns 6 and 10; but 64 x 500 with 32 alternatives 13 and 11. More than 32
// take more threads than a warp's.
constexpr int kShort = 512;
template <class T, bool TOP, int PER>
__global__ void __launch_bounds__(kThreads, 4) logprobs_short_kernel(const LogprobArgs a) {
    using Tm = Team<32>;
    __shared__ TopBuf<32> tops[TOP ? Tm::kPerCta : 1];
    const int64_t row = (int64_t)blockIdx.x * Tm::kPerCta + Tm::id();
    if (row >= a.N) return;
    const int t = Tm::tid(), M = a.x.M;
    const int64_t tok = a.tokens ? a.tokens[row] : 0;
    if (tok < 0 || tok >= M) return leave_out(a, row, t, 32);
    const T* p = row_at<const T>(a.x, row);
    float f[PER], own = neg_inf();
#pragma unroll
    for (int i = 0; i < PER; ++i) f[i] = t + 32 * i < M ? Elem<T>::get(__ldcg(p + t + 32 * i)) : neg_inf();
    const float xt = t == 0 ? Elem<T>::get(p[tok]) : 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) own = max_nan(own, f[i]);
    State st;
    st.m = warp_max(own);
    Tops<32> best(tops[TOP ? Tm::id() : 0], a.top);
    if (TOP) {
        best.clear();
        const uint32_t bound = best.bound(own, sizeof(T) == 2 ? 1u << 12 : 1u);
        const float bar = bound ? of_ord(bound) : lowest();
        int n = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool in = f[i] >= bar;
            const uint32_t who = __ballot_sync(~0u, in);
            if (who == 0) continue;
            if (32 * i >= TopBuf<32>::kCap && n + __popc(who) > TopBuf<32>::kCap) {
                if (t == 0) best.b.cnt = n;
                best.cut();
                n = best.b.cnt;
                __syncwarp();  // all have read it
            }
            if (in) best.b.key[n + __popc(who & ((1u << t) - 1))] = key_of(f[i], t + 32 * i);
            n += __popc(who);
        }
        if (t == 0) best.b.cnt = n;  // read after a barrier, in write_row
    }
    if (st.m != neg_inf()) {
        float2 s = make_float2(0.f, 0.f), h = s;
#pragma unroll
        for (int i = 0; i < PER; i += 2) {
            if (32 * i >= M) break;
            float2 d = sub2(make_float2(f[i], f[i + 1]), st.m);
            d = make_float2(max_nan(d.x, -1e30f), max_nan(d.y, -1e30f));
            const float2 x = mul2(d, a.sc.c), e = make_float2(ex2(x.x), ex2(x.y));
            s = add2(s, e), h = fma2(e, d, h);
        }
        st.s = s.x + s.y, st.h = h.x + h.y;
        warp_sum(st);
    }
    write_row<32, TOP>(a, row, st, xt, best, nullptr);
}

template <class T, bool TOP>
void run_short(const LogprobArgs& a, const Shape& sh, cudaStream_t s) {
    if (a.x.M <= 128) launch(logprobs_short_kernel<T, TOP, 4>, sh, s, a);
    else if (a.x.M <= 256) launch(logprobs_short_kernel<T, TOP, 8>, sh, s, a);
    else if (a.x.M <= 384) launch(logprobs_short_kernel<T, TOP, 12>, sh, s, a);
    else launch(logprobs_short_kernel<T, TOP, 16>, sh, s, a);
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
    uint4 next[kUnroll];
    x.load(next, sl.begin + t, TEAM, sl.end);
    if (TEAM != 32 && t == 0) x.ahead(sl.begin + TEAM * kUnroll, TEAM * kUnroll, sl.end, true);
    look_up<T, TEAM>(a, p, list, 0, a.x.M);
    if (rank == 0) sum_list<TEAM>(a, list);
    State st = read_slice<T, TEAM, REST>(a, x, sl, list, marks[REST ? Tm::id() : 0], next);
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
void run_logprobs(LogprobArgs a, cudaStream_t s) {
    HookScope h("token_logprobs", s);
    const int64_t row = (int64_t)a.x.M * (int64_t)sizeof(T);
    // Up to 32 alternatives for a warp a row: its 32 maxima bound no more than the 32nd largest score. Few rows with
    // alternatives: CTAs of kLongThreads, which alone come in clusters there. Against a CTA of 256 a row, cold: 1 x 131072 bf16,
    // 5 alternatives, 15 us and 17; 8 rows 15 and 19; 64 rows 18 and 19. Where a cluster is small or the row short they lose: 64
    // alternatives, 128 x 131072 24 and 21 us, 600 x 65536 36 and 30; 5 alternatives, 600 x 4096 21 and 12.
    const bool large = a.top && a.N < kResident;
    Shape sh = shape_of(a.N, row, a.top <= 32 ? kWarpBytes : 0, large ? kResidentLong : kResident);
    a.under_way = kResident;
    if (a.x.M <= kShort && a.top <= 32) {
        sh.cluster = 1, sh.grid = (unsigned)((a.N + 7) / 8);
        if (a.top) run_short<T, true>(a, sh, s);
        else run_short<T, false>(a, sh, s);
    } else if (sh.warp) {
        if (a.top) launch(logprobs_kernel<T, 32, true>, sh, s, a);
        else launch(logprobs_kernel<T, 32, false>, sh, s, a);
    } else if (!a.top) {
        launch(logprobs_kernel<T, kThreads, false>, sh, s, a);
    } else if (!large) {
        launch(logprobs_kernel<T, kThreads, true>, sh, s, a);
    } else {
        sh.threads = kLongThreads;
        launch(logprobs_kernel<T, kLongThreads, true>, sh, s, a);
    }
}
template <class T>
void run_distill(const DistillArgs& a, cudaStream_t s) {
    HookScope h("topk_distillation", s);
    const Shape sh = shape_of(a.N, (int64_t)a.x.M * (int64_t)sizeof(T), kWarpBytes, kResident);
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
