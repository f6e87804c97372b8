// Device-side building blocks of the stored-row consumers (include/tp_logits.h): row addressing, 16-byte
// loads at any alignment, the running softmax state of a row and its reduction over a CTA.
//
// Running state of a set of scores x: m = max x, s = sum 2^(c (x - m)), h = sum 2^(c (x - m)) (x - m), with
// c = log2(e)/T. s and h are enough for everything a row gives: log-sum-exp = m/T + ln s, entropy = ln s -
// h/(s T). x - m is formed before the product with c: it is exact where it matters (scores near the
// maximum), whereas c x - c m would carry the rounding of c m, 2^-24 |c m|, into every term.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tp_device.cuh"
#include "tp_logits_args.h"

namespace tp {
namespace rows {

constexpr int kThreads = 256;  // per CTA of every kernel here
constexpr int kUnroll = 4;     // 16-byte vectors a thread has in flight
constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.69314718055994530942;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float ex2(float x) { return ExpTraits<float>::bexp(x); }
// maximum that keeps a NaN of either operand, so that a NaN score reaches the row's results
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <class T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kVec = 4;  // elements of a 16-byte vector
    __device__ __forceinline__ static float get(float v) { return v; }
    __device__ __forceinline__ static float put(float v) { return v; }
    __device__ __forceinline__ static uint4 pack(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    __device__ __forceinline__ static void unpack(const uint4& v, float* f) {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    }
};
template <>
struct Elem<__half> {
    static constexpr int kVec = 8;
    __device__ __forceinline__ static float get(__half v) { return __half2float(v); }
    __device__ __forceinline__ static __half put(float v) { return __float2half_rn(v); }
    __device__ __forceinline__ static uint32_t two(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static uint4 pack(const float* f) {
        return make_uint4(two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7]));
    }
    __device__ __forceinline__ static void pair(uint32_t u, float* f) {
        const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&u));
        f[0] = r.x, f[1] = r.y;
    }
    __device__ __forceinline__ static void unpack(const uint4& v, float* f) {
        pair(v.x, f), pair(v.y, f + 2), pair(v.z, f + 4), pair(v.w, f + 6);
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kVec = 8;
    __device__ __forceinline__ static float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    __device__ __forceinline__ static __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
    __device__ __forceinline__ static uint32_t two(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static uint4 pack(const float* f) {
        return make_uint4(two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7]));
    }
    __device__ __forceinline__ static void pair(uint32_t u, float* f) {
        f[0] = __uint_as_float(u << 16), f[1] = __uint_as_float(u & 0xffff0000u);
    }
    __device__ __forceinline__ static void unpack(const uint4& v, float* f) {
        pair(v.x, f), pair(v.y, f + 2), pair(v.z, f + 4), pair(v.w, f + 6);
    }
};

template <class T>
__device__ __forceinline__ T* row_at(const View& r, int64_t i) {
    const int64_t g = (uint32_t)i / (uint32_t)r.group;
    return static_cast<T*>(r.data) + g * r.group_stride + (i - g * r.group) * r.row_stride;
}

// A row as 16-byte vectors: vector j covers elements j V - off .. j V - off + V - 1, where off is the row's
// distance from the 16-byte boundary below it. Vectors that lie inside the row are read at once; the first
// and the last may hang over it and are read element by element, with -inf outside.
template <class T>
struct RowVecs {
    static constexpr int V = Elem<T>::kVec;
    const T* p;
    int off, M, n;
    __device__ __forceinline__ RowVecs(const T* row, int M_) : p(row), M(M_) {
        off = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
        n = (int)(((int64_t)M + off + V - 1) / V);
    }
    __device__ __forceinline__ int64_t first(int j) const { return (int64_t)j * V - off; }
    // vectors j0 .. j1 - 1 all lie inside the row
    __device__ __forceinline__ bool inside(int j0, int j1) const { return first(j0) >= 0 && first(j1) <= M; }
    __device__ __forceinline__ const uint4* at(int j) const { return reinterpret_cast<const uint4*>(p + first(j)); }
    __device__ __forceinline__ uint4 raw(int j) const { return __ldg(at(j)); }
    __device__ __forceinline__ void edge(int j, float* f) const {
        const int64_t e = first(j);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = (j < n && e + i >= 0 && e + i < M) ? Elem<T>::get(p[e + i]) : neg_inf();
    }
};

// 16 bytes from byte `shift` (0 .. 15, a multiple of 2) of the 32 bytes (a, b).
__device__ __forceinline__ uint4 window(const uint4& a, const uint4& b, int shift) {
    uint32_t w0 = a.x, w1 = a.y, w2 = a.z, w3 = a.w, w4 = b.x, w5 = b.y;
    if (shift & 8) w0 = a.z, w1 = a.w, w2 = b.x, w3 = b.y, w4 = b.z, w5 = b.w;
    if (shift & 4) w0 = w1, w1 = w2, w2 = w3, w3 = w4, w4 = w5;
    const int r = (shift & 2) * 8;
    return make_uint4(__funnelshift_r(w0, w1, r), __funnelshift_r(w1, w2, r), __funnelshift_r(w2, w3, r), __funnelshift_r(w3, w4, r));
}

// The threads that share a row: a warp (several rows a CTA), or the CTA. kThreads threads a CTA either way.
template <int TEAM>
struct Team {
    static constexpr int kPerCta = kThreads / TEAM;
    static constexpr bool kWarp = TEAM == 32;
    __device__ __forceinline__ static int id() { return kWarp ? threadIdx.x >> 5 : 0; }
    __device__ __forceinline__ static int tid() { return kWarp ? threadIdx.x & 31 : threadIdx.x; }
    __device__ __forceinline__ static void sync() {
        if (kWarp) __syncwarp();
        else __syncthreads();
    }
    __device__ __forceinline__ static bool any(bool v) { return kWarp ? __any_sync(~0u, v) : __syncthreads_or(v); }
    __device__ __forceinline__ static int count(bool v) { return kWarp ? __popc(__ballot_sync(~0u, v)) : __syncthreads_count(v); }
};

// Thread-block clusters: the CTAs of a cluster share one row, rank r the r-th slice of its vectors.
__device__ __forceinline__ int cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}
__device__ __forceinline__ int cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return (int)r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// the same shared-memory object in the CTA of another rank
template <class P>
__device__ __forceinline__ P* of_rank(P* p, int rank) {
    uint64_t a;
    asm("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<P*>(a);
}

struct Slice {
    int begin, end;  // vectors of the row
};
__device__ __forceinline__ Slice slice_of(int n, int rank, int parts) {
    const int per = (n + parts - 1) / parts;
    Slice s;
    s.begin = min(n, rank * per), s.end = min(n, s.begin + per);
    return s;
}

// Order of fp32 values as unsigned integers (-inf lowest); +0 and -0 are one value.
__device__ __forceinline__ uint32_t ord_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float of_ord(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
// (value, column) as one key: larger value first, then lower column.
__device__ __forceinline__ unsigned long long key_of(float v, int col) {
    return ((unsigned long long)ord_of(v) << 32) | (uint32_t)~(uint32_t)col;
}

struct State {
    float m = neg_inf();
    float s = 0.f, lo = 0.f;  // s + lo: the sum and what its additions rounded off
    float h = 0.f;

    // s + lo += v, exactly (Knuth's two-sum) but for lo's own rounding
    __device__ __forceinline__ void add(float v) {
        const float t = s + v, b = t - s;
        lo += (s - (t - b)) + (v - b);
        s = t;
    }
    // refer the sums to a larger maximum
    __device__ __forceinline__ void raise(float to, float c) {
        if (m != to) {
            // a sum of nothing stays nothing; a distance beyond 1e28 has weight 0 and must not make 0 x inf
            const float d = fmaxf(m - to, -1e28f);
            const float f = m == neg_inf() ? 0.f : ex2(d * c);
            h = f * fmaf(d, s, h);
            s *= f, lo *= f;
            m = to;
        }
    }
};

// n scores into the state.
template <int N>
__device__ __forceinline__ void add_scores(State& st, const float (&f)[N], float c) {
    float top = f[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = max_nan(top, f[i]);
    top = max_nan(top, st.m);
    if (top == neg_inf()) return;
    st.raise(top, c);
    float s[4] = {0.f, 0.f, 0.f, 0.f}, h[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float d = max_nan(f[i] - top, -1e30f);  // -inf (masked): weight 0 times a finite distance
        const float e = ex2(d * c);
        s[i & 3] += e;
        h[i & 3] = fmaf(e, d, h[i & 3]);
    }
    st.add((s[0] + s[1]) + (s[2] + s[3]));
    st.h += (h[0] + h[1]) + (h[2] + h[3]);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(~0u, v, o));
    return v;
}
// sum of the (already aligned) states of a warp, in every lane
__device__ __forceinline__ void warp_sum(State& st) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float s = __shfl_xor_sync(~0u, st.s, o), lo = __shfl_xor_sync(~0u, st.lo, o);
        st.h += __shfl_xor_sync(~0u, st.h, o);
        st.add(s);
        st.lo += lo;
    }
}

struct ReduceBuf {
    float m[kThreads / 32], s[kThreads / 32], lo[kThreads / 32], h[kThreads / 32];
};

// The state of all scores of the team, in every thread. A CTA's takes two barriers; the buffer may be used
// again after the caller's next one.
template <int TEAM>
__device__ __forceinline__ State team_state(State st, float c, ReduceBuf& b) {
    constexpr int W = TEAM / 32;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float wm = warp_max(st.m);
    if (W == 1) {
        st.raise(wm, c);
        warp_sum(st);
        return st;
    }
    if (lane == 0) b.m[w] = wm;
    __syncthreads();
    const float m = warp_max(b.m[lane < W ? lane : 0]);
    st.raise(m, c);
    warp_sum(st);
    if (lane == 0) b.s[w] = st.s, b.lo[w] = st.lo, b.h[w] = st.h;
    __syncthreads();
    st.s = lane < W ? b.s[lane] : 0.f, st.lo = lane < W ? b.lo[lane] : 0.f, st.h = lane < W ? b.h[lane] : 0.f;
    warp_sum(st);
    return st;
}

constexpr int kMaxCluster = 8;
struct ClusterBuf {
    float4 part[kMaxCluster];
};
// Every CTA's state to every CTA of the cluster; the caller then crosses a cluster barrier and merges.
__device__ __forceinline__ void cluster_share(const State& st, ClusterBuf& b, int rank, int size) {
    if ((int)threadIdx.x < size) of_rank(&b, threadIdx.x)->part[rank] = make_float4(st.m, st.s, st.lo, st.h);
}
__device__ __forceinline__ State cluster_merge(const ClusterBuf& b, int size, float c) {
    float m = b.part[0].x;
    for (int r = 1; r < size; ++r) m = max_nan(m, b.part[r].x);
    State all;
    all.m = m;
    for (int r = 0; r < size; ++r) {
        const float4 v = b.part[r];
        State p;
        p.m = v.x, p.s = v.y, p.lo = v.z, p.h = v.w;
        p.raise(m, c);
        all.add(p.s);
        all.lo += p.lo, all.h += p.h;
    }
    return all;
}

// c is rounded: the sum's first-order correction to the exact 1/T (see Scale in tp_logits_args.h)
__device__ __forceinline__ double exact_sum(const State& st, const Scale& sc) {
    return (double)st.s + ((double)st.lo + (double)sc.delta * st.h);
}

// ln z for z >= 2^-120 in fp64: an fp32 logarithm and one correction through the fp64 exponential,
// ln z = l + ln(z e^-l) with z e^-l within 1e-6 of 1. About 18 fp64 operations; the pipe has 2 lanes a clock.
__device__ __forceinline__ double ln64(double z) {
    const double l = (double)logf((float)z);
    const double r = fma(z, exp_table(-l), -1.0);
    return l + fma(-0.5 * r, r, r);
}

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// A teacher's list of one row in shared memory.
struct ListBuf {
    int id[kMaxList];
    float y[kMaxList], x[kMaxList];  // the teacher's value, the row's score
    float q[kMaxList];               // the teacher's share
    unsigned char first[kMaxList];   // no earlier entry has its column
    __device__ __forceinline__ bool ok(int k) const { return id[k] >= 0; }
};

// Loads the list of a row whose scores start at p; false when no entry counts. Scores are read of the columns
// from e0 to e1 only (what another CTA may be overwriting is its own to read). Ends with a barrier.
template <class T, int TEAM>
__device__ __forceinline__ bool load_list(const DistillArgs& a, int64_t row, const T* p, ListBuf& l, int64_t e0, int64_t e1) {
    bool some = false;
    for (int k = Team<TEAM>::tid(); k < a.K; k += TEAM) {
        const int64_t id = a.ids[row * a.K + k];
        const float y = a.values[row * a.K + k];
        const bool ok = id >= 0 && id < a.x.M && !(y == neg_inf());
        l.id[k] = ok ? (int)id : -1;
        l.y[k] = y;
        l.x[k] = ok && id >= e0 && id < e1 ? Elem<T>::get(p[id]) : 0.f;
        some |= ok;
    }
    if (!Team<TEAM>::any(some)) return false;
    Team<TEAM>::sync();
    return true;
}
// Marks the first entry of each column; true when a column is listed twice. Ends with a barrier.
template <int TEAM>
__device__ __forceinline__ bool mark_first(ListBuf& l, int K) {
    bool twice = false;
    for (int k = Team<TEAM>::tid(); k < K; k += TEAM) {
        bool first = true;
        for (int j = 0; j < k; ++j) first &= l.id[j] != l.id[k];
        l.first[k] = first;
        twice |= !first && l.ok(k);
    }
    twice = Team<TEAM>::any(twice);
    Team<TEAM>::sync();
    return twice;
}

struct RowStats {
    float loss;
    float m, ls;    // maximum and log of the sum relative to it, over all columns
    float gm, gls;  // the same over the columns that the list leaves (rest), else over all
    float Z;        // sum of the shares
    float coef;     // gradient of a column that is not listed: coef exp((x - gm)/T - gls) / T
};

// The list's part of a row, by one warp: the teacher's shares q (left in l.q), the loss, and what the gradient
// takes. `st` is the state of all columns, or of the unlisted ones (rest; l.first and every l.x are then
// read). In fp64: what is left of a loss near zero is the difference of logarithms that agree to several digits.
__device__ __forceinline__ RowStats distill_row(const DistillArgs& a, const State& st, ListBuf& l) {
    const int lane = threadIdx.x & 31;
    const double inv = a.sc.inv64;
    const double zs = exact_sum(st, a.sc);
    float m = st.m;  // maximum over all columns
    double z = zs;   // sum over all columns, relative to m
    double q[4], lq[4];
    if (a.rest) {
        float lm = neg_inf();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = lane + 32 * j;
            if (k < a.K && l.ok(k)) lm = max_nan(lm, l.x[k]);
        }
        m = max_nan(st.m, warp_max(lm));
        double sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = lane + 32 * j;
            const bool ok = k < a.K && l.ok(k);
            lq[j] = ok ? l.y[k] : 0.0;
            q[j] = ok ? exp_table(lq[j]) : 0.0;
            if (ok && l.first[k] && l.x[k] > neg_inf()) sum += exp_table(((double)l.x[k] - m) * inv);
        }
        z = warp_sum64(sum);
        if (st.m > neg_inf()) z += zs * exp_table(((double)st.m - m) * inv);
        if (m != m) z = m;  // NaN
    } else {
        float ym = neg_inf();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = lane + 32 * j;
            if (k < a.K && l.ok(k)) ym = max_nan(ym, l.y[k]);
        }
        ym = warp_max(ym);
        double sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = lane + 32 * j;
            const bool ok = k < a.K && l.ok(k);
            lq[j] = ok ? ((double)l.y[k] - ym) * inv : 0.0;
            q[j] = ok ? exp_table(lq[j]) : 0.0;
            sum += q[j];
        }
        sum = warp_sum64(sum);
        const double ln = ln64(sum), r = 1.0 / sum;
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] *= r, lq[j] -= ln;
    }
    const double m0 = m == neg_inf() ? 0.0 : (double)m, ls = m == neg_inf() ? 0.0 : ln64(z);
    double loss = 0, Z = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = lane + 32 * j;
        if (q[j] > 0) loss += q[j] * (lq[j] - (((double)l.x[k] - m0) * inv - ls));
        Z += q[j];
        if (k < a.K) l.q[k] = (float)q[j];
    }
    loss = warp_sum64(loss), Z = warp_sum64(Z);
    RowStats s;
    s.m = s.gm = m, s.ls = s.gls = (float)ls, s.coef = (float)Z;
    if (a.rest) {
        s.coef = 0.f;
        if (st.m != neg_inf()) {
            const double q_r = 1.0 - Z >= kLeastRest ? 1.0 - Z : 0.0, lr = ln64(zs), lp = ((double)st.m - m0) * inv + lr - ls;
            if (q_r > 0) loss += q_r * (ln64(q_r) - lp);
            Z += q_r;
            s.gm = st.m, s.gls = (float)lr, s.coef = (float)(Z * exp_table(lp) - q_r);
        }
    }
    s.Z = (float)Z, s.loss = (float)loss;
    return s;
}

}  // namespace rows
}  // namespace tp
