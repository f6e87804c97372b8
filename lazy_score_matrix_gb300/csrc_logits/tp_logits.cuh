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
#include "tp_logits_two.cuh"

namespace tp {
namespace rows {

constexpr int kThreads = 256;      // per CTA
constexpr int kLongThreads = 512;  // where a row is read twice (fewer rows under way, for the second reading to hit
                                   // the cache), and of clusters (few rows)
constexpr int kUnroll = 4;         // 16-byte vectors of a thread's chunk
constexpr int kAhead = 2;          // chunks that are brought into the L2 cache ahead of a thread's loads
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float lowest() { return __uint_as_float(0xff7fffffu); }
__device__ __forceinline__ float ex2(float x) { return ExpTraits<float>::bexp(x); }
// maximum that keeps a NaN of either operand, so that a NaN score reaches the row's results
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Two fp32 values in one register pair: one instruction for both.
__device__ __forceinline__ float2 sub2(float2 a, float b) {
    float2 r;
    const float2 m = make_float2(-b, -b);
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(m)));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float b) {
    float2 r;
    const float2 m = make_float2(b, b);
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(m)));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
          "l"(reinterpret_cast<const uint64_t&>(c)));
    return r;
}

template <class T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kVec = 4;  // elements of a 16-byte vector
    __device__ __forceinline__ static float get(float v) { return v; }
    __device__ __forceinline__ static float put(float v) { return v; }
    // whether an element of r reaches a bar
    __device__ __forceinline__ static float bar(float v) { return v; }
    __device__ __forceinline__ static bool reaches(const uint4& r, float b) {
        return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w))) >= b;
    }
    __device__ __forceinline__ static uint4 none() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
    template <int N>
    __device__ __forceinline__ static float top(const uint4 (&r)[N]) {
        float m = neg_inf();
#pragma unroll
        for (int u = 0; u < N; ++u)
            m = max_nan(max_nan(m, max_nan(__uint_as_float(r[u].x), __uint_as_float(r[u].y))),
                        max_nan(__uint_as_float(r[u].z), __uint_as_float(r[u].w)));
        return m;
    }
    __device__ __forceinline__ static uint4 pack(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    __device__ __forceinline__ static void unpack(const uint4& v, float* f) {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    }
    __device__ __forceinline__ static void minus(const uint4& v, float m, float* f) {
        unpack(v, f);
        const float2 a = sub2(make_float2(f[0], f[1]), m), b = sub2(make_float2(f[2], f[3]), m);
        f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
    }
};
template <>
struct Elem<__half> {
    static constexpr int kVec = 8;
    __device__ __forceinline__ static float get(__half v) { return __half2float(v); }
    __device__ __forceinline__ static uint4 none() { return make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u); }
    // largest element, two at a time; NaN if there is one
    template <int N>
    __device__ __forceinline__ static float top(const uint4 (&r)[N]) {
        __half2 m = of(r[0].x);
#pragma unroll
        for (int u = 0; u < N; ++u)
            m = __hmax2_nan(__hmax2_nan(m, __hmax2_nan(of(r[u].x), of(r[u].y))), __hmax2_nan(of(r[u].z), of(r[u].w)));
        return max_nan(__half2float(__low2half(m)), __half2float(__high2half(m)));
    }
    // the smallest value of the type that reaches v, twice
    __device__ __forceinline__ static __half2 bar(float v) { return __half2half2(__float2half_ru(v)); }
    __device__ __forceinline__ static bool reaches(const uint4& r, __half2 b) {
        return (__hge2_mask(of(r.x), b) | __hge2_mask(of(r.y), b) | __hge2_mask(of(r.z), b) | __hge2_mask(of(r.w), b)) != 0;
    }
    __device__ __forceinline__ static __half2 of(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
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
    // x - m in fp32, straight from the two halves of a word
    __device__ __forceinline__ static void minus(const uint4& v, float m, float* f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n sub.rn.f32.f16 %0, lo, %3;\n sub.rn.f32.f16 %1, hi, %3;\n}"
                : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
                : "r"(w[i]), "f"(m));
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kVec = 8;
    __device__ __forceinline__ static float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    __device__ __forceinline__ static uint4 none() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
    // largest element, two at a time; NaN if there is one
    template <int N>
    __device__ __forceinline__ static float top(const uint4 (&r)[N]) {
        __nv_bfloat162 m = of(r[0].x);
#pragma unroll
        for (int u = 0; u < N; ++u)
            m = __hmax2_nan(__hmax2_nan(m, __hmax2_nan(of(r[u].x), of(r[u].y))), __hmax2_nan(of(r[u].z), of(r[u].w)));
        return max_nan(__bfloat162float(__low2bfloat16(m)), __bfloat162float(__high2bfloat16(m)));
    }
    // the smallest value of the type that reaches v, twice
    __device__ __forceinline__ static __nv_bfloat162 bar(float v) { return __bfloat162bfloat162(__float2bfloat16_ru(v)); }
    __device__ __forceinline__ static bool reaches(const uint4& r, __nv_bfloat162 b) {
        return (__hge2_mask(of(r.x), b) | __hge2_mask(of(r.y), b) | __hge2_mask(of(r.z), b) | __hge2_mask(of(r.w), b)) != 0;
    }
    __device__ __forceinline__ static __nv_bfloat162 of(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); }
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
    // x - m in fp32, straight from the two halves of a word
    __device__ __forceinline__ static void minus(const uint4& v, float m, float* f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n sub.rn.f32.bf16 %0, lo, %3;\n sub.rn.f32.bf16 %1, hi, %3;\n}"
                : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
                : "r"(w[i]), "f"(m));
    }
};

template <class T>
__device__ __forceinline__ T* row_at(const View& r, int64_t i) {
    T* p = static_cast<T*>(r.data);
    if (!r.grouped) return p + i * r.row_stride;
    const int64_t g = (uint32_t)i / (uint32_t)r.group;
    return p + g * r.group_stride + (i - g * r.group) * r.row_stride;
}

// A row as 16-byte vectors: vector j covers elements j V - off .. j V - off + V - 1, where off is the row's
// distance from the 16-byte boundary below it. The first and the last may hang over the row's ends: those are
// read element by element, with -inf outside. (M <= 2^30, so every index fits 32 bits.)
template <class T>
struct RowVecs {
    static constexpr int V = Elem<T>::kVec;
    const T* p;
    const uint4* base;  // the boundary below the row
    int off, M, n;
    int lo, hi;  // vectors lo .. hi - 1 lie inside the row
    __device__ __forceinline__ RowVecs(const T* row, int M_) : p(row), M(M_) {
        off = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
        base = reinterpret_cast<const uint4*>(row - off);
        n = (M + off + V - 1) / V;
        lo = off ? 1 : 0, hi = (M + off) / V;
    }
    __device__ __forceinline__ int first(int j) const { return j * V - off; }
    __device__ __forceinline__ bool inside(int j) const { return j >= lo && j < hi; }
    __device__ __forceinline__ uint4 edge(int j) const {
        const int e = first(j);
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = (e + i >= 0 && e + i < M) ? Elem<T>::get(p[e + i]) : neg_inf();
        return Elem<T>::pack(f);
    }
    // Has a chunk of `step` vectors brought into the L2 cache, kAhead chunks behind the one at j; kAhead chunks from j on
    // where `first`. By one thread, in bulk: what is under way from memory then does not have to fit the
    // registers, and a load that follows waits for the cache only. Two chunks (16 KB each) ahead: 4096 rows of
    // 131072 bf16 took 173 us without, 166 with one or two, 171 with four and 206 with eight, when what is ahead on
    // the whole card falls out of the cache again.
    __device__ __forceinline__ void ahead(int j, int step, int end, bool first = false) const {
        const int j0 = max(first ? j : j + kAhead * step, lo), j1 = min(min(j + (kAhead + (first ? 0 : 1)) * step, hi), end);
        if (j0 < j1)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(base + j0), "r"((j1 - j0) * 16) : "memory");
    }
    // vectors from + u step, u < N; -inf from `end` on
    template <int N>
    __device__ __forceinline__ void load(uint4 (&r)[N], int from, int step, int end) const {
        if (from >= lo && from + (N - 1) * step < min(end, hi)) {  // no branch between the loads
#pragma unroll
            for (int u = 0; u < N; ++u) r[u] = __ldcg(base + from + u * step);
            return;
        }
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int j = from + u * step;
            if (j < end && inside(j)) r[u] = __ldcg(base + j);
            else if (j < end) r[u] = edge(j);
            else r[u] = Elem<T>::none();
        }
    }
};

// Brings the first chunks of a later row into the L2 cache: the one whose CTA takes this one's place on the SM.
template <class T>
__device__ __forceinline__ void begin_row(const View& v, int64_t N, int64_t row, int step) {
    if (row >= N) return;
    const RowVecs<T> x(row_at<const T>(v, row), v.M);
    x.ahead(0, step, x.n, true);
}

// 16 bytes from byte `shift` (0 .. 15, a multiple of 2) of the 32 bytes (a, b).
__device__ __forceinline__ uint4 window(const uint4& a, const uint4& b, int shift) {
    uint32_t w0 = a.x, w1 = a.y, w2 = a.z, w3 = a.w, w4 = b.x, w5 = b.y;
    if (shift & 8) w0 = a.z, w1 = a.w, w2 = b.x, w3 = b.y, w4 = b.z, w5 = b.w;
    if (shift & 4) w0 = w1, w1 = w2, w2 = w3, w3 = w4, w4 = w5;
    const int r = (shift & 2) * 8;
    return make_uint4(__funnelshift_r(w0, w1, r), __funnelshift_r(w1, w2, r), __funnelshift_r(w2, w3, r), __funnelshift_r(w3, w4, r));
}

// The threads that share a row: a warp (kThreads / 32 rows a CTA), or a CTA of TEAM threads.
template <int TEAM>
struct Team {
    static constexpr int kPerCta = TEAM == 32 ? kThreads / 32 : 1;
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

// N vectors of scores into the state. Instructions for two 16-bit scores: one maximum, two of x - m, one product with c,
// two ex2, one sum s; about 8 a score with the loads and the loop. MOMENT: h too; a masked score's distance (-inf) is bounded, as its weight 0 times
// it would be NaN. Without h, the product is formed with both words of c instead (c_lo > 0, so that -inf stays).
// Returns the largest of them.
template <class T, bool MOMENT, int N>
__device__ __forceinline__ float add_scores(State& st, const uint4 (&r)[N], const Scale& sc) {
    constexpr int V = Elem<T>::kVec;
    const float here = Elem<T>::top(r), top = max_nan(here, st.m);
    if (top == neg_inf()) return here;
    st.raise(top, sc.c);
    float2 s[2], h[2];
    s[0] = s[1] = h[0] = h[1] = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < N; ++u) {
        float f[V];
        Elem<T>::minus(r[u], top, f);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const int k = i / 2 & 1;
            float2 d = make_float2(f[i], f[i + 1]), x;
            if (MOMENT) {
                d = make_float2(max_nan(d.x, -1e30f), max_nan(d.y, -1e30f));
                x = mul2(d, sc.c);
            } else {
                x = fma2(d, make_float2(sc.c_lo, sc.c_lo), mul2(d, sc.c_hi));
            }
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            s[k] = add2(s[k], e);
            if (MOMENT) h[k] = fma2(e, d, h[k]);
        }
    }
    const float2 sum = add2(s[0], s[1]);
    st.add(sum.x + sum.y);
    if (MOMENT) h[0] = add2(h[0], h[1]), st.h += h[0].x + h[0].y;
    return here;
}

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
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
    float m[32], s[32], lo[32], h[32];
};

// The state of all scores of the team, in every thread of its first warp; the others have its maximum. A CTA's
// takes two barriers; the buffer may be used again after the caller's next one.
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
    if (w != 0) return st;
    st.s = lane < W ? b.s[lane] : 0.f, st.lo = lane < W ? b.lo[lane] : 0.f, st.h = lane < W ? b.h[lane] : 0.f;
    warp_sum(st);
    return st;
}

constexpr int kMaxCluster = 8;
struct ClusterBuf {
    float4 part[kMaxCluster];
};
// Every CTA's state to every CTA of the cluster (by its first warp); the caller then crosses a cluster barrier and
// merges.
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

// r with the elements whose bits are set masked (few vectors have any)
template <class T>
__device__ __forceinline__ uint4 without(const uint4& r, uint32_t bits) {
    constexpr int V = Elem<T>::kVec;
    if (!(bits & ((1u << V) - 1))) return r;
    float f[V];
    Elem<T>::unpack(r, f);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (bits & (1u << i)) f[i] = neg_inf();
    return Elem<T>::pack(f);
}

// What a row's loss takes from the list alone. lm is the largest listed score (0 if all are -inf).
struct ListSums {
    Two Z;      // sum of the shares
    Two zl;     // rest: sum over the listed columns, each once, of exp((x - lm)/T)
    Two q_r_ln;
    Two ln;     // log of what the entries' q are divided by to become shares (rest: 0)
    float scale, q_r, lm;  // scale: the shares are scale q
};

// A teacher's list of one row in shared memory.
struct ListBuf {
    alignas(16) int id[kMaxList];    // -1: the entry does not count
    float y[kMaxList], x[kMaxList];  // the teacher's value, the row's score
    float q[kMaxList], q_lo[kMaxList];  // the teacher's share before it is scaled, two words
    float2 u[kMaxList];              // log q - (x - lm)/T, two words
    float2 z[kMaxList];              // rest: exp((x - lm)/T), two words; 0 for a column listed before
    ListSums sums;
    unsigned char first[kMaxList];   // no earlier entry has its column
    __device__ __forceinline__ bool ok(int k) const { return id[k] >= 0; }
};

// Loads a row's list; false when no entry counts. Ends with a barrier.
template <int TEAM>
__device__ __forceinline__ bool load_list(const DistillArgs& a, int64_t row, ListBuf& l) {
    bool some = false;
    for (int k = Team<TEAM>::tid(); k < a.K; k += TEAM) {
        const int64_t id = a.ids[row * a.K + k];
        const float y = a.values[row * a.K + k];
        const bool ok = id >= 0 && id < a.x.M && !(y == neg_inf());
        l.id[k] = ok ? (int)id : -1;
        l.y[k] = y;
        some |= ok;
    }
    if (!Team<TEAM>::any(some)) return false;
    Team<TEAM>::sync();
    return true;
}
// Scores of the listed columns from e0 to e1 (what another CTA may be overwriting is its own to read) of the row
// at p, and the first entry of each column; true when a column is listed twice. Ends with a barrier.
template <class T, int TEAM>
__device__ __forceinline__ bool look_up(const DistillArgs& a, const T* p, ListBuf& l, int e0, int e1) {
    bool twice = false;
    for (int k = Team<TEAM>::tid(); k < a.K; k += TEAM) {
        const int id = l.id[k];
        const float x = id >= e0 && id < e1 && id >= 0 ? Elem<T>::get(p[id]) : 0.f;
        bool first = true;
        int j = 0;
        for (; j + 4 <= k; j += 4) {
            const int4 v = *reinterpret_cast<const int4*>(l.id + j);
            first &= v.x != id && v.y != id && v.z != id && v.w != id;
        }
        for (; j < k; ++j) first &= l.id[j] != id;
        l.first[k] = first;
        twice |= !first && id >= 0;
        l.x[k] = x;
    }
    twice = Team<TEAM>::any(twice);
    Team<TEAM>::sync();
    return twice;
}

// (x - m)/T; one word where it is -inf, or as good as. That word may be -inf for a finite x (the lowest value over T < 1),
// so what goes on to a sum is asked far_below first.
__device__ __forceinline__ Two over_T(float x, float m, const Scale& sc) {
    const float d = x - m;
    if (!(d > -1e30f)) return Two{d * sc.inv, 0.f};
    return mul(two_sum(x, -m), Two{sc.inv, sc.inv_lo});
}
// Whether x lies so far below a finite maximum m that its distance is all that counts beside logarithms of sums (and
// its probability is 0); false where either is NaN.
__device__ __forceinline__ bool far_below(float x, float m) { return x - m <= -1e30f && m < __int_as_float(0x7f800000); }
// q (m - x)/T 2^-64 for such an x and q > 0: neither the distance nor its quotient needs to be in fp32's range, where the
// product is. +inf for a masked x.
__device__ __forceinline__ float far_term(const Two& q, float x, float m, const Scale& sc) {
    if (x == neg_inf()) return -x;
    return mul(q, mul(two_sum(m * 0x1p-64f, -x * 0x1p-64f), Two{sc.inv, sc.inv_lo})).h;
}

// The list's sums into l.sums, and its entries' q and u; by the warps that hold an entry a thread, whose first does the
// sums, while the others go on to the row (a named barrier holds only those warps). With one warp for all of it, the
// team waited for that warp at the end of the row: 3000 x 150016 bf16 with 128 entries took 351 us, and 347 so.
template <int TEAM>
__device__ __forceinline__ void sum_list(const DistillArgs& a, ListBuf& l) {
    const int lane = threadIdx.x & 31, w = TEAM == 32 ? 0 : threadIdx.x >> 5, warps = TEAM == 32 ? 1 : (a.K + 31) / 32;
    if (w >= warps) return;
    float lm = neg_inf(), ym = neg_inf();
    for (int k = lane; k < a.K; k += 32)
        if (l.ok(k)) lm = max_nan(lm, l.x[k]), ym = max_nan(ym, l.y[k]);
    lm = warp_max(lm);
    if (lm == neg_inf()) lm = 0.f;
    if (!a.rest) ym = warp_max(ym);
    for (int k = Team<TEAM>::tid(); k < a.K; k += TEAM) {
        Two q{0.f, 0.f}, z{0.f, 0.f}, u{0.f, 0.f};
        if (l.ok(k)) {
            const Two lq = a.rest ? Two{l.y[k], 0.f} : over_T(l.y[k], ym, a.sc), d = over_T(l.x[k], lm, a.sc);
            q = exp_two(lq);
            if (a.rest && l.first[k]) z = exp_two(d);
            u = d.h == neg_inf() ? Two{-d.h, 0.f} : add(lq, neg(d));
        }
        l.q[k] = q.h, l.q_lo[k] = q.l;
        l.u[k] = make_float2(u.h, u.l), l.z[k] = make_float2(z.h, z.l);
    }
    if (warps > 1) asm volatile("bar.sync 1, %0;" ::"r"(warps * 32) : "memory");
    else __syncwarp();
    if (w != 0) return;
    Two sum{0.f, 0.f}, zl{0.f, 0.f};
    for (int k = lane; k < a.K; k += 32) {
        sum = add(sum, Two{l.q[k], l.q_lo[k]});
        if (a.rest) zl = add(zl, Two{l.z[k].x, l.z[k].y});
    }
    sum = warp_add(sum);
    if (a.rest) zl = warp_add(zl);
    ListSums r;
    r.lm = lm, r.zl = zl, r.Z = sum, r.ln = r.q_r_ln = Two{0.f, 0.f}, r.scale = 1.f, r.q_r = 0.f;
    if (a.rest) {
        const Two left = add(Two{1.f, 0.f}, neg(sum));
        if (left.h >= kLeastRest) r.q_r = left.h, r.q_r_ln = ln_two(left);
    } else {
        r.ln = ln_two(sum), r.scale = 1.f / sum.h, r.Z = Two{1.f, 0.f};
    }
    if (lane == 0) l.sums = r;
    __syncwarp();
}

// Unlisted columns are told by a bit map of this many columns of the row at a time.
template <int TEAM>
struct Marks {
    static constexpr int kCols = TEAM == 32 ? 1 << 12 : 1 << 18;
    alignas(16) uint32_t bits[kCols / 32];
    // bit i < n of the map becomes: element e0 + i is listed. Barriers on both sides.
    __device__ __forceinline__ void set(const ListBuf& l, int K, int e0, int n) {
        Team<TEAM>::sync();
        for (int i = Team<TEAM>::tid(); i < (n + 127) / 128; i += TEAM) reinterpret_cast<uint4*>(bits)[i] = make_uint4(0, 0, 0, 0);
        Team<TEAM>::sync();
        for (int k = Team<TEAM>::tid(); k < K; k += TEAM) {
            const int at = l.ok(k) ? l.id[k] - e0 : -1;
            if (at >= 0 && at < n) atomicOr(&bits[at >> 5], 1u << (at & 31));
        }
        Team<TEAM>::sync();
    }
};

// The thread's state of the slice's columns; of the unlisted ones where REST. next: the thread's first chunk.
template <class T, int TEAM, bool REST>
__device__ __forceinline__ State read_slice(const DistillArgs& a, const RowVecs<T>& x, const Slice& sl, const ListBuf& list,
                                            Marks<TEAM>& marks, uint4 (&next)[kUnroll]) {
    constexpr int V = Elem<T>::kVec, kMarkVecs = Marks<TEAM>::kCols / V;
    const int t = Team<TEAM>::tid();
    State st;
    for (int part = sl.begin; part < sl.end; part += REST ? kMarkVecs : sl.end) {
        const int end = REST ? min(sl.end, part + kMarkVecs) : sl.end;
        if (part != sl.begin) x.load(next, part + t, TEAM, end);
        if (REST) marks.set(list, a.K, x.first(part), (end - part) * V);
        for (int base = part; base < end; base += TEAM * kUnroll) {
            uint4 r[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) r[u] = next[u];
            if (base + TEAM * kUnroll < end) x.load(next, base + TEAM * kUnroll + t, TEAM, end);  // under way while this one is reduced
            if (TEAM != 32 && t == 0) x.ahead(base + TEAM * kUnroll, TEAM * kUnroll, sl.end);
            if (REST) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int bit = (base - part + u * TEAM + t) * V & (Marks<TEAM>::kCols - 1);
                    r[u] = without<T>(r[u], marks.bits[bit >> 5] >> (bit & 31));
                }
            }
            add_scores<T, false>(st, r, a.sc);
        }
    }
    return st;
}

struct RowStats {
    float loss;
    float m, ls;    // maximum and log of the sum relative to it, over all columns
    float gm, gls;  // the same over the columns that the list leaves (rest), else over all
    float Z;        // sum of the shares
    float coef;     // gradient of a column that is not listed: coef exp((x - gm)/T - gls) / T
};

// The row's loss and what its gradient takes, by the warp that summed the list. `st` is the state of all columns,
// or of the unlisted ones (rest).
__device__ __forceinline__ RowStats close_row(const DistillArgs& a, const State& st, const ListBuf& b) {
    const ListSums& l = b.sums;
    const Two zs = two_sum(st.s, st.lo);
    float m = st.m;  // maximum over all columns
    Two z = zs;      // sum over all columns, relative to m
    if (a.rest && l.zl.h > 0.f) {
        m = max_nan(st.m, l.lm);
        z = mul(l.zl, exp_two(over_T(l.lm, m, a.sc)));
        if (st.m != neg_inf()) z = add(z, mul(zs, exp_two(over_T(st.m, m, a.sc))));
    }
    const bool some = m != neg_inf();
    const Two ls = some ? ln_two(z) : Two{0.f, 0.f};
    // scale sum q (log q - (x - lm)/T + c), c = ln z - (lm - m)/T - ln of the q's sum; c is of use unless all of the list
    // is far below m
    const Two c = add(add(ls, neg(over_T(l.lm, some ? m : 0.f, a.sc))), neg(l.ln));
    float loss = 0.f, far = 0.f;
    for (int k = threadIdx.x & 31; k < a.K; k += 32)
        if (!(b.q[k] <= 0.f)) {  // a NaN among the teacher's values shows
            const Two u{b.u[k].x, b.u[k].y};
            if (far_below(b.x[k], m)) far += far_term(Two{b.q[k], b.q_lo[k]}, b.x[k], m, a.sc);
            else loss += b.q[k] * (u.h < __int_as_float(0x7f800000) ? add(u, c).h : u.h);
        }
#pragma unroll
    for (int o = 16; o; o >>= 1) loss += __shfl_xor_sync(~0u, loss, o);
    loss *= l.scale;
    if (__any_sync(~0u, far != 0.f)) {
#pragma unroll
        for (int o = 16; o; o >>= 1) far += __shfl_xor_sync(~0u, far, o);
        loss += far * l.scale * 0x1p64f;
    }
    RowStats s;
    s.m = s.gm = m, s.ls = s.gls = ls.h, s.coef = l.Z.h, s.Z = l.Z.h;
    if (a.rest) {
        s.coef = 0.f;
        if (st.m != neg_inf()) {
            const Two lr = ln_two(zs), Z = add(l.Z, Two{l.q_r, 0.f});
            s.gm = st.m, s.gls = lr.h, s.Z = Z.h;
            if (far_below(st.m, m)) {  // p_r = 0
                if (l.q_r > 0.f) loss += far_term(Two{l.q_r, 0.f}, st.m, m, a.sc) * 0x1p64f;
                s.coef = -l.q_r;
            } else {
                const Two lp = add(add(over_T(st.m, m, a.sc), lr), neg(ls));  // log p_r
                if (l.q_r > 0.f) loss += l.q_r * add(l.q_r_ln, neg(lp)).h;
                s.coef = add(mul(Z, exp_two(lp)), Two{-l.q_r, 0.f}).h;
            }
        }
    }
    if (!(m < __int_as_float(0x7f800000))) loss = m - m;  // NaN
    s.loss = loss;
    return s;
}

}  // namespace rows
}  // namespace tp
