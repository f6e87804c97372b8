// Writing a gradient row: 16-byte vectors of the gradient's own alignment, whatever the scores' is.
#pragma once

#include "tp_logits.cuh"

namespace tp {
namespace rows {

// The row o as 16-byte vectors (RowVecs): how many, and the first element of the j-th.
template <class T>
__device__ __forceinline__ int off_of(const T* o) {
    return (int)((reinterpret_cast<uintptr_t>(o) & 15u) / sizeof(T));
}
template <class T>
__device__ __forceinline__ int vecs_of(const T* o, int M) {
    constexpr int V = Elem<T>::kVec;
    return (int)(((int64_t)M + off_of(o) + V - 1) / V);
}
template <class T>
__device__ __forceinline__ int64_t first_of(const T* o, int j) {
    return (int64_t)j * Elem<T>::kVec - off_of(o);
}

// o[e] = f(score e) for e0 <= e < e1. from.get(e, v) fetches V adjacent scores, or declines; from.one(e) fetches
// one. f(float[V], e) turns the scores of e .. e + V - 1 into gradients. A vector that e0 or e1 cuts is written
// element by element: what lies beyond may be another CTA's.
template <class T, int TEAM, class From, class F>
__device__ __forceinline__ void map_range(T* o, int64_t e0, int64_t e1, const From& from, F f) {
    constexpr int V = Elem<T>::kVec;
    const int off = off_of(o);
    const int end = (int)((e1 + off + V - 1) / V);
    for (int base = (int)((e0 + off) / V) + Team<TEAM>::tid(); base < end; base += TEAM * kUnroll) {
        uint4 r[kUnroll];
        bool got[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t e = first_of(o, base + u * TEAM);
            got[u] = e >= e0 && e + V <= e1 && from.get(e, r[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t e = first_of(o, base + u * TEAM);
            if (e >= e1) break;
            float v[V];
            if (got[u]) {
                Elem<T>::unpack(r[u], v);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = e + i >= e0 && e + i < e1 ? from.one(e + i) : neg_inf();
            }
            f(v, e);
            if (e >= e0 && e + V <= e1) {
                __stcs(reinterpret_cast<uint4*>(o + e), Elem<T>::pack(v));
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e + i >= e0 && e + i < e1) o[e + i] = Elem<T>::put(v[i]);
            }
        }
    }
}

struct Nothing {
    __device__ __forceinline__ bool get(int64_t, uint4& v) const {
        v = make_uint4(0, 0, 0, 0);
        return true;
    }
    __device__ __forceinline__ float one(int64_t) const { return 0.f; }
};
template <class T, int TEAM>
__device__ __forceinline__ void zero_range(T* o, int64_t e0, int64_t e1) {
    map_range<T, TEAM>(o, e0, e1, Nothing(), [](float* f, int64_t) {
#pragma unroll
        for (int i = 0; i < Elem<T>::kVec; ++i) f[i] = 0.f;
    });
}

// The elements of a part of the row o: whole vectors of it, but at the row's ends.
struct Range {
    int64_t e0, e1;
};
template <class T>
__device__ __forceinline__ Range range_of(const T* o, int M, int rank, int parts) {
    const Slice s = slice_of(vecs_of(o, M), rank, parts);
    return Range{max(first_of(o, s.begin), (int64_t)0), min(first_of(o, s.end), (int64_t)M)};
}

// The teacher's shares into l.q, by one warp (what distill_row leaves there, in fp32).
__device__ __forceinline__ void shares(const DistillArgs& a, ListBuf& l) {
    const int lane = threadIdx.x & 31;
    float y[4], top = a.rest ? 0.f : neg_inf(), sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = lane + 32 * j;
        y[j] = k < a.K && l.ok(k) ? l.y[k] : neg_inf();
        if (!a.rest) top = max_nan(top, y[j]);
    }
    if (!a.rest) top = warp_max(top);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        y[j] = expf(a.rest ? y[j] : (y[j] - top) * a.sc.inv);
        sum += y[j];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (lane + 32 * j < a.K) l.q[lane + 32 * j] = a.rest ? y[j] : y[j] / sum;
}

// Gradient of the columns from e0 to e1 as if none were listed; w: the row's weight over T.
template <class T, int TEAM, class From>
__device__ __forceinline__ void distill_row_grad(const DistillArgs& a, const RowStats& s, float w, T* o, int64_t e0,
                                                 int64_t e1, const From& from) {
    const float coef = s.coef * w, gm = s.gm, gls2 = s.gls * kLog2e, c = a.sc.c;
    map_range<T, TEAM>(o, e0, e1, from, [&](float* f, int64_t) {
#pragma unroll
        for (int i = 0; i < Elem<T>::kVec; ++i) f[i] = coef * ex2(fmaf(f[i] - gm, c, -gls2));
    });
}
// and of the listed columns from e0 to e1, after a barrier.
template <class T, int TEAM>
__device__ __forceinline__ void distill_list_grad(const DistillArgs& a, const RowStats& s, float w, T* o, int64_t e0,
                                                  int64_t e1, const ListBuf& l, bool twice) {
    for (int k = Team<TEAM>::tid(); k < a.K; k += TEAM) {
        if (!l.ok(k) || !l.first[k] || l.id[k] < e0 || l.id[k] >= e1) continue;
        float q = l.q[k];
        if (twice)
            for (int j = k + 1; j < a.K; ++j)
                if (l.id[j] == l.id[k]) q += l.q[j];
        o[l.id[k]] = Elem<T>::put(w * (s.Z * expf((l.x[k] - s.m) * a.sc.inv - s.ls) - q));
    }
}

}  // namespace rows
}  // namespace tp
