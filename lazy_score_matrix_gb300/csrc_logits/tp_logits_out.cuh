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
    return (M + off_of(o) + Elem<T>::kVec - 1) / Elem<T>::kVec;
}
template <class T>
__device__ __forceinline__ int first_of(const T* o, int j) {
    return j * Elem<T>::kVec - off_of(o);
}

// Where a gradient row finds its scores, in vectors of the gradient's alignment: vector j is bytes shift ..
// shift + 15 of (q[j], q[j + 1]), for lo <= j < hi; element e is p[e].
template <class T>
struct Source {
    const T* p;
    const uint4* q;
    int shift, lo, hi;
    __device__ __forceinline__ uint4 get(int j) const {
        if (shift) return window(q[j], q[j + 1], shift);  // neighbours read the same bytes: cached
        return __ldcs(q + j);
    }
};

// The scores of a row in memory. Plain loads, not .nc: the gradient may overwrite the scores.
template <class T>
__device__ __forceinline__ Source<T> from_row(const T* p, int M, const T* o) {
    constexpr int V = Elem<T>::kVec;
    Source<T> s;
    const int off = off_of(o);
    const uintptr_t at = reinterpret_cast<uintptr_t>(p - off);  // score of the gradient's element -off
    s.p = p;
    s.shift = (int)(at & 15u);
    s.q = reinterpret_cast<const uint4*>(at - s.shift);
    // the first byte of q[lo] and the last of q[hi - 1 + (shift != 0)] belong to the row
    const int back = s.shift / (int)sizeof(T);
    s.lo = (off + back + V - 1) / V;
    s.hi = (M + off + back) / V - (s.shift ? 1 : 0);
    return s;
}

// The whole vectors of a range of the gradient row o, and the first chunk of their scores, under way. AHEAD: the chunks
// after it are brought into the L2 cache in bulk (RowVecs::ahead); not for scores that lie there already.
template <class T, int TEAM, bool AHEAD>
struct Fetch {
    static constexpr int V = Elem<T>::kVec;
    const Source<T>& from;
    int off, ja, jb;
    uint4 next[kUnroll];
    __device__ __forceinline__ Fetch(const T* o, int e0, int e1, const Source<T>& from_) : from(from_), off(off_of(o)) {
        ja = max((e0 + off + V - 1) / V, from.lo), jb = max(ja, min((e1 + off) / V, from.hi));
        load(ja + Team<TEAM>::tid());
        ahead(ja, ja + TEAM * kUnroll);
    }
    // vectors j - TEAM kUnroll + kAhead chunks on, or those from `from_j` to there
    __device__ __forceinline__ void ahead(int j, int from_j) const {
        if (!AHEAD || TEAM == 32 || threadIdx.x != 0) return;
        const int j1 = min(j + (1 + kAhead) * TEAM * kUnroll, jb);
        if (from_j < j1)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from.q + from_j), "r"((j1 - from_j) * 16) : "memory");
    }
    __device__ __forceinline__ void load(int j) {
        if (j + (kUnroll - 1) * TEAM < jb) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) next[u] = from.get(j + u * TEAM);
        } else {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (j + u * TEAM < jb) next[u] = from.get(j + u * TEAM);
        }
    }
};

// o[e] = f(score e) for e0 <= e < e1. f(float[V], e) turns the scores of e .. e + V - 1 into gradients. Whole
// vectors are written as such; what e0, e1 or the source's ends cut is done element by element.
template <class T, int TEAM, bool AHEAD, class F>
__device__ __forceinline__ void map_range(T* o, int e0, int e1, Fetch<T, TEAM, AHEAD>& x, F f) {
    constexpr int V = Elem<T>::kVec;
    const int off = x.off, t = Team<TEAM>::tid(), ja = x.ja, jb = x.jb;
    const Source<T>& from = x.from;
    uint4* out = reinterpret_cast<uint4*>(o - off);
    for (int j = ja + t; j < jb; j += TEAM * kUnroll) {
        uint4 r[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) r[u] = x.next[u];
        x.load(j + TEAM * kUnroll);
        x.ahead(j + TEAM * kUnroll, j + (1 + kAhead) * TEAM * kUnroll);
        const bool all = j + (kUnroll - 1) * TEAM < jb;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (!all && j + u * TEAM >= jb) break;
            float v[V];
            Elem<T>::unpack(r[u], v);
            f(v, (j + u * TEAM) * V - off);
            __stcs(out + j + u * TEAM, Elem<T>::pack(v));
        }
    }
    const int head = min(e1, ja * V - off), tail = max(head, jb * V - off);
    const auto one = [&](int e) {
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = neg_inf();
        v[0] = Elem<T>::get(from.p[e]);
        f(v, e);
        o[e] = Elem<T>::put(v[0]);
    };
    for (int e = e0 + t; e < head; e += TEAM) one(e);
    for (int e = tail + t; e < e1; e += TEAM) one(e);
}

template <class T, int TEAM>
__device__ __forceinline__ void zero_range(T* o, int e0, int e1) {
    constexpr int V = Elem<T>::kVec;
    const int off = off_of(o), t = Team<TEAM>::tid();
    const int ja = (e0 + off + V - 1) / V, jb = max(ja, (e1 + off) / V);
    for (int j = ja + t; j < jb; j += TEAM) __stcs(reinterpret_cast<uint4*>(o - off) + j, make_uint4(0, 0, 0, 0));
    const int head = min(e1, ja * V - off), tail = max(head, jb * V - off);
    for (int e = e0 + t; e < head; e += TEAM) o[e] = Elem<T>::put(0.f);
    for (int e = tail + t; e < e1; e += TEAM) o[e] = Elem<T>::put(0.f);
}

// The elements of a part of the row o: whole vectors of it, but at the row's ends.
struct Range {
    int e0, e1;
};
template <class T>
__device__ __forceinline__ Range range_of(const T* o, int M, int rank, int parts) {
    const Slice s = slice_of(vecs_of(o, M), rank, parts);
    return Range{max(first_of(o, s.begin), 0), min(first_of(o, s.end), M)};
}

// The teacher's shares into l.q and their scale, by one warp (what sum_list leaves there, in fp32).
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
        if (lane + 32 * j < a.K) l.q[lane + 32 * j] = y[j];
    if (lane == 0) l.sums.scale = a.rest ? 1.f : 1.f / sum;
}

// Gradient of the columns from e0 to e1 as if none were listed; w: the row's weight over T.
template <class T, int TEAM, bool AHEAD>
__device__ __forceinline__ void distill_row_grad(const DistillArgs& a, const RowStats& s, float w, T* o, int e0, int e1,
                                                 Fetch<T, TEAM, AHEAD>& x) {
    const float coef = s.coef * w, gm = s.gm, gls2 = s.gls * kLog2e, c = a.sc.c;
    map_range<T, TEAM>(o, e0, e1, x, [&](float* f, int) {
#pragma unroll
        for (int i = 0; i < Elem<T>::kVec; ++i) f[i] = coef * ex2(fmaf(f[i] - gm, c, -gls2));
    });
}
// and of the listed columns from e0 to e1, after a barrier.
template <class T, int TEAM>
__device__ __forceinline__ void distill_list_grad(const DistillArgs& a, const RowStats& s, float w, T* o, int e0,
                                                  int e1, const ListBuf& l, bool twice) {
    for (int k = Team<TEAM>::tid(); k < a.K; k += TEAM) {
        if (!l.ok(k) || !l.first[k] || l.id[k] < e0 || l.id[k] >= e1) continue;
        float q = l.q[k];
        if (twice)
            for (int j = k + 1; j < a.K; ++j)
                if (l.id[j] == l.id[k]) q += l.q[j];
        q *= l.sums.scale;
        o[l.id[k]] = Elem<T>::put(w * (s.Z * expf((l.x[k] - s.m) * a.sc.inv - s.ls) - q));
    }
}

}  // namespace rows
}  // namespace tp
