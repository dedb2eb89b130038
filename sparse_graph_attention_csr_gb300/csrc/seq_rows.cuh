// Single rows of packed-sequence attention, each by one warp over the row's own
// interval alone.
//
// The tiled passes multiply the weights of masked pairs, which are zero, with
// whatever the masked rows hold; an infinity or NaN there would turn the product
// into NaN.  A pass therefore computes every row whose result is not finite
// again here.  Nothing is spent on this while the inputs are finite, nor where
// the row itself makes every weight NaN (a batch that has gone NaN throughout):
// its result is NaN with or without the masked pairs.
#pragma once

#include "seq.h"

namespace sga {
namespace seq {

// A head's row, D / 32 consecutive elements a lane.
template <typename T, int D> struct RowFrag {
    static constexpr int W = D / 32;
    float x[W];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = 0.f;
    }
    __device__ __forceinline__ void load(const void *base, int64_t off) {
        const T *p = static_cast<const T *>(base) + off + (threadIdx.x & 31) * W;
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = to_f32<T>(p[i]);
    }
    __device__ __forceinline__ float dot(const RowFrag &o) const {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) s = fmaf(x[i], o.x[i], s);
        return group_sum<32>(s);
    }
    __device__ __forceinline__ void add(float w, const RowFrag &o) {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = fmaf(w, o.x[i], x[i]);
    }
    __device__ __forceinline__ bool has_nan() const {   // (of the whole row)
        bool b = false;
#pragma unroll
        for (int i = 0; i < W; ++i) b |= x[i] != x[i];
        return __any_sync(SGA_FULL_MASK, b);
    }
    // store the columns [c0, c0 + n)
    __device__ __forceinline__ void store(void *base, int64_t off, float f, int c0, int n) const {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int c = (threadIdx.x & 31) * W + i;
            if (c >= c0 && c < c0 + n) static_cast<T *>(base)[off + c] = from_f32<T>(x[i] * f);
        }
    }
};

// out of one query row over the keys [lo, hi); the caller leaves out rows whose
// sum of weights is NaN.
template <typename T, int D>
__device__ __forceinline__ void out_row_alone(const SeqArgs &a, int64_t row, int h, int hk, int64_t lo, int64_t hi) {
    RowFrag<T, D> q, k, v, acc;
    q.load(a.Q, (row * a.H + h) * D);
    acc.zero();
    float m = -INFINITY, l = 0.f;
    for (int64_t j = lo; j < hi; ++j) {
        k.load(a.K, (j * a.Hkv + hk) * D);
        v.load(a.V, (j * a.Hkv + hk) * D);
        const float s = q.dot(k) * (a.scale * kLog2e);
        const float mn = fmaxf(m, s), al = exp2_diff(m, mn), p = exp2_diff(s, mn);
        l = fmaf(l, al, p);
        m = mn;
#pragma unroll
        for (int i = 0; i < RowFrag<T, D>::W; ++i) acc.x[i] *= al;
        acc.add(p, v);
    }
    acc.store(a.out_w, (row * a.H + h) * D, 1.f / l, 0, D);
}

// Columns [c0, c0 + n) of dK (DK) or dV of one key row over the queries [lo, hi).
template <typename T, int D>
__device__ __forceinline__ void key_row_alone(const SeqArgs &a, bool DK, int64_t row, int hk, int64_t lo, int64_t hi,
                                              int c0, int n) {
    RowFrag<T, D> k, v, q, g, acc;
    const int64_t at = (row * a.Hkv + hk) * D;
    k.load(a.K, at);
    v.load(a.V, at);
    if (k.has_nan() || (DK && v.has_nan())) return;   // every score (for dK: or dP) of the row is NaN
    acc.zero();
    const int grp = a.H / a.Hkv;
    for (int h = hk * grp; h < (hk + 1) * grp; ++h)
        for (int64_t r = lo; r < hi; ++r) {
            q.load(a.Q, (r * a.H + h) * D);
            g.load(a.dOut, (r * a.H + h) * D);
            const int64_t t = (int64_t)h * a.rows_pad + r;
            const float p = fast_exp2(fmaf(q.dot(k), a.scale * kLog2e, a.ws_nlse[t]));
            if (DK) acc.add(p * (g.dot(v) + a.ws_ndelta[t]), q);
            else acc.add(p, g);
        }
    acc.store(DK ? a.dK : a.dV, at, DK ? a.scale : 1.f, c0, n);
}

// Columns [c0, c0 + n) of dQ of one query row over the keys [lo, hi).
template <typename T, int D>
__device__ __forceinline__ void query_row_alone(const SeqArgs &a, int64_t row, int h, int64_t lo, int64_t hi, int c0, int n) {
    RowFrag<T, D> q, g, k, v, acc;
    const int64_t at = (row * a.H + h) * D, t = (int64_t)h * a.rows_pad + row;
    const int hk = h / (a.H / a.Hkv);
    q.load(a.Q, at);
    g.load(a.dOut, at);
    if (q.has_nan() || g.has_nan()) return;   // every score or dP of the row is NaN
    acc.zero();
    for (int64_t j = lo; j < hi; ++j) {
        k.load(a.K, (j * a.Hkv + hk) * D);
        v.load(a.V, (j * a.Hkv + hk) * D);
        const float p = fast_exp2(fmaf(q.dot(k), a.scale * kLog2e, a.ws_nlse[t]));
        acc.add(p * (g.dot(v) + a.ws_ndelta[t]), k);
    }
    acc.store(a.dQ, at, a.scale, c0, n);
}

}  // namespace seq
}  // namespace sga
