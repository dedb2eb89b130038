// Single rows of packed-sequence attention, each by one warp over the row's own
// interval alone.
//
// The tiled passes multiply the weights of masked pairs, which are zero, with
// whatever the masked rows hold; an infinity or NaN there turns the product into
// NaN.  A pass therefore looks at every row whose result is not finite: if a row
// that its tiles hold, but its interval does not, is not finite in one of those
// columns, they are computed again here.  Otherwise the row's own pairs made
// them so, and they stand.  Nothing is spent on this while the inputs are finite.
//
// An infinity or NaN in one row costs the rows of at most a few tiles a walk over
// their intervals (those that share a tile with it and do not see it); the rows
// that see it are looked at and stand, and a walk ends where all it is for are
// NaN.  Walks take kStep rows at a time, all their loads in flight.  8192 causal
// rows, 4/2 heads of 64, bf16, forward and backward (0.23 ms): a token that is NaN
// 12 ms, an infinity in V 6.5, a NaN in dOut 22, V all NaN 0.29 (with a walk for
// every row that is not finite, a pair at a time: 319, 215, 306 and 78).
#pragma once

#include "seq.h"

namespace sga {
namespace seq {

constexpr int kStep = 8;

// What a row sees, or what sees it: the interval [lo, hi), and before it the
// sinks [slo, shi) of a windowed plan's query where they do not touch it.
template <bool WIN> struct View {
    int64_t lo = 0, hi = 0;
};
template <> struct View<true> {
    int64_t lo = 0, hi = 0, slo = 0, shi = 0;
    int32_t begin = -1;   // of the row's sequence
};
template <bool WIN> __device__ __forceinline__ View<WIN> query_view(const SeqArgs &a, int64_t row) {
    View<WIN> v;
    const int2 se = __ldg(a.range + row);
    v.lo = se.x;
    v.hi = a.causal ? row + 1 : se.y;
    if constexpr (WIN) {
        v.begin = se.x;
        const int64_t lo = max((int64_t)se.x, row - a.window + 1), hi = min(v.hi, row + a.window), s = min((int64_t)se.x + a.sinks, v.hi);
        if (s >= lo) {
            v.hi = max(hi, s);
        } else {
            v.lo = lo;
            v.hi = hi;
            v.slo = se.x;
            v.shi = s;
        }
    }
    return v;
}
template <bool WIN> __device__ __forceinline__ View<WIN> key_view(const SeqArgs &a, int64_t row) {
    View<WIN> v;
    const int2 se = __ldg(a.range + row);
    v.lo = a.causal ? row : (int64_t)se.x;
    v.hi = se.y;
    if constexpr (WIN)
        if (row - se.x >= a.sinks) {
            v.lo = max(v.lo, row - a.window + 1);
            v.hi = min(v.hi, row + a.window);
        }
    return v;
}

// What a row's result came from: its view, within the rows [w0, w1) of the tiles
// that were walked for it (and [v0, v1) of its sinks' tiles).
template <bool WIN> struct Span : View<WIN> {
    int64_t w0 = 0, w1 = 0, v0 = 0, v1 = 0;
};
// The span of lane src's row, whose view is `v` there, over the tiles of `t`.
template <bool WIN> __device__ __forceinline__ Span<WIN> span_of_lane(const SeqArgs &a, const View<WIN> &v, int src, const SeqTile &t, int tile_rows) {
    Span<WIN> sp;
    sp.lo = __shfl_sync(SGA_FULL_MASK, v.lo, src);
    sp.hi = __shfl_sync(SGA_FULL_MASK, v.hi, src);
    sp.w0 = (int64_t)t.t0 * tile_rows;
    sp.w1 = min(a.rows, (int64_t)t.t1 * tile_rows);
    if constexpr (WIN) {
        sp.slo = __shfl_sync(SGA_FULL_MASK, v.slo, src);
        sp.shi = __shfl_sync(SGA_FULL_MASK, v.shi, src);
        sp.v0 = (int64_t)t.g0 * tile_rows;
        sp.v1 = min(a.rows, (int64_t)t.g1 * tile_rows);
    }
    return sp;
}

// Part 0: the sinks; part 1: the interval.
template <bool WIN> __device__ __forceinline__ int64_t first_of(const Span<WIN> &sp, int part) {
    if constexpr (WIN)
        if (part == 0) return sp.slo;
    return sp.lo;
}
template <bool WIN> __device__ __forceinline__ int64_t end_of(const Span<WIN> &sp, int part) {
    if constexpr (WIN)
        if (part == 0) return sp.shi;
    return sp.hi;
}

// A head's row, D / 32 consecutive elements a lane.
template <typename T, int D> struct RowFrag {
    static constexpr int W = D / 32;
    struct alignas(W * sizeof(T)) Raw {
        T x[W];
    };
    float x[W];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = 0.f;
    }
    __device__ __forceinline__ void load(const void *base, int64_t off) {
        const Raw r = *reinterpret_cast<const Raw *>(static_cast<const T *>(base) + off + (threadIdx.x & 31) * W);
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = to_f32<T>(r.x[i]);
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
    // this lane's columns that are not finite, or NaN, as bits
    __device__ __forceinline__ uint32_t not_finite() const {
        uint32_t b = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) b |= !(fabsf(x[i]) < INFINITY) ? 1u << i : 0u;
        return b;
    }
    __device__ __forceinline__ uint32_t nan() const {
        uint32_t b = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) b |= x[i] != x[i] ? 1u << i : 0u;
        return b;
    }
    __device__ __forceinline__ bool any_nan() const { return __any_sync(SGA_FULL_MASK, nan() != 0); }   // (of the whole row)
    // all the columns `want` of the row are NaN
    __device__ __forceinline__ bool all_nan(uint32_t want) const { return __all_sync(SGA_FULL_MASK, (want & ~nan()) == 0); }
    __device__ __forceinline__ void store(void *base, int64_t off, float f, uint32_t want) const {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if ((want >> i) & 1u) static_cast<T *>(base)[off + (threadIdx.x & 31) * W + i] = from_f32<T>(x[i] * f);
    }
};

// This lane's columns of the 32-column slices that are `part` modulo `parts`
// (counted from `first`), as bits.
template <int D> __device__ __forceinline__ uint32_t slice_columns(int first, int part, int parts) {
    constexpr int W = D / 32;
    const int slice = first + (int)(threadIdx.x & 31) * W / 32;
    return slice % parts == part ? (1u << W) - 1u : 0u;
}

// Whether a row of head h of `base` that the span's tiles hold, but its interval
// does not, is not finite in one of the columns `want`.
template <typename T, int D, bool WIN>
__device__ __forceinline__ bool masked_row_spoils(const void *base, int heads, int h, const Span<WIN> &sp, uint32_t want) {
    // before and behind the interval; of a windowed plan, what the two walks hold
    // before the sinks, between them and the interval, and behind it
    for (int side = 0; side < (WIN ? 6 : 2); ++side) {
        int64_t b = side ? sp.hi : sp.w0, e = side ? sp.w1 : sp.lo;
        if constexpr (WIN) {
            const int64_t x0 = side < 3 ? sp.v0 : sp.w0, x1 = side < 3 ? sp.v1 : sp.w1;
            const bool two = sp.slo < sp.shi;
            const int64_t s0 = two ? sp.slo : sp.lo, s1 = two ? sp.shi : sp.lo;
            b = side % 3 == 0 ? x0 : side % 3 == 1 ? max(x0, s1) : max(x0, sp.hi);
            e = side % 3 == 0 ? min(x1, s0) : side % 3 == 1 ? min(x1, sp.lo) : x1;
        }
        for (int64_t j = b; j < e; j += kStep) {
            uint32_t bad = 0;
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                RowFrag<T, D> r;
                r.load(base, (min(j + u, e - 1) * heads + h) * D);
                bad |= r.not_finite();
            }
            if (__any_sync(SGA_FULL_MASK, (bad & want) != 0)) return true;
        }
    }
    return false;
}

// The columns of out of one query row that are not finite; the caller leaves out
// rows whose sum of weights is NaN.
template <typename T, int D, bool WIN>
__device__ __forceinline__ void out_row_alone(const SeqArgs &a, int64_t row, int h, int hk, const Span<WIN> &sp) {
    RowFrag<T, D> q, acc;
    const int64_t at = (row * a.H + h) * D;
    acc.load(a.out_w, at);
    const uint32_t want = acc.not_finite();
    if (!masked_row_spoils<T, D, WIN>(a.V, a.Hkv, hk, sp, want)) return;
    q.load(a.Q, at);
    acc.zero();
    float m = -INFINITY, l = 0.f;
    for (int part = WIN ? 0 : 1; part < 2; ++part) {   // (the sinks, the interval)
        for (int64_t j = first_of(sp, part), e = end_of(sp, part); j < e && !acc.all_nan(want); j += kStep) {
            RowFrag<T, D> v[kStep];
            float s[kStep], mn = m;
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                RowFrag<T, D> k;
                const int64_t r = (min(j + u, e - 1) * a.Hkv + hk) * D;
                k.load(a.K, r);
                v[u].load(a.V, r);
                s[u] = q.dot(k) * (a.scale * kLog2e);
                mn = fmaxf(mn, s[u]);   // (the last row again behind the interval)
            }
            const float al = exp2_diff(m, mn);
            m = mn;
            l *= al;
#pragma unroll
            for (int i = 0; i < RowFrag<T, D>::W; ++i) acc.x[i] *= al;
#pragma unroll
            for (int u = 0; u < kStep; ++u)
                if (j + u < e) {
                    const float p = exp2_diff(s[u], m);
                    l += p;
                    acc.add(p, v[u]);
                }
        }
    }
    acc.store(a.out_w, at, 1.f / l, want);
}

// The columns `mine` of dK (DK) or dV of one key row that are not finite.
template <typename T, int D, bool WIN>
__device__ __forceinline__ void key_row_alone(const SeqArgs &a, bool DK, int64_t row, int hk, const Span<WIN> &sp, uint32_t mine) {
    RowFrag<T, D> k, v, acc;
    const int64_t at = (row * a.Hkv + hk) * D;
    k.load(a.K, at);
    v.load(a.V, at);
    if (k.any_nan() || (DK && v.any_nan())) return;   // every score (for dK: or dP) of the row is NaN
    void *res = DK ? a.dK : a.dV;
    acc.load(res, at);
    const uint32_t want = acc.not_finite() & mine;
    const int h0 = hk * (a.H / a.Hkv), h1 = h0 + a.H / a.Hkv;
    bool spoilt = false;
    for (int h = h0; h < h1 && !spoilt; ++h) spoilt = masked_row_spoils<T, D, WIN>(DK ? a.Q : a.dOut, a.H, h, sp, want);
    if (!spoilt) return;
    acc.zero();
    for (int h = h0; h < h1; ++h)
        for (int64_t r = sp.lo; r < sp.hi && !acc.all_nan(want); r += kStep) {
            RowFrag<T, D> q[kStep], g[kStep];
            float w[kStep];
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                const int64_t y = min(r + u, sp.hi - 1), t = (int64_t)h * a.rows_pad + y;
                q[u].load(a.Q, (y * a.H + h) * D);
                g[u].load(a.dOut, (y * a.H + h) * D);
                w[u] = fast_exp2(fmaf(q[u].dot(k), a.scale * kLog2e, a.ws_nlse[t]));
                if (DK) w[u] *= g[u].dot(v) + a.ws_ndelta[t];
            }
#pragma unroll
            for (int u = 0; u < kStep; ++u)
                if (r + u < sp.hi) acc.add(w[u], DK ? q[u] : g[u]);
        }
    acc.store(res, at, DK ? a.scale : 1.f, want);
}

// The columns `mine` of dQ of one query row that are not finite.
template <typename T, int D, bool WIN>
__device__ __forceinline__ void query_row_alone(const SeqArgs &a, int64_t row, int h, const Span<WIN> &sp, uint32_t mine) {
    RowFrag<T, D> q, g, acc;
    const int64_t at = (row * a.H + h) * D, t = (int64_t)h * a.rows_pad + row;
    const int hk = h / (a.H / a.Hkv);
    const float nlse = a.ws_nlse[t], nd = a.ws_ndelta[t];
    if (nlse != nlse || nd != nd) return;   // every dS of the row is NaN
    acc.load(a.dQ, at);
    const uint32_t want = acc.not_finite() & mine;
    if (!masked_row_spoils<T, D, WIN>(a.K, a.Hkv, hk, sp, want)) return;
    q.load(a.Q, at);
    g.load(a.dOut, at);
    acc.zero();
    for (int part = WIN ? 0 : 1; part < 2; ++part) {   // (the sinks, the interval)
        for (int64_t j = first_of(sp, part), e = end_of(sp, part); j < e && !acc.all_nan(want); j += kStep) {
            RowFrag<T, D> k[kStep];
            float w[kStep];
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                RowFrag<T, D> v;
                const int64_t r = (min(j + u, e - 1) * a.Hkv + hk) * D;
                k[u].load(a.K, r);
                v.load(a.V, r);
                w[u] = fast_exp2(fmaf(q.dot(k[u]), a.scale * kLog2e, nlse)) * (g.dot(v) + nd);
            }
#pragma unroll
            for (int u = 0; u < kStep; ++u)
                if (j + u < e) acc.add(w[u], k[u]);
        }
    }
    acc.store(a.dQ, at, a.scale, want);
}

}  // namespace seq
}  // namespace sga
