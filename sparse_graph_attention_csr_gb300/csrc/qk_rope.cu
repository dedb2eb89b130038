// Norm of every query and key head and their rotary positions, in one pass over
// them, forward and backward.
//   r = 1 / sqrt(sum x^2 / D + eps),  y = x r w   (per head; w [D], shared by the heads)
//   a pair (y_a, y_b) at position p turns by the angle p f of its frequency:
//     (y_a cos - y_b sin, y_a sin + y_b cos)
//   backward: dn = the gradient turned back, xhat = x r, g = dn w,
//     dx = r (g - xhat sum(g xhat) / D),  dw = sum over rows and heads of dn xhat
//
// Bound by DRAM: the forward reads and writes Q and K once, the backward reads
// them and their gradients and writes one gradient.  A head is held by D / (2 EL)
// lanes, each with two 16-byte chunks that hold both elements of its pairs, so a
// rotation needs no exchange.  A block takes a few rows: the cosines and sines of
// their pairs are formed once, in shared memory, and serve all heads of a row.
//
// Angles: a frequency is kept as turns a position in units of 2^-64, so that
// position x frequency, a product of integers that wraps, is the exact fraction of
// a turn of the stored frequency at any position, negative ones too; in fp32 the
// product would be off by 0.01 radian from position 200,000 on.
//
// Weight gradients: each thread sums its columns in registers, a block adds its
// groups in order, and a second kernel adds the blocks in order: no atomics,
// bitwise reproducible.  Statistics and sums are fp32.
#include <algorithm>
#include <cmath>

#include "common.cuh"

namespace sga {

void set_cuda_error(cudaError_t e);   // (api.cu)

namespace {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

sga_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return SGA_OK;
    set_cuda_error(e);
    return SGA_ECUDA;
}

constexpr int kThreads = 256, kMaxRows = 32;   // of a block

struct RopeArgs {
    sga_rotary rot;
    const void *Q, *K, *pos, *wq, *wk, *dQo, *dKo;
    void *Qo, *Ko;           // forward: results; backward: dQ, dK
    float *rq, *rk;          // 1 / sqrt of the mean square (forward: written; null: rotation alone)
    const float *rq_in, *rk_in;
    float *part;             // [blocks][2][D] sums of dwq, dwk, or null
    int64_t T, ldq, ldk;     // rows; elements from a row of Q, K to the next
    int H, Hkv, rows;        // heads; rows a block takes at a time
    float eps;
    int wide;                // 64-bit positions
};

template <typename T> __device__ __forceinline__ uint4 load16(const T *p) { return *reinterpret_cast<const uint4 *>(p); }

// Where a lane's two chunks of EL elements lie in a head, and which pair its
// e-th element (of EL) belongs to.
//   halves: pair i is elements (i, i + rot / 2); a lane's chunks are that far
//     apart, so its e-th pair is (x0[e], x1[e]); chunks past the rotated ones
//     follow by twos.
//   interleaved: pair i is elements (2 i, 2 i + 1); the chunks are half a head
//     apart, pairs e < EL / 2 in the first.
template <int D, int EL> struct Lane {
    int c0, c1, pair;    // chunks; halves: the first pair, or -1 (nothing rotated)
    __device__ __forceinline__ Lane(const sga_rotary &r, int lane) {
        constexpr int G = D / (2 * EL);
        const int half = r.rot / (2 * EL);   // (halves: lanes with a rotated chunk)
        if (r.interleaved) {
            c0 = lane;
            c1 = lane + G;
            pair = lane * EL / 2;
        } else if (lane < half) {
            c0 = lane;
            c1 = lane + half;
            pair = lane * EL;
        } else {
            c0 = 2 * lane;   // (2 half + 2 (lane - half))
            c1 = c0 + 1;
            pair = -1;
        }
    }
};

// cos, sin of the angles of a block's rows: [row][e / 2][lane] as float4 (two
// pairs).  Pairs past the rotated ones turn by nothing.
template <int D, int EL>
__device__ __forceinline__ void fill_turns(const RopeArgs &a, float4 *cs, int64_t t0, int rows) {
    constexpr int G = D / (2 * EL), P = D / 2;
    const sga_rotary &r = a.rot;
    for (int i = threadIdx.x; i < rows * P; i += kThreads) {
        const int row = i / P, e = i % P / G, lane = i % G;
        int pair;
        if (r.interleaved) pair = e < EL / 2 ? lane * (EL / 2) + e : (lane + G) * (EL / 2) + e - EL / 2;
        else pair = lane * EL + e;
        float s = 0.f, c = 1.f;
        if (2 * pair < r.rot) {
            const int64_t at = (t0 + row) * r.axes + r.axis[pair];
            const int64_t p = a.wide ? __ldg(static_cast<const long long *>(a.pos) + at)
                                     : (int64_t)__ldg(static_cast<const int *>(a.pos) + at);
            const uint64_t turn = (uint64_t)p * r.turn[pair];
            // half turns in [-1, 1): the top 32 bits, rounded
            const float x = (float)(int32_t)(uint32_t)((turn + 0x80000000ull) >> 32) * 0x1p-31f;
            sincospif(x, &s, &c);
        }
        reinterpret_cast<float2 *>(cs + (row * (EL / 2) + e / 2) * G + lane)[e & 1] = make_float2(c, s);
    }
}

// Turns the lane's pairs (back: by the negative angles).
template <int EL, int G, bool BACK>
__device__ __forceinline__ void turn_pairs(const RopeArgs &a, float *x0, float *x1, const float4 *cs, int pair) {
    if (!a.rot.interleaved && pair < 0) return;   // (x0 and x1 belong to no pair)
#pragma unroll
    for (int e = 0; e < EL; e += 2) {
        const float4 t = cs[(e / 2) * G];
        float *u, *v;
        if (!a.rot.interleaved) {
            const float u0 = x0[e], v0 = x1[e], u1 = x0[e + 1], v1 = x1[e + 1];
            const float s0 = BACK ? -t.y : t.y, s1 = BACK ? -t.w : t.w;
            x0[e] = u0 * t.x - v0 * s0;
            x1[e] = u0 * s0 + v0 * t.x;
            x0[e + 1] = u1 * t.z - v1 * s1;
            x1[e + 1] = u1 * s1 + v1 * t.z;
        } else {   // pairs e, e + 1: elements 2 e .. 2 e + 3 of the lane's 2 EL
            u = 2 * e < EL ? x0 + 2 * e : x1 + 2 * e - EL;
            v = u + 1;
            const int p = e < EL / 2 ? pair + e : pair + e + (G - 1) * (EL / 2);
            const float s0 = BACK ? -t.y : t.y, s1 = BACK ? -t.w : t.w;
            const float u0 = u[0], v0 = v[0], u1 = u[2], v1 = v[2];
            if (2 * p < a.rot.rot) {
                u[0] = u0 * t.x - v0 * s0;
                v[0] = u0 * s0 + v0 * t.x;
            }
            if (2 * (p + 1) < a.rot.rot) {
                u[2] = u1 * t.z - v1 * s1;
                v[2] = u1 * s1 + v1 * t.z;
            }
        }
    }
}

// The weights as fp32: [2][D], ones where there are none.
template <typename TW, int D> __device__ __forceinline__ void fill_weights(const RopeArgs &a, float *w) {
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        const TW *src = static_cast<const TW *>(i < D ? a.wq : a.wk);
        w[i] = src ? to_f32<TW>(src[i % D]) : 1.f;
    }
}

template <int EL> __device__ __forceinline__ void load_f32(const float *p, float *x) {
#pragma unroll
    for (int i = 0; i < EL; i += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(p + i);
        x[i] = q.x;
        x[i + 1] = q.y;
        x[i + 2] = q.z;
        x[i + 3] = q.w;
    }
}

// Item `it` of a block: a head (queries' first, then keys') of one of its rows.
struct Item {
    int row, head;
    bool key;
    __device__ __forceinline__ Item(const RopeArgs &a, int it) {
        const int heads = a.H + a.Hkv;
        row = it / heads;
        head = it - row * heads;
        key = head >= a.H;
        if (key) head -= a.H;
    }
};

template <typename T, typename TW, int D> __global__ void __launch_bounds__(kThreads) qk_rope_fwd_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int EL = Elt<T>::EL, G = D / (2 * EL), GROUPS = kThreads / G, U = 2;
    extern __shared__ float4 cs[];   // [rows][EL / 2][G]
    __shared__ __align__(16) float w[2 * D];
    let_next_start();
    wait_previous();
    fill_weights<TW, D>(a, w);
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const Lane<D, EL> at(a.rot, lane);
    const bool norm = a.rq != nullptr;
    for (int64_t t0 = (int64_t)blockIdx.x * a.rows; t0 < a.T; t0 += (int64_t)gridDim.x * a.rows) {
        const int rows = (int)min((int64_t)a.rows, a.T - t0), items = rows * (a.H + a.Hkv);
        uint4 x[U][2];
        auto fetch = [&](int it0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int it = it0 + u * GROUPS;
                x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
                if (it < items) {
                    const Item m(a, it);
                    const T *src = static_cast<const T *>(m.key ? a.K : a.Q) + (t0 + m.row) * (m.key ? a.ldk : a.ldq) + m.head * D;
                    x[u][0] = load16(src + at.c0 * EL);
                    x[u][1] = load16(src + at.c1 * EL);
                }
            }
        };
        fetch(grp);
        __syncthreads();   // the rows before are done with cs
        fill_turns<D, EL>(a, cs, t0, rows);
        __syncthreads();
        // every group of a warp runs the same number of rounds: the sums are warp-wide calls
        for (int i0 = 0; i0 < items; i0 += U * GROUPS) {
            float y[U][2 * EL];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                unpack<T>(x[u][0], y[u]);
                unpack<T>(x[u][1], y[u] + EL);
            }
            fetch(i0 + U * GROUPS + grp);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int it = i0 + u * GROUPS + grp;
                const Item m(a, it);
                if (norm) {
                    float s = 0.f, wr[2 * EL];
#pragma unroll
                    for (int i = 0; i < 2 * EL; ++i) s = fmaf(y[u][i], y[u][i], s);
                    const float r = rsqrtf(group_sum<G>(s) * (1.f / D) + a.eps);
                    load_f32<EL>(w + m.key * D + at.c0 * EL, wr);
                    load_f32<EL>(w + m.key * D + at.c1 * EL, wr + EL);
#pragma unroll
                    for (int i = 0; i < 2 * EL; ++i) y[u][i] *= r * wr[i];
                    if (lane == 0 && it < items) {
                        if (m.key) a.rk[(t0 + m.row) * a.Hkv + m.head] = r;
                        else a.rq[(t0 + m.row) * a.H + m.head] = r;
                    }
                }
                if (it < items) {
                    turn_pairs<EL, G, false>(a, y[u], y[u] + EL, cs + m.row * (EL / 2) * G + lane, at.pair);
                    T *dst = static_cast<T *>(m.key ? a.Ko : a.Qo) + ((t0 + m.row) * (m.key ? a.Hkv : a.H) + m.head) * D;
                    *reinterpret_cast<uint4 *>(dst + at.c0 * EL) = pack<T>(y[u]);
                    *reinterpret_cast<uint4 *>(dst + at.c1 * EL) = pack<T>(y[u] + EL);
                }
            }
        }
    }
}

// A block's sums of one weight's gradient: its groups added in order.
template <int D, int EL, int G>
__device__ __forceinline__ void block_sums(float *sm, const float *acc, const Lane<D, EL> &at, float *out) {
    const int grp = threadIdx.x / G;
    // the groups of a warp first (lanes G apart), then the warps
    float s[2 * EL];
#pragma unroll
    for (int i = 0; i < 2 * EL; ++i) {
        s[i] = acc[i];
#pragma unroll
        for (int o = 16; o >= G; o >>= 1) s[i] += __shfl_xor_sync(SGA_FULL_MASK, s[i], o);
    }
    constexpr int PER = 32 / G;   // groups of a warp
    __syncthreads();
    if (grp % PER == 0)
#pragma unroll
        for (int i = 0; i < 2 * EL; ++i) sm[(threadIdx.x / 32) * D + (i < EL ? at.c0 * EL + i : at.c1 * EL + i - EL)] = s[i];
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kThreads) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) t += sm[k * D + i];
        out[i] = t;
    }
}

template <typename T, typename TW, int D> __global__ void __launch_bounds__(kThreads) qk_rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int EL = Elt<T>::EL, G = D / (2 * EL), GROUPS = kThreads / G;
    extern __shared__ float4 cs[];   // [rows][EL / 2][G]
    __shared__ __align__(16) float w[2 * D];
    __shared__ float sums[kThreads / 32 * D];
    let_next_start();
    wait_previous();
    fill_weights<TW, D>(a, w);
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const Lane<D, EL> at(a.rot, lane);
    const bool norm = a.rq_in != nullptr;
    float aq[2 * EL], ak[2 * EL];   // this thread's sums of dwq, dwk
#pragma unroll
    for (int i = 0; i < 2 * EL; ++i) aq[i] = ak[i] = 0.f;
    for (int64_t t0 = (int64_t)blockIdx.x * a.rows; t0 < a.T; t0 += (int64_t)gridDim.x * a.rows) {
        const int rows = (int)min((int64_t)a.rows, a.T - t0), items = rows * (a.H + a.Hkv);
        uint4 x[2], g[2];
        float r_next = 0.f;
        auto fetch = [&](int it) {
            x[0] = x[1] = g[0] = g[1] = make_uint4(0, 0, 0, 0);
            r_next = 0.f;
            if (it < items) {
                const Item m(a, it);
                const T *src = static_cast<const T *>(m.key ? a.dKo : a.dQo) + ((t0 + m.row) * (m.key ? a.Hkv : a.H) + m.head) * D;
                g[0] = load16(src + at.c0 * EL);
                g[1] = load16(src + at.c1 * EL);
                if (norm) {
                    src = static_cast<const T *>(m.key ? a.K : a.Q) + (t0 + m.row) * (m.key ? a.ldk : a.ldq) + m.head * D;
                    x[0] = load16(src + at.c0 * EL);
                    x[1] = load16(src + at.c1 * EL);
                    r_next = m.key ? a.rk_in[(t0 + m.row) * a.Hkv + m.head] : a.rq_in[(t0 + m.row) * a.H + m.head];
                }
            }
        };
        fetch(grp);
        __syncthreads();
        fill_turns<D, EL>(a, cs, t0, rows);
        __syncthreads();
        for (int i0 = 0; i0 < items; i0 += GROUPS) {
            const int it = i0 + grp;
            float xh[2 * EL], dn[2 * EL];
            const float r = r_next;
            unpack<T>(g[0], dn);
            unpack<T>(g[1], dn + EL);
            unpack<T>(x[0], xh);
            unpack<T>(x[1], xh + EL);
            fetch(it + GROUPS);
            const Item m(a, it);
            if (it < items) turn_pairs<EL, G, true>(a, dn, dn + EL, cs + m.row * (EL / 2) * G + lane, at.pair);
            if (norm) {
                float wr[2 * EL], s = 0.f;
                load_f32<EL>(w + m.key * D + at.c0 * EL, wr);
                load_f32<EL>(w + m.key * D + at.c1 * EL, wr + EL);
#pragma unroll
                for (int i = 0; i < 2 * EL; ++i) xh[i] *= r;
                if (m.key) {
#pragma unroll
                    for (int i = 0; i < 2 * EL; ++i) ak[i] = fmaf(dn[i], xh[i], ak[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * EL; ++i) aq[i] = fmaf(dn[i], xh[i], aq[i]);
                }
#pragma unroll
                for (int i = 0; i < 2 * EL; ++i) {
                    dn[i] *= wr[i];
                    s = fmaf(dn[i], xh[i], s);
                }
                s = group_sum<G>(s) * (1.f / D);
#pragma unroll
                for (int i = 0; i < 2 * EL; ++i) dn[i] = r * (dn[i] - xh[i] * s);
            }
            if (it < items) {
                T *dst = static_cast<T *>(m.key ? a.Ko : a.Qo) + ((t0 + m.row) * (m.key ? a.Hkv : a.H) + m.head) * D;
                *reinterpret_cast<uint4 *>(dst + at.c0 * EL) = pack<T>(dn);
                *reinterpret_cast<uint4 *>(dst + at.c1 * EL) = pack<T>(dn + EL);
            }
        }
    }
    if (!a.part) return;
    float *out = a.part + (int64_t)blockIdx.x * 2 * D;
    block_sums<D, EL, G>(sums, aq, at, out);
    block_sums<D, EL, G>(sums, ak, at, out + D);
}

// dwq, dwk from the blocks' sums: 32 columns a block; its 32 warps take every
// 32nd block's, four in flight, and are added in order.
template <typename TW>
__global__ void __launch_bounds__(1024) qk_rope_reduce_kernel(const float *__restrict__ part, int blocks, int D, TW *dwq, TW *dwk) {
    __shared__ float sm[32][33];
    wait_previous();
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, n = 2 * D;
    const int i = blockIdx.x * 32 + lane;   // (n is a multiple of 32)
    float s = 0.f;
    for (int b = wp; b < blocks; b += 128) {
        float v[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) v[z] = b + 32 * z < blocks ? part[(int64_t)(b + 32 * z) * n + i] : 0.f;
        s += (v[0] + v[1]) + (v[2] + v[3]);
    }
    sm[wp][lane] = s;
    __syncthreads();
    s = group_sum<32>(sm[lane][wp]);   // warp wp: column wp of the block
    const int c = blockIdx.x * 32 + wp;
    if (lane == 0) (c < D ? dwq : dwk)[c < D ? c : c - D] = from_f32<TW>(s);
}

constexpr int kBwdBlocksPerSm = 4;   // most of the backward pass, each with a row of sums

// Rows a block takes at a time: enough heads for four rounds of its groups, but
// no fewer blocks than SMs where there are rows for them.
int rows_of(int64_t T, int heads, int groups) {
    const int64_t want = (4 * groups + heads - 1) / heads, spread = std::max<int64_t>(1, T / device_sms());
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, spread), kMaxRows));
}

template <typename T, typename TW, int D> cudaError_t launch_fwd(RopeArgs &a, cudaStream_t s) {
    a.rows = rows_of(a.T, a.H + a.Hkv, kThreads / (D / (2 * Elt<T>::EL)));
    const int64_t blocks = std::min<int64_t>((a.T + a.rows - 1) / a.rows, (int64_t)device_sms() * 64);
    note_launch(SGA_KERN_QK_ROPE_FWD, s, false);
    const cudaError_t e = launch_early(qk_rope_fwd_kernel<T, TW, D>, dim3((unsigned)blocks), dim3(kThreads),
                                       (size_t)a.rows * D / 2 * sizeof(float2), s, a);
    note_launch(SGA_KERN_QK_ROPE_FWD, s, true);
    return e;
}

template <typename T, typename TW, int D> cudaError_t launch_bwd(RopeArgs &a, void *dwq, void *dwk, cudaStream_t s) {
    a.rows = rows_of(a.T, a.H + a.Hkv, kThreads / (D / (2 * Elt<T>::EL)));
    // as many blocks as are resident at once
    static std::atomic<int> per_sm[kMaxDevices];
    cudaError_t asked = cudaSuccess;
    const int fit = per_device(per_sm, [&] {
        int n = 0;
        asked = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, qk_rope_bwd_kernel<T, TW, D>, kThreads,
                                                              kMaxRows * D / 2 * sizeof(float2));
        return asked == cudaSuccess ? std::max(1, std::min(n, kBwdBlocksPerSm)) : 0;
    });
    if (asked != cudaSuccess) return asked;
    const int blocks = (int)std::min<int64_t>((a.T + a.rows - 1) / a.rows, (int64_t)device_sms() * fit);
    note_launch(SGA_KERN_QK_ROPE_BWD, s, false);
    cudaError_t e = launch_early(qk_rope_bwd_kernel<T, TW, D>, dim3((unsigned)blocks), dim3(kThreads),
                                 (size_t)a.rows * D / 2 * sizeof(float2), s, a);
    note_launch(SGA_KERN_QK_ROPE_BWD, s, true);
    if (e != cudaSuccess || !a.part) return e;
    note_launch(SGA_KERN_QK_ROPE_REDUCE, s, false);
    e = launch_early(qk_rope_reduce_kernel<TW>, dim3(2 * D / 32), dim3(1024), 0, s, static_cast<const float *>(a.part), blocks, D,
                     static_cast<TW *>(dwq), static_cast<TW *>(dwk));
    note_launch(SGA_KERN_QK_ROPE_REDUCE, s, true);
    return e;
}

template <typename F> cudaError_t by_type(int D, sga_dtype dt, sga_dtype wdt, F f) {
    auto width = [&](auto t, auto w) {
        return D == 32 ? f(t, w, std::integral_constant<int, 32>())
               : D == 64 ? f(t, w, std::integral_constant<int, 64>()) : f(t, w, std::integral_constant<int, 128>());
    };
    if (dt == SGA_F32) return width(float(), float());
    if (wdt == SGA_F32) return width(__nv_bfloat16(), float());
    return width(__nv_bfloat16(), __nv_bfloat16());
}

// What both passes ask of their arguments; SGA_OK with T = 0 too.
sga_status check_rope(const sga_rotary *r, int64_t T, int H, int Hkv, int64_t ldq, int64_t ldk, int pos_bytes, sga_dtype dt, sga_dtype wdt) {
    if (!r || T < 0 || H < 1 || Hkv < 1) return SGA_EINVAL;
    if (pos_bytes != 4 && pos_bytes != 8) return SGA_EINVAL;
    if (dt != SGA_F32 && dt != SGA_BF16) return SGA_EUNSUPPORTED;
    if (wdt != SGA_F32 && wdt != dt) return SGA_EUNSUPPORTED;
    // (a table that sga_rotary_init has not filled, or that was changed)
    if ((r->D != 32 && r->D != 64 && r->D != 128) || r->rot < 0 || r->rot > r->D || r->rot % 16 || r->axes < 1 || r->axes > SGA_MAX_AXES)
        return SGA_EINVAL;
    for (int i = 0; 2 * i < r->rot; ++i)
        if (r->axis[i] >= r->axes) return SGA_EINVAL;
    if ((int64_t)(H + (int64_t)Hkv) * r->D > 32768) return SGA_EUNSUPPORTED;
    const int64_t el = dt == SGA_F32 ? 4 : 8;
    if (ldq < (int64_t)H * r->D || ldk < (int64_t)Hkv * r->D || ldq % el || ldk % el) return SGA_EINVAL;
    return SGA_OK;
}

}  // namespace
}  // namespace sga

using namespace sga;

extern "C" {

sga_status sga_rotary_init(sga_rotary *r, int D, int rot, const double *freqs, const int32_t *sections, int axes, int interleaved) {
    if (!r) return SGA_EINVAL;
    if (D != 32 && D != 64 && D != 128) return SGA_EUNSUPPORTED;
    if (rot < 0 || rot > D || rot % 16 || (rot > 0 && !freqs)) return SGA_EINVAL;
    if (axes < 1 || axes > SGA_MAX_AXES || (axes > 1 && !sections) || (interleaved != 0 && interleaved != 1)) return SGA_EINVAL;
    *r = sga_rotary{};
    r->D = D;
    r->rot = rot;
    r->axes = axes;
    r->interleaved = interleaved;
    int64_t at = 0;
    if (sections) {
        for (int x = 0; x < axes; ++x) {
            if (sections[x] < 0 || at + sections[x] > rot / 2) return SGA_EINVAL;
            for (int i = 0; i < sections[x]; ++i) r->axis[at++] = (uint8_t)x;
        }
        if (at != rot / 2) return SGA_EINVAL;
    }
    for (int i = 0; i < rot / 2; ++i) {
        if (!std::isfinite(freqs[i])) return SGA_EINVAL;
        double t = freqs[i] / 6.283185307179586476925;   // turns a position
        t -= std::floor(t);                              // (whole turns are none; negative ones wrap)
        const double f = std::ldexp(t, 64);
        r->turn[i] = f >= 0x1p64 ? 0 : (uint64_t)f;
    }
    return SGA_OK;
}

sga_status qk_norm_rope_fwd(const sga_rotary *rot, const void *Q, int64_t ldq, const void *K, int64_t ldk, const void *pos,
                            int pos_bytes, const void *wq, const void *wk, int64_t T, int H, int Hkv, float eps, sga_dtype dt,
                            sga_dtype wdt, void *Qo, void *Ko, float *rq, float *rk, void *stream) {
    const sga_status st = check_rope(rot, T, H, Hkv, ldq, ldk, pos_bytes, dt, wdt);
    if (st != SGA_OK) return st;
    if (!(eps >= 0.f) || !(eps < INFINITY) || !wq != !wk) return SGA_EINVAL;
    if (T == 0) return SGA_OK;   // (whose tensors may have no address)
    if (!rq != !rk || (wq && !rq)) return SGA_EINVAL;
    const size_t we = wdt == SGA_F32 ? 4 : 2;
    for (const void *p : {Q, K, static_cast<const void *>(Qo), static_cast<const void *>(Ko)})
        if (!p || !aligned(p, 16)) return SGA_EINVAL;
    if (!pos || !aligned(pos, pos_bytes) || !aligned(wq, we) || !aligned(wk, we) || !aligned(rq, 4) || !aligned(rk, 4)) return SGA_EINVAL;
    RopeArgs a{};
    a.rot = *rot;
    a.Q = Q;
    a.K = K;
    a.pos = pos;
    a.wq = wq;
    a.wk = wk;
    a.Qo = Qo;
    a.Ko = Ko;
    a.rq = rq;
    a.rk = rk;
    a.T = T;
    a.ldq = ldq;
    a.ldk = ldk;
    a.H = H;
    a.Hkv = Hkv;
    a.eps = eps;
    a.wide = pos_bytes == 8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return status_of(by_type(rot->D, dt, wdt, [&](auto t, auto w, auto d) { return launch_fwd<decltype(t), decltype(w), decltype(d)::value>(a, s); }));
}

size_t sga_qk_norm_rope_bwd_workspace_bytes(int64_t T, int D) {
    if (T <= 0 || D <= 0) return 0;
    return (size_t)std::min<int64_t>((int64_t)device_sms() * kBwdBlocksPerSm, T) * 2 * (size_t)D * sizeof(float);
}

sga_status qk_norm_rope_bwd(const sga_rotary *rot, const void *Q, int64_t ldq, const void *K, int64_t ldk, const void *pos,
                            int pos_bytes, const void *wq, const void *wk, const float *rq, const float *rk, const void *dQo,
                            const void *dKo, int64_t T, int H, int Hkv, sga_dtype dt, sga_dtype wdt, void *dQ, void *dK, void *dwq,
                            void *dwk, void *workspace, size_t workspace_bytes, void *stream) {
    const sga_status st = check_rope(rot, T, H, Hkv, ldq, ldk, pos_bytes, dt, wdt);
    if (st != SGA_OK) return st;
    if (!wq != !wk || !dwq != !dwk || (dwq && !wq)) return SGA_EINVAL;
    const size_t we = wdt == SGA_F32 ? 4 : 2;
    if (!aligned(wq, we) || !aligned(wk, we) || !aligned(dwq, we) || !aligned(dwk, we)) return SGA_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {   // an empty sum
        cudaError_t e = cudaSuccess;
        if (dwq) e = cudaMemsetAsync(dwq, 0, rot->D * we, s);
        if (dwk && e == cudaSuccess) e = cudaMemsetAsync(dwk, 0, rot->D * we, s);
        return status_of(e);
    }
    if (!rq != !rk || (wq && !rq)) return SGA_EINVAL;
    for (const void *p : {Q, K, dQo, dKo, static_cast<const void *>(dQ), static_cast<const void *>(dK)})
        if (!p || !aligned(p, 16)) return SGA_EINVAL;
    if (!pos || !aligned(pos, pos_bytes) || !aligned(rq, 4) || !aligned(rk, 4)) return SGA_EINVAL;
    if (dwq) {
        if (!workspace || !aligned(workspace, 16)) return SGA_EINVAL;
        if (workspace_bytes < sga_qk_norm_rope_bwd_workspace_bytes(T, rot->D)) return SGA_EWORKSPACE;
    }
    RopeArgs a{};
    a.rot = *rot;
    a.Q = Q;
    a.K = K;
    a.pos = pos;
    a.wq = wq;
    a.wk = wk;
    a.rq_in = rq;
    a.rk_in = rk;
    a.dQo = dQo;
    a.dKo = dKo;
    a.Qo = dQ;
    a.Ko = dK;
    a.part = dwq ? static_cast<float *>(workspace) : nullptr;
    a.T = T;
    a.ldq = ldq;
    a.ldk = ldk;
    a.H = H;
    a.Hkv = Hkv;
    a.wide = pos_bytes == 8;
    return status_of(by_type(rot->D, dt, wdt, [&](auto t, auto w, auto d) { return launch_bwd<decltype(t), decltype(w), decltype(d)::value>(a, dwq, dwk, s); }));
}

}  // extern "C"
