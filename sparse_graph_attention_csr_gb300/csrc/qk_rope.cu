// Norm of every query and key head and their rotary positions, in one pass over
// them, forward and backward.
//   r = 1 / sqrt(sum x^2 / D + eps),  y = x r w   (per head; w [D], shared by the heads)
//   a pair (y_a, y_b) at position p turns by the angle p f of its frequency:
//     (y_a cos - y_b sin, y_a sin + y_b cos)
//   backward: dn = the gradient turned back, xhat = x r, g = dn w,
//     dx = r (g - xhat sum(g xhat) / D),  dw = sum over rows and heads of dn xhat
//
// Bound by DRAM: the forward reads and writes Q and K once, the backward reads
// them and their gradients and writes one gradient.  A row belongs to a group of D /
// (2 EL) lanes, which take its heads one after the other: a lane holds two 16-byte
// chunks of a head with both elements of its pairs, so a rotation needs no exchange,
// and the cosines and sines of its pairs, formed once a row, and its columns'
// weights stay in registers.  (With a block's rows and heads dealt to its groups,
// turns and weights through shared memory, instructions bound it: 69636 rows of
// 16/4 heads of 128 bf16 216 us forward, 255 backward.)  Where rows are few their
// heads are dealt to several groups.
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
#include <type_traits>

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

constexpr int kThreads = 128;   // of a block

struct RopeArgs {
    sga_rotary rot;
    const void *Q, *K, *pos, *wq, *wk, *dQo, *dKo;
    void *Qo, *Ko;           // forward: results; backward: dQ, dK
    float *rq, *rk;          // 1 / sqrt of the mean square (forward: written; null: rotation alone)
    const float *rq_in, *rk_in;
    float *part;             // [blocks][2][D] sums of dwq, dwk, or null
    int64_t T, ldq, ldk;     // rows; elements from a row of Q, K to the next
    int H, Hkv;
    int per, parts, qparts;  // heads a group takes at a time (0: all of a row's); shares of a row, those of its queries
    float eps;
    int wide;                // 64-bit positions
};

template <typename T> __device__ __forceinline__ uint4 load16(const T *p) { return *reinterpret_cast<const uint4 *>(p); }

// A lane's 2 EL elements of a head as the first (a) and second (b) elements of its
// EL pairs.
//   halves: pair i is elements (i, i + rot / 2); the lane's chunks are that far apart,
//     a one, b the other; chunks past the rotated ones follow by twos.
//   interleaved: pair i is elements (2 i, 2 i + 1); the chunks are half a head apart,
//     a their even elements, b their odd ones.
template <typename T, int D, bool INTER> struct Lane {
    static constexpr int EL = Elt<T>::EL, G = D / (2 * EL);
    int c0, c1;   // chunks (offsets in elements)
    int lane, rot;
    __device__ __forceinline__ Lane(const sga_rotary &r, int l) : lane(l), rot(r.rot) {
        const int half = r.rot / (2 * EL);
        c0 = EL * (INTER || lane < half ? lane : 2 * lane);   // (2 half + 2 (lane - half))
        c1 = INTER ? c0 + EL * G : lane < half ? c0 + EL * half : c0 + EL;
    }
    // the pair that the lane's e-th is (of those that turn), or past rot / 2
    __device__ __forceinline__ int pair(int e) const {
        if (INTER) return e < EL / 2 ? lane * (EL / 2) + e : (lane + G) * (EL / 2) + e - EL / 2;
        return lane * EL + e;
    }
    __device__ __forceinline__ static void split(const uint4 &x, const uint4 &y, float *a, float *b) {
        float t[2 * EL];
        unpack<T>(x, t);
        unpack<T>(y, t + EL);
#pragma unroll
        for (int e = 0; e < EL; ++e) {
            a[e] = t[INTER ? 2 * e : e];
            b[e] = t[INTER ? 2 * e + 1 : EL + e];
        }
    }
    __device__ __forceinline__ void load(const T *head, uint4 *raw) const {
        raw[0] = load16(head + c0);
        raw[1] = load16(head + c1);
    }
    __device__ __forceinline__ void store(T *head, const float *a, const float *b) const {
        float t[2 * EL];
#pragma unroll
        for (int e = 0; e < EL; ++e) {
            t[INTER ? 2 * e : e] = a[e];
            t[INTER ? 2 * e + 1 : EL + e] = b[e];
        }
        *reinterpret_cast<uint4 *>(head + c0) = pack<T>(t);
        *reinterpret_cast<uint4 *>(head + c1) = pack<T>(t + EL);
    }
    // where element i of (a, b) lies in a head
    __device__ __forceinline__ int column(bool second, int e) const {
        const int i = INTER ? 2 * e + second : e;
        return (INTER ? i < EL : !second) ? c0 + i : c1 + (INTER ? i - EL : i);
    }
    // the weights of the lane's columns, ones without
    template <typename TW> __device__ __forceinline__ void weights(const TW *w, float *a, float *b) const {
#pragma unroll
        for (int e = 0; e < EL; ++e) {
            a[e] = w ? to_f32<TW>(w[column(false, e)]) : 1.f;
            b[e] = w ? to_f32<TW>(w[column(true, e)]) : 1.f;
        }
    }
    // cosines and sines of the row's angles; pairs that do not turn: 1 and 0
    __device__ __forceinline__ void turns(const RopeArgs &a, int64_t row, float *c, float *s) const {
        const sga_rotary &r = a.rot;
        int64_t p = 0;
        int axis = -1;
#pragma unroll
        for (int e = 0; e < EL; ++e) {
            const int i = pair(e);
            c[e] = 1.f;
            s[e] = 0.f;
            if (2 * i >= rot) continue;
            if (r.axis[i] != axis) {
                axis = r.axis[i];
                const int64_t at = row * r.axes + axis;
                p = a.wide ? (int64_t)__ldg(static_cast<const long long *>(a.pos) + at) : (int64_t)__ldg(static_cast<const int *>(a.pos) + at);
            }
            // half turns in [-1, 1): the top 32 bits, rounded
            const uint64_t turn = (uint64_t)p * r.turn[i];
            sincospif((float)(int32_t)(uint32_t)((turn + 0x80000000ull) >> 32) * 0x1p-31f, s + e, c + e);
        }
    }
    // (a, b) turned (BACK: by the negative angles).  What does not turn stays bit for
    // bit (0 times an infinity would not).
    template <bool BACK> __device__ __forceinline__ void turn(float *a, float *b, const float *c, const float *s) const {
#pragma unroll
        for (int e = 0; e < EL; e += 2) {
            const float2 u = make_float2(a[e], a[e + 1]), v = make_float2(b[e], b[e + 1]), cc = make_float2(c[e], c[e + 1]),
                         ss = make_float2(s[e], s[e + 1]), ns = make_float2(-s[e], -s[e + 1]);
            const float2 x = ffma2(v, BACK ? ss : ns, fmul2(u, cc)), y = ffma2(u, BACK ? ns : ss, fmul2(v, cc));
            if (2 * pair(e) < rot) {
                a[e] = x.x;
                b[e] = y.x;
            }
            if (2 * pair(e + 1) < rot) {
                a[e + 1] = x.y;
                b[e + 1] = y.y;
            }
        }
    }
};

template <int EL> __device__ __forceinline__ void mul(float *x, const float *y) {
#pragma unroll
    for (int e = 0; e < EL; e += 2) {
        const float2 t = fmul2(make_float2(x[e], x[e + 1]), make_float2(y[e], y[e + 1]));
        x[e] = t.x;
        x[e + 1] = t.y;
    }
}
template <int EL> __device__ __forceinline__ void mul(float *x, float y) {
#pragma unroll
    for (int e = 0; e < EL; e += 2) {
        const float2 t = fmul2(make_float2(x[e], x[e + 1]), make_float2(y, y));
        x[e] = t.x;
        x[e + 1] = t.y;
    }
}

// A group's share of a row: all of its heads, or `per` of its queries' or keys'.
struct Share {
    int64_t row;
    bool in;
    int part;
    __device__ __forceinline__ Share(const RopeArgs &a, int64_t u) {
        row = a.per ? u / a.parts : u;
        part = a.per ? (int)(u - row * a.parts) : 0;
        in = row < a.T;
    }
};
// Calls phase(keys, first head, end, steps): the steps are the same in all groups of
// a warp, whose sums are warp-wide calls.
template <typename F> __device__ __forceinline__ void each_phase(const RopeArgs &a, const Share &s, F phase) {
    if (a.per == 0) {
        phase(false, 0, s.in ? a.H : 0, a.H);
        phase(true, 0, s.in ? a.Hkv : 0, a.Hkv);
    } else {
        const bool key = s.part >= a.qparts;
        const int h0 = (key ? s.part - a.qparts : s.part) * a.per;
        phase(key, h0, s.in ? min(key ? a.Hkv : a.H, h0 + a.per) : h0, a.per);
    }
}

template <typename T, typename TW, int D, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_rope_fwd_kernel(const __grid_constant__ RopeArgs a) {
    using L = Lane<T, D, INTER>;
    constexpr int EL = L::EL, G = L::G, U = 4;
    let_next_start();
    wait_previous();
    const L at(a.rot, threadIdx.x % G);
    const bool norm = a.rq != nullptr;
    const int64_t units = a.T * a.parts, step = (int64_t)gridDim.x * (kThreads / G);
    // (whole warps: a group past the last row takes part in the sums)
    for (int64_t u0 = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / 32 * (32 / G); u0 < units; u0 += step) {
        const Share sh(a, u0 + threadIdx.x % 32 / G);
        float c[EL], s[EL];
        bool turned = false;
        each_phase(a, sh, [&](bool key, int h0, int h1, int steps) {
            const T *src = static_cast<const T *>(key ? a.K : a.Q) + (sh.in ? sh.row : 0) * (key ? a.ldk : a.ldq) + h0 * D;
            T *dst = static_cast<T *>(key ? a.Ko : a.Qo) + ((sh.in ? sh.row : 0) * (key ? a.Hkv : a.H) + h0) * D;
            float *r = norm ? (key ? a.rk : a.rq) + (sh.in ? sh.row : 0) * (key ? a.Hkv : a.H) + h0 : nullptr;
            const int n = h1 - h0;
            uint4 x[U][2];
            auto fetch = [&](int u, int i) {
                x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
                if (i < n) at.load(src + i * D, x[u]);
            };
#pragma unroll
            for (int u = 0; u < U; ++u) fetch(u, u);
            float wa[EL], wb[EL];
            at.template weights<TW>(static_cast<const TW *>(key ? a.wk : a.wq), wa, wb);
            if (!turned && sh.in) at.turns(a, sh.row, c, s);   // (while the first heads arrive)
            turned = true;
            for (int i0 = 0; i0 < steps; i0 += U) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u;
                    float ya[EL], yb[EL];
                    L::split(x[u][0], x[u][1], ya, yb);
                    fetch(u, i + U);
                    if (norm) {
                        float2 q = make_float2(0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < EL; e += 2) {
                            const float2 va = make_float2(ya[e], ya[e + 1]), vb = make_float2(yb[e], yb[e + 1]);
                            q = ffma2(vb, vb, ffma2(va, va, q));
                        }
                        const float inv = rsqrtf(group_sum<G>(q.x + q.y) * (1.f / D) + a.eps);
                        mul<EL>(ya, inv);
                        mul<EL>(yb, inv);
                        mul<EL>(ya, wa);
                        mul<EL>(yb, wb);
                        if (at.lane == 0 && i < n) r[i] = inv;
                    }
                    if (i < n) {
                        at.template turn<false>(ya, yb, c, s);
                        at.store(dst + i * D, ya, yb);
                    }
                }
            }
        });
    }
}

// A block's sums of one weight's gradient: the groups of a warp first (lanes G
// apart), then the warps in order.
template <typename L, int D> __device__ __forceinline__ void block_sums(float *sm, const float *sa, const float *sb, const L &at, float *out) {
    constexpr int EL = L::EL, G = L::G;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2 * EL; ++i) {
        float t = i < EL ? sa[i % EL] : sb[i % EL];
#pragma unroll
        for (int o = 16; o >= G; o >>= 1) t += __shfl_xor_sync(SGA_FULL_MASK, t, o);
        if (threadIdx.x % 32 < G) sm[threadIdx.x / 32 * D + at.column(i >= EL, i % EL)] = t;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kThreads) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) t += sm[k * D + i];
        out[i] = t;
    }
}

// Blocks an SM of the backward pass, each with a row of sums, and heads in flight: as
// registers allow (69636 rows of 16/4 heads of 128 bf16 192 us with three blocks and
// two heads, 202 with four blocks, or one head; 30011 rows of 4/4 heads of 64 fp32 38
// with three blocks and four heads, 39 with four blocks, 42 and 46 with four and three
// of two).
constexpr int kBwdBlocksPerSm = 3;

// The queries of all rows, then the keys: one weight's sums at a time in registers,
// which pays for forming the turns again (another pair would leave room for fewer blocks).
template <typename T, typename TW, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, kBwdBlocksPerSm) qk_rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
    using L = Lane<T, D, INTER>;
    constexpr int EL = L::EL, G = L::G, U = sizeof(T) == 4 ? 4 : 2;
    __shared__ float sums[kThreads / 32 * D];
    let_next_start();
    wait_previous();
    const L at(a.rot, threadIdx.x % G);
    const bool norm = a.rq_in != nullptr;
    const int64_t step = (int64_t)gridDim.x * (kThreads / G);
    for (int key = 0; key < 2; ++key) {
        const int heads = key ? a.Hkv : a.H, steps = a.per ? a.per : heads, parts = a.per ? (heads + a.per - 1) / a.per : 1;
        const int64_t units = a.T * parts;
        float wa[EL], wb[EL], sa[EL], sb[EL];
        at.template weights<TW>(static_cast<const TW *>(key ? a.wk : a.wq), wa, wb);
#pragma unroll
        for (int e = 0; e < EL; ++e) sa[e] = sb[e] = 0.f;   // this thread's sums of the weight's gradient
        for (int64_t u0 = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / 32 * (32 / G); u0 < units; u0 += step) {
            const int64_t unit = u0 + threadIdx.x % 32 / G;
            const bool in = unit < units;
            const int64_t row = !in ? 0 : a.per ? unit / parts : unit;
            const int h0 = in && a.per ? (int)(unit - row * parts) * a.per : 0, n = in ? min(heads - h0, steps) : 0;
            const int64_t first = row * heads + h0;
            const T *src = static_cast<const T *>(key ? a.K : a.Q) + row * (key ? a.ldk : a.ldq) + h0 * D;
            const T *grad = static_cast<const T *>(key ? a.dKo : a.dQo) + first * D;
            const float *r = norm ? (key ? a.rk_in : a.rq_in) + first : nullptr;
            T *dst = static_cast<T *>(key ? a.Ko : a.Qo) + first * D;
            uint4 x[U][2], g[U][2];
            float inv[U];
            auto fetch = [&](int u, int i) {
                x[u][0] = x[u][1] = g[u][0] = g[u][1] = make_uint4(0, 0, 0, 0);
                inv[u] = 0.f;
                if (i < n) {
                    at.load(grad + i * D, g[u]);
                    if (norm) {
                        at.load(src + i * D, x[u]);
                        inv[u] = r[i];
                    }
                }
            };
#pragma unroll
            for (int u = 0; u < U; ++u) fetch(u, u);
            float c[EL], s[EL];
            at.turns(a, row, c, s);   // (while the first heads arrive)
            for (int i0 = 0; i0 < steps; i0 += U) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u;
                    float da[EL], db[EL];
                    L::split(g[u][0], g[u][1], da, db);
                    const uint4 x0 = x[u][0], x1 = x[u][1];
                    const float rr = inv[u];
                    fetch(u, i + U);
                    if (i < n) at.template turn<true>(da, db, c, s);
                    if (norm) {
                        float xa[EL], xb[EL];
                        L::split(x0, x1, xa, xb);
                        mul<EL>(xa, rr);
                        mul<EL>(xb, rr);
#pragma unroll
                        for (int e = 0; e < EL; e += 2) {
                            const float2 y = ffma2(make_float2(da[e], da[e + 1]), make_float2(xa[e], xa[e + 1]), make_float2(sa[e], sa[e + 1]));
                            const float2 z = ffma2(make_float2(db[e], db[e + 1]), make_float2(xb[e], xb[e + 1]), make_float2(sb[e], sb[e + 1]));
                            sa[e] = y.x;
                            sa[e + 1] = y.y;
                            sb[e] = z.x;
                            sb[e + 1] = z.y;
                        }
                        mul<EL>(da, wa);
                        mul<EL>(db, wb);
                        float2 q = make_float2(0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < EL; e += 2)
                            q = ffma2(make_float2(db[e], db[e + 1]), make_float2(xb[e], xb[e + 1]),
                                      ffma2(make_float2(da[e], da[e + 1]), make_float2(xa[e], xa[e + 1]), q));
                        const float m = -group_sum<G>(q.x + q.y) * (1.f / D);
                        const float2 mm = make_float2(m, m), ri = make_float2(rr, rr);
#pragma unroll
                        for (int e = 0; e < EL; e += 2) {
                            const float2 y = fmul2(ri, ffma2(mm, make_float2(xa[e], xa[e + 1]), make_float2(da[e], da[e + 1])));
                            const float2 z = fmul2(ri, ffma2(mm, make_float2(xb[e], xb[e + 1]), make_float2(db[e], db[e + 1])));
                            da[e] = y.x;
                            da[e + 1] = y.y;
                            db[e] = z.x;
                            db[e + 1] = z.y;
                        }
                    }
                    if (i < n) at.store(dst + i * D, da, db);
                }
            }
        }
        if (a.part) block_sums<L, D>(sums, sa, sb, at, a.part + (int64_t)blockIdx.x * 2 * D + key * D);
    }
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

// Deals a row's heads to several groups where one group a row would leave SMs
// without work, four heads at least each (or all of a row's).
void deal_heads(RopeArgs &a, int groups) {
    const int64_t want = (int64_t)device_sms() * groups * 2;
    a.per = 0;
    a.parts = 1;
    if (a.T >= want || a.H + a.Hkv <= 4) return;
    const int64_t share = std::min<int64_t>((want + a.T - 1) / a.T, (a.H + a.Hkv + 3) / 4);   // shares of a row
    a.per = (int)((a.H + a.Hkv + share - 1) / share);
    a.qparts = (a.H + a.per - 1) / a.per;
    a.parts = a.qparts + (a.Hkv + a.per - 1) / a.per;
}

template <typename T, typename TW, int D, bool INTER> cudaError_t launch_fwd(RopeArgs &a, cudaStream_t s) {
    constexpr int groups = kThreads / Lane<T, D, INTER>::G;
    deal_heads(a, groups);
    const int64_t blocks = std::min<int64_t>((a.T * a.parts + groups - 1) / groups, (int64_t)device_sms() * 64);
    note_launch(SGA_KERN_QK_ROPE_FWD, s, false);
    const cudaError_t e = launch_early(qk_rope_fwd_kernel<T, TW, D, INTER>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
    note_launch(SGA_KERN_QK_ROPE_FWD, s, true);
    return e;
}

template <typename T, typename TW, int D, bool INTER> cudaError_t launch_bwd(RopeArgs &a, void *dwq, void *dwk, cudaStream_t s) {
    constexpr int groups = kThreads / Lane<T, D, INTER>::G;
    deal_heads(a, groups);
    // as many blocks as are resident at once
    static std::atomic<int> per_sm[kMaxDevices];
    cudaError_t asked = cudaSuccess;
    const int fit = per_device(per_sm, [&] {
        int n = 0;
        asked = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, qk_rope_bwd_kernel<T, TW, D, INTER>, kThreads, 0);
        return asked == cudaSuccess ? std::max(1, std::min(n, kBwdBlocksPerSm)) : 0;
    });
    if (asked != cudaSuccess) return asked;
    const int blocks = (int)std::min<int64_t>((a.T * a.parts + groups - 1) / groups, (int64_t)device_sms() * fit);
    note_launch(SGA_KERN_QK_ROPE_BWD, s, false);
    cudaError_t e = launch_early(qk_rope_bwd_kernel<T, TW, D, INTER>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
    note_launch(SGA_KERN_QK_ROPE_BWD, s, true);
    if (e != cudaSuccess || !a.part) return e;
    note_launch(SGA_KERN_QK_ROPE_REDUCE, s, false);
    e = launch_early(qk_rope_reduce_kernel<TW>, dim3(2 * D / 32), dim3(1024), 0, s, static_cast<const float *>(a.part), blocks, D,
                     static_cast<TW *>(dwq), static_cast<TW *>(dwk));
    note_launch(SGA_KERN_QK_ROPE_REDUCE, s, true);
    return e;
}

template <typename F> cudaError_t by_type(const sga_rotary &r, sga_dtype dt, sga_dtype wdt, F f) {
    auto pairing = [&](auto t, auto w, auto d) { return r.interleaved ? f(t, w, d, std::true_type()) : f(t, w, d, std::false_type()); };
    auto width = [&](auto t, auto w) {
        return r.D == 32 ? pairing(t, w, std::integral_constant<int, 32>())
               : r.D == 64 ? pairing(t, w, std::integral_constant<int, 64>()) : pairing(t, w, std::integral_constant<int, 128>());
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
    return status_of(by_type(*rot, dt, wdt, [&](auto t, auto w, auto d, auto i) {
        return launch_fwd<decltype(t), decltype(w), decltype(d)::value, decltype(i)::value>(a, s);
    }));
}

size_t sga_qk_norm_rope_bwd_workspace_bytes(int64_t T, int D) {
    if (T <= 0 || D <= 0) return 0;
    return (size_t)device_sms() * kBwdBlocksPerSm * 2 * (size_t)D * sizeof(float);
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
    return status_of(by_type(*rot, dt, wdt, [&](auto t, auto w, auto d, auto i) {
        return launch_bwd<decltype(t), decltype(w), decltype(d)::value, decltype(i)::value>(a, dwq, dwk, s);
    }));
}

}  // extern "C"
