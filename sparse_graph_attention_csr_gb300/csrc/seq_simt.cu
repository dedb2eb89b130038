// Packed-sequence attention in fp32, on the FMA pipes, and the row terms of
// the backward pass for both dtypes.
//
// The tensor cores have no fp32 product, and the tolerance of the fp32 layers
// (1e-5) rules out tf32, so these kernels are bound by the FMA pipes (two
// products of the forward, three and four of the backward's two passes).
// Blocks of 256 threads (16 x 16) take a 64-row tile of one side and walk the
// 64-row tiles of the other through shared memory, the next tiles copied while
// one is in use; each thread holds a 4 x 4 piece of the scores and a 4 x D/16
// piece of the result.  Tiles are row-major with rows of D + 4 floats: both
// products read them 16 bytes at a time along a row without bank conflicts, so
// no tile is stored transposed.  Two blocks an SM where registers and shared
// memory allow (forward, 2048 rows, 8 heads of 64, full: 366 -> 285 us, 30
// TFLOP/s; backward with D = 32 593 -> 496 us; with D = 64 it spills and loses).
//   forward: S = Q K^T, online softmax (running maximum and sum per row),
//     O = O alpha + P V;
//   dQ pass (a tile of queries): S, dP = dOut V^T, dS = P (dP - Delta),
//     dQ += dS K;
//   dK/dV pass (a tile of keys, over the query heads of its group): S^T =
//     K Q^T, dP^T = V dOut^T, dV += P^T dOut, dK += dS^T Q.
// The scores are computed twice in the backward pass so that every output row
// is owned by one block: no atomics, bitwise reproducible.
// A row whose result is not finite is computed again over its own interval alone
// (seq_rows.cuh).  Leaving masked pairs out of every sum instead, with a test a
// pair, took 78 instead of 66 us on five sequences of 1 to 512 rows, D = 32.
#include "seq_rows.cuh"
#include "tc.cuh"

namespace sga {
namespace {

constexpr int kT = 64;         // rows of a tile
constexpr int kThreads = 256;
constexpr int kPP = kT + 4;    // pitch of a score tile

template <int D> constexpr int kPitch = D + 4;
template <int D> constexpr int kTileFloats = kT * (D + 4);
constexpr int kScoreFloats = kT * kPP;

// rows [r0, r0 + 64) of head h of a [T][heads][D] tensor, asynchronously (rows
// past `rows` as zeros)
template <int D>
__device__ __forceinline__ void load_tile(float *dst, const void *src, int64_t r0, int64_t rows, int heads, int h) {
    constexpr int C4 = D / 4;
    for (int i = threadIdx.x; i < kT * C4; i += kThreads) {
        const int r = i / C4, c = i % C4;
        const bool in = r0 + r < rows;
        tc::cp16(tc::smem_u32(dst + r * kPitch<D> + 4 * c),
                 static_cast<const float *>(src) + ((in ? r0 + r : 0) * heads + h) * D + 4 * c, in);
    }
}

// s[a][c] = row (ty + 16 a) of A . row (tx + 16 c) of B
template <int D>
__device__ __forceinline__ void dot_tiles(float (&s)[4][4], const float *A, const float *B, int ty, int tx) {
    float2 acc[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[a][c] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) x[a] = *reinterpret_cast<const float4 *>(A + (ty + 16 * a) * kPitch<D> + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = *reinterpret_cast<const float4 *>(B + (tx + 16 * c) * kPitch<D> + d);
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                acc[a][c] = ffma2(make_float2(x[a].x, x[a].y), make_float2(y[c].x, y[c].y), acc[a][c]);
                acc[a][c] = ffma2(make_float2(x[a].z, x[a].w), make_float2(y[c].z, y[c].w), acc[a][c]);
            }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[a][c] = acc[a][c].x + acc[a][c].y;
}

// Columns of the result that a thread holds: 4 tx .. + 3 (and + 64 for D =
// 128); 2 tx, 2 tx + 1 for D = 32.
template <int D> constexpr int kCols = D / 16;
template <int D> __device__ __forceinline__ int col_of(int tx, int x) {
    return D == 32 ? 2 * tx + x : 4 * tx + (x & 3) + 64 * (x >> 2);
}

template <int D> __device__ __forceinline__ void load_cols(float (&v)[kCols<D>], const float *row, int tx) {
    if constexpr (D == 32) {
        const float2 t = *reinterpret_cast<const float2 *>(row + 2 * tx);
        v[0] = t.x;
        v[1] = t.y;
    } else {
#pragma unroll
        for (int x = 0; x < kCols<D>; x += 4) {
            const float4 t = *reinterpret_cast<const float4 *>(row + 4 * tx + 16 * x);
            v[x] = t.x;
            v[x + 1] = t.y;
            v[x + 2] = t.z;
            v[x + 3] = t.w;
        }
    }
}

// acc[a][x] += sum_j P[ty + 16 a][j] B[j][col x] over the 64 rows of B
template <int D>
__device__ __forceinline__ void add_product(float (&acc)[4][kCols<D>], const float *P, const float *B, int ty, int tx) {
    constexpr int NC = kCols<D>;
#pragma unroll 2
    for (int j = 0; j < kT; j += 4) {
        float4 p[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) p[a] = *reinterpret_cast<const float4 *>(P + (ty + 16 * a) * kPP + j);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float v[NC];
            load_cols<D>(v, B + (j + u) * kPitch<D>, tx);
#pragma unroll
            for (int a = 0; a < 4; ++a) axpy2<NC>(acc[a], u == 0 ? p[a].x : u == 1 ? p[a].y : u == 2 ? p[a].z : p[a].w, v);
        }
    }
}

// Stores the rows, scaled, and returns whether any element of this thread's row
// a was not finite, as bit a.
template <int D>
__device__ __forceinline__ uint32_t store_rows(float *dst, const float (&acc)[4][kCols<D>], const float (&f)[4], int64_t r0,
                                               int64_t rows, int heads, int h, int ty, int tx) {
    uint32_t bad = 0;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const int64_t row = r0 + ty + 16 * a;
        if (row >= rows) continue;
        float *o = dst + (row * heads + h) * D;
#pragma unroll
        for (int x = 0; x < kCols<D>; ++x) {
            const float y = acc[a][x] * f[a];
            o[col_of<D>(tx, x)] = y;
            if (!(fabsf(y) < INFINITY)) bad |= 1u << a;
        }
    }
    return bad;
}

// Calls redo(a, half) for every row (ty + 16 a of the warp's half) of which a
// thread found an element that is not finite; the warp together, after its stores.
template <typename F> __device__ __forceinline__ void each_bad_row(uint32_t bad, F redo) {
    if (!__any_sync(SGA_FULL_MASK, bad != 0)) return;
    __syncwarp();
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const uint32_t who = __ballot_sync(SGA_FULL_MASK, (bad >> a) & 1u);
        for (int half = 0; half < 2; ++half)
            if ((who >> (16 * half)) & 0xffffu) redo(a, half);
    }
}

__device__ __forceinline__ float half_max(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(SGA_FULL_MASK, v, o));
    return v;
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(SGA_FULL_MASK, v, o);
    return v;
}

// What each of a thread's four rows sees: queries of a key row, or keys of a
// query row.  Rows past the last see nothing.
__device__ __forceinline__ void intervals(const SeqArgs &a, bool keys, int64_t r0, int ty, int64_t (&lo)[4], int64_t (&hi)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = r0 + ty + 16 * i;
        lo[i] = hi[i] = 0;
        if (row < a.rows) {
            const int2 se = __ldg(a.range + row);
            lo[i] = keys && a.causal ? row : se.x;
            hi[i] = !keys && a.causal ? row + 1 : se.y;
        }
    }
}
__device__ __forceinline__ void in_tile(const int64_t (&lo)[4], const int64_t (&hi)[4], int64_t t0, int (&l)[4], int (&h)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        l[i] = (int)max((int64_t)0, min((int64_t)kT, lo[i] - t0));
        h[i] = (int)max((int64_t)0, min((int64_t)kT, hi[i] - t0));
    }
}

// ---- forward ------------------------------------------------------------------

template <int D> __global__ void __launch_bounds__(kThreads, D < 128 ? 2 : 1) seq_fwd_f32_kernel(const SeqArgs a) {
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *sK = sQ + kTileFloats<D>, *sV = sK + kTileFloats<D>, *sP = sV + kTileFloats<D>;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const SeqTile t = a.qtiles[blockIdx.x / a.H];
    const int h = blockIdx.x % a.H, hk = h / (a.H / a.Hkv);
    const int64_t q0 = (int64_t)t.tile * kT;
    const float scale2 = a.scale * kLog2e;
    load_tile<D>(sQ, a.Q, q0, a.rows, a.H, h);
    load_tile<D>(sK, a.K, (int64_t)t.t0 * kT, a.rows, a.Hkv, hk);
    tc::cp_commit();
    load_tile<D>(sV, a.V, (int64_t)t.t0 * kT, a.rows, a.Hkv, hk);
    tc::cp_commit();
    int64_t lo[4], hi[4];
    intervals(a, false, q0, ty, lo, hi);
    float m[4], l[4], acc[4][kCols<D>];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int x = 0; x < kCols<D>; ++x) acc[i][x] = 0.f;
    }
    for (int kt = t.t0; kt < t.t1; ++kt) {
        const int64_t k0 = (int64_t)kt * kT;
        const bool full = kt >= t.f0 && kt < t.f1;
        int kl[4], kh[4];
        in_tile(lo, hi, k0, kl, kh);
        tc::cp_wait<1>();   // this K (V may be on its way)
        __syncthreads();
        float s[4][4];
        dot_tiles<D>(s, sQ, sK, ty, tx);
        __syncthreads();
        if (kt + 1 < t.t1) load_tile<D>(sK, a.K, k0 + kT, a.rows, a.Hkv, hk);   // beside the softmax and P V
        tc::cp_commit();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int j = tx + 16 * c;
                s[i][c] = full || (j >= kl[i] && j < kh[i]) ? s[i][c] * scale2 : -INFINITY;
                mx = fmaxf(mx, s[i][c]);
            }
            const float mn = fmaxf(m[i], half_max(mx));
            const float al = exp2_diff(m[i], mn);
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float p = exp2_diff(s[i][c], mn);
                sP[(ty + 16 * i) * kPP + tx + 16 * c] = p;
                sum += p;
            }
            l[i] = l[i] * al + half_sum(sum);
            m[i] = mn;
#pragma unroll
            for (int x = 0; x < kCols<D>; ++x) acc[i][x] *= al;
        }
        tc::cp_wait<1>();   // this V
        __syncthreads();
        add_product<D>(acc, sP, sV, ty, tx);
        __syncthreads();
        if (kt + 1 < t.t1) load_tile<D>(sV, a.V, k0 + kT, a.rows, a.Hkv, hk);   // beside the next scores
        tc::cp_commit();
    }
    float inv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        inv[i] = 1.f / l[i];
        const int64_t row = q0 + ty + 16 * i;
        if (tx == 0 && row < a.rows) a.lse_w[row * a.H + h] = (m[i] + log2f(l[i])) * kLn2;
    }
    const uint32_t bad = store_rows<D>(static_cast<float *>(a.out_w), acc, inv, q0, a.rows, a.H, h, ty, tx);
    each_bad_row(bad, [&](int i, int half) {
        seq::out_row_alone<float, D>(a, q0 + (ty & ~1) + half + 16 * i, h, hk, __shfl_sync(SGA_FULL_MASK, lo[i], 16 * half),
                                     __shfl_sync(SGA_FULL_MASK, hi[i], 16 * half));
    });
}

// ---- backward -------------------------------------------------------------------

template <int D> __device__ __forceinline__ void dq_pass(const SeqArgs &a, float *sm, uint32_t unit) {
    float *sQ = sm, *sG = sQ + kTileFloats<D>, *sV = sG + kTileFloats<D>, *sP = sV + kTileFloats<D>,
          *sK = sP + kScoreFloats;   // two K tiles
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const SeqTile t = a.qtiles[unit / a.H];
    const int h = unit % a.H, hk = h / (a.H / a.Hkv);
    const int64_t q0 = (int64_t)t.tile * kT;
    const float scale2 = a.scale * kLog2e;
    load_tile<D>(sQ, a.Q, q0, a.rows, a.H, h);
    load_tile<D>(sG, a.dOut, q0, a.rows, a.H, h);
    load_tile<D>(sK, a.K, (int64_t)t.t0 * kT, a.rows, a.Hkv, hk);
    load_tile<D>(sV, a.V, (int64_t)t.t0 * kT, a.rows, a.Hkv, hk);
    tc::cp_commit();
    int64_t lo[4], hi[4];
    intervals(a, false, q0, ty, lo, hi);
    float ls[4], dl[4], acc[4][kCols<D>];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = (int64_t)h * a.rows_pad + q0 + ty + 16 * i;
        ls[i] = a.ws_nlse[r];
        dl[i] = a.ws_ndelta[r];
#pragma unroll
        for (int x = 0; x < kCols<D>; ++x) acc[i][x] = 0.f;
    }
    for (int kt = t.t0; kt < t.t1; ++kt) {
        const int64_t k0 = (int64_t)kt * kT;
        const bool full = kt >= t.f0 && kt < t.f1;
        float *sKi = sK + (kt - t.t0) % 2 * kTileFloats<D>, *sKn = sK + (kt - t.t0 + 1) % 2 * kTileFloats<D>;
        int kl[4], kh[4];
        in_tile(lo, hi, k0, kl, kh);
        tc::cp_wait<0>();
        __syncthreads();   // this K and V; the last dS K is done with the other K and with dS
        if (kt + 1 < t.t1) load_tile<D>(sKn, a.K, k0 + kT, a.rows, a.Hkv, hk);
        float s[4][4], g[4][4];
        dot_tiles<D>(g, sG, sV, ty, tx);
        __syncthreads();
        if (kt + 1 < t.t1) load_tile<D>(sV, a.V, k0 + kT, a.rows, a.Hkv, hk);
        tc::cp_commit();
        dot_tiles<D>(s, sQ, sKi, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int j = tx + 16 * c;
                const bool on = full || (j >= kl[i] && j < kh[i]);
                sP[(ty + 16 * i) * kPP + j] = on ? fast_exp2(fmaf(s[i][c], scale2, ls[i])) * (g[i][c] + dl[i]) : 0.f;
            }
        __syncthreads();
        add_product<D>(acc, sP, sKi, ty, tx);
    }
    const float f[4] = {a.scale, a.scale, a.scale, a.scale};
    const uint32_t bad = store_rows<D>(static_cast<float *>(a.dQ), acc, f, q0, a.rows, a.H, h, ty, tx);
    each_bad_row(bad, [&](int i, int half) {
        seq::query_row_alone<float, D>(a, q0 + (ty & ~1) + half + 16 * i, h, __shfl_sync(SGA_FULL_MASK, lo[i], 16 * half),
                                       __shfl_sync(SGA_FULL_MASK, hi[i], 16 * half), 0, D);
    });
}

template <int D> __device__ __forceinline__ void dkdv_pass(const SeqArgs &a, float *sm, uint32_t unit) {
    float *sK = sm, *sV = sK + kTileFloats<D>, *sP = sV + kTileFloats<D>,
          *sS = sP + kScoreFloats;   // two pairs of Q and dOut tiles
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const SeqTile t = a.ktiles[unit / a.Hkv];
    const int hk = unit % a.Hkv, grp = a.H / a.Hkv;
    const int64_t k0 = (int64_t)t.tile * kT;
    const float scale2 = a.scale * kLog2e;
    const int nt = t.t1 - t.t0, n = nt * grp;   // steps: (head of the group, query tile)
    auto fetch = [&](int i) {
        float *dst = sS + i % 2 * 2 * kTileFloats<D>;
        const int64_t q0 = (int64_t)(t.t0 + i % nt) * kT;
        load_tile<D>(dst, a.Q, q0, a.rows, a.H, hk * grp + i / nt);
        load_tile<D>(dst + kTileFloats<D>, a.dOut, q0, a.rows, a.H, hk * grp + i / nt);
    };
    load_tile<D>(sK, a.K, k0, a.rows, a.Hkv, hk);
    load_tile<D>(sV, a.V, k0, a.rows, a.Hkv, hk);
    fetch(0);
    tc::cp_commit();
    int64_t lo[4], hi[4];
    intervals(a, true, k0, ty, lo, hi);
    float dk[4][kCols<D>], dv[4][kCols<D>];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < kCols<D>; ++x) dk[i][x] = dv[i][x] = 0.f;
    for (int step = 0; step < n; ++step) {
        const float *sQ = sS + step % 2 * 2 * kTileFloats<D>, *sG = sQ + kTileFloats<D>;
        const int qt = t.t0 + step % nt;
        const int64_t q0 = (int64_t)qt * kT;
        const bool full = qt >= t.f0 && qt < t.f1;
        int ql[4], qh[4];
        in_tile(lo, hi, q0, ql, qh);
        float ls[4], dl[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int64_t r = (int64_t)(hk * grp + step / nt) * a.rows_pad + q0 + tx + 16 * c;
            ls[c] = a.ws_nlse[r];
            dl[c] = a.ws_ndelta[r];
        }
        tc::cp_wait<0>();
        __syncthreads();   // these tiles; the last dS^T Q is done with the other ones and with dS
        if (step + 1 < n) fetch(step + 1);
        tc::cp_commit();
        float s[4][4], g[4][4];
        dot_tiles<D>(s, sK, sQ, ty, tx);
        dot_tiles<D>(g, sV, sG, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int j = tx + 16 * c;
                const bool on = full || (j >= ql[i] && j < qh[i]);
                const float p = on ? fast_exp2(fmaf(s[i][c], scale2, ls[c])) : 0.f;
                sP[(ty + 16 * i) * kPP + j] = p;
                g[i][c] = on ? p * (g[i][c] + dl[c]) : 0.f;
            }
        __syncthreads();
        add_product<D>(dv, sP, sG, ty, tx);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) sP[(ty + 16 * i) * kPP + tx + 16 * c] = g[i][c];   // dS^T over P^T
        __syncthreads();
        add_product<D>(dk, sP, sQ, ty, tx);
    }
    const float one[4] = {1.f, 1.f, 1.f, 1.f}, f[4] = {a.scale, a.scale, a.scale, a.scale};
    const uint32_t bad_v = store_rows<D>(static_cast<float *>(a.dV), dv, one, k0, a.rows, a.Hkv, hk, ty, tx);
    const uint32_t bad_k = store_rows<D>(static_cast<float *>(a.dK), dk, f, k0, a.rows, a.Hkv, hk, ty, tx);
    for (int x = 0; x < 2; ++x)
        each_bad_row(x ? bad_k : bad_v, [&](int i, int half) {
            seq::key_row_alone<float, D>(a, x == 1, k0 + (ty & ~1) + half + 16 * i, hk,
                                         __shfl_sync(SGA_FULL_MASK, lo[i], 16 * half),
                                         __shfl_sync(SGA_FULL_MASK, hi[i], 16 * half), 0, D);
        });
}

// Both passes in one launch, the dK/dV units (the longer ones) first.
template <int D> __global__ void __launch_bounds__(kThreads, D == 32 ? 2 : 1) seq_bwd_f32_kernel(const SeqArgs a) {
    extern __shared__ __align__(16) float sm[];
    const uint32_t kv = (uint32_t)a.n_tiles * a.Hkv;
    if (blockIdx.x < kv) dkdv_pass<D>(a, sm, blockIdx.x);
    else dq_pass<D>(a, sm, blockIdx.x - kv);
}

// Row terms: D / EL lanes of 16 bytes a (row, head), four of them in flight.
// Rows behind the last sequence (to the end of its tile) get -lse = -inf, so
// that their weights are zero, and Delta = 0.
constexpr int kTerms = 4;
template <typename T, int D> __global__ void __launch_bounds__(256) seq_row_terms_kernel(const SeqArgs a) {
    constexpr int EL = Elt<T>::EL, L = D / EL, G = 256 / L;   // G items of a block at a time
    const int sub = threadIdx.x % L;
    const int64_t n = a.rows_pad * a.H, g0 = (int64_t)blockIdx.x * (G * kTerms) + threadIdx.x / L;
    uint4 x[kTerms], y[kTerms];
#pragma unroll
    for (int k = 0; k < kTerms; ++k) {
        const int64_t g = g0 + k * G;
        x[k] = y[k] = make_uint4(0, 0, 0, 0);
        if (g < a.rows * a.H) {   // (an item's elements follow the one's before)
            x[k] = ldg16(static_cast<const T *>(a.out) + g * D + sub * EL);
            y[k] = ldg16(static_cast<const T *>(a.dOut) + g * D + sub * EL);
        }
    }
#pragma unroll
    for (int k = 0; k < kTerms; ++k) {
        const int64_t g = g0 + k * G;
        float u[EL], v[EL], d = 0.f;
        unpack<T>(x[k], u);
        unpack<T>(y[k], v);
#pragma unroll
        for (int i = 0; i < EL; ++i) d = fmaf(u[i], v[i], d);
        d = group_sum<L>(d);
        if (sub == 0 && g < n) {
            const int64_t row = g / a.H, at = (g % a.H) * a.rows_pad + row;
            const bool in = row < a.rows;
            a.ws_nlse[at] = in ? -(a.lse[g] * kLog2e) : -INFINITY;
            a.ws_ndelta[at] = in ? -d : 0.f;
        }
    }
}

template <int D> cudaError_t launch_fwd(const SeqArgs &a, cudaStream_t s) {
    constexpr size_t smem = sizeof(float) * (3 * kTileFloats<D> + kScoreFloats);
    if (cudaError_t e = allow_smem<seq_fwd_f32_kernel<D>>(smem); e != cudaSuccess) return e;
    note_launch(SGA_KERN_SEQ_FWD, s, false);
    seq_fwd_f32_kernel<D><<<(unsigned)((int64_t)a.n_tiles * a.H), kThreads, smem, s>>>(a);
    note_launch(SGA_KERN_SEQ_FWD, s, true);
    return cudaGetLastError();
}

template <int D> cudaError_t launch_bwd(const SeqArgs &a, cudaStream_t s) {
    constexpr size_t smem = sizeof(float) * (6 * kTileFloats<D> + kScoreFloats);   // (dK/dV; dQ takes a tile less)
    static_assert(smem <= 227 * 1024, "shared memory");
    cudaError_t e = allow_smem<seq_bwd_f32_kernel<D>>(smem);
    if (e == cudaSuccess) e = seq_row_terms<float>(a, D, s);
    if (e != cudaSuccess) return e;
    note_launch(SGA_KERN_SEQ_BWD, s, false);
    seq_bwd_f32_kernel<D><<<(unsigned)((int64_t)a.n_tiles * (a.Hkv + a.H)), kThreads, smem, s>>>(a);
    note_launch(SGA_KERN_SEQ_BWD, s, true);
    return cudaGetLastError();
}

template <typename T, int D> cudaError_t launch_terms(const SeqArgs &a, cudaStream_t s) {
    constexpr int per = kTerms * 256 / (D / Elt<T>::EL);   // items of a block
    note_launch(SGA_KERN_SEQ_BWD_ROWS, s, false);
    seq_row_terms_kernel<T, D><<<(unsigned)((a.rows_pad * a.H + per - 1) / per), 256, 0, s>>>(a);
    note_launch(SGA_KERN_SEQ_BWD_ROWS, s, true);
    return cudaGetLastError();
}

}  // namespace

template <typename T> cudaError_t seq_row_terms(const SeqArgs &a, int D, cudaStream_t s) {
    return D == 32 ? launch_terms<T, 32>(a, s) : D == 64 ? launch_terms<T, 64>(a, s) : launch_terms<T, 128>(a, s);
}
template cudaError_t seq_row_terms<float>(const SeqArgs &, int, cudaStream_t);
template cudaError_t seq_row_terms<__nv_bfloat16>(const SeqArgs &, int, cudaStream_t);

cudaError_t seq_fwd_f32(const SeqArgs &a, int D, cudaStream_t s) {
    return D == 32 ? launch_fwd<32>(a, s) : D == 64 ? launch_fwd<64>(a, s) : launch_fwd<128>(a, s);
}
cudaError_t seq_bwd_f32(const SeqArgs &a, int D, cudaStream_t s) {
    return D == 32 ? launch_bwd<32>(a, s) : D == 64 ? launch_bwd<64>(a, s) : launch_bwd<128>(a, s);
}

}  // namespace sga
