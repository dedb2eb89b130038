// Packed-sequence attention in fp32, on the FMA pipes, and the row terms of
// the backward pass for both dtypes.
//
// The tensor cores have no fp32 product, and the tolerance of the fp32 layers
// (1e-5) rules out a single tf32 one; operands split into two or three tf32 parts,
// with three products or more for one, have not been tried.  So these kernels are
// bound by the FMA pipes (two products of the forward, three and four of the
// backward's two passes).
// Blocks of TY x 16 threads take TY RA rows of one side (a 64-row tile or a part
// of one) and walk the 64-row tiles of the other through shared memory, the next
// tiles copied while one is in use; each thread holds an RA x 4 piece of the
// scores and an RA x D/16 piece of the result.  Tiles are row-major with rows of
// D + 4 floats: both products read them 16 bytes at a time along a row without
// bank conflicts, so no tile is stored transposed.  RA = 4 reads half as much
// shared memory a product as RA = 2, and 128 threads leave a thread the
// registers to read ahead: 2048 rows, 8 heads of 64, full, forward 272 us (32
// TFLOP/s), backward 789 (938 with 256 threads).
//   forward: S = Q K^T, online softmax (running maximum and sum per row),
//     O = O alpha + P V;
//   dQ pass (a tile of queries): S, dP = dOut V^T, dS = P (dP - Delta),
//     dQ += dS K;
//   dK/dV pass (a tile of keys, over the query heads of its group): S^T =
//     K Q^T, dP^T = V dOut^T, dV += P^T dOut, dK += dS^T Q.
// The scores are computed twice in the backward pass so that every output row
// is owned by one block: no atomics, bitwise reproducible.
// What is not finite in a row for a row that is masked for it is computed again
// over its own interval alone (seq_rows.cuh).  Leaving masked pairs out of every sum instead, with a test a
// pair, took a fifth longer on five sequences of 1 to 512 rows, D = 32.
#include "seq_rows.cuh"
#include "tc.cuh"

namespace sga {
namespace {

constexpr int kT = 64;         // rows of a tile
constexpr int kPP = kT + 4;    // pitch of a score tile

template <int D> constexpr int kPitch = D + 4;
template <int D> constexpr int kTileFloats = kT * (D + 4);
template <int D, int RA, int TY> constexpr int kOwnFloats = TY * RA * (D + 4);   // an owner tile: TY RA rows
template <int RA, int TY> constexpr int kScoreFloats = TY * RA * kPP;
template <int TY> constexpr bool kTwoScores = TY == 8;   // score tiles of the dK/dV pass

// rows [r0, r0 + ROWS) of head h of a [T][heads][D] tensor, asynchronously (rows
// past `rows` as zeros)
template <int D, int TY, int ROWS = kT>
__device__ __forceinline__ void load_tile(float *dst, const void *src, int64_t r0, int64_t rows, int heads, int h) {
    constexpr int C4 = D / 4;
    for (int i = threadIdx.x; i < ROWS * C4; i += 16 * TY) {
        const int r = i / C4, c = i % C4;
        const bool in = r0 + r < rows;
        tc::cp16(tc::smem_u32(dst + r * kPitch<D> + 4 * c),
                 static_cast<const float *>(src) + ((in ? r0 + r : 0) * heads + h) * D + 4 * c, in);
    }
}

// s[a][c] = row (ty + TY a) of A . row (tx + 16 c) of B
template <int D, int RA, int TY>
__device__ __forceinline__ void dot_tiles(float (&s)[RA][4], const float *A, const float *B, int ty, int tx) {
    float2 acc[RA][4];
#pragma unroll
    for (int a = 0; a < RA; ++a)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[a][c] = make_float2(0.f, 0.f);
#pragma unroll 8
    for (int d = 0; d < D; d += 4) {
        float4 x[RA], y[4];
#pragma unroll
        for (int a = 0; a < RA; ++a) x[a] = *reinterpret_cast<const float4 *>(A + (ty + TY * a) * kPitch<D> + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = *reinterpret_cast<const float4 *>(B + (tx + 16 * c) * kPitch<D> + d);
#pragma unroll
        for (int a = 0; a < RA; ++a)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                acc[a][c] = ffma2(make_float2(x[a].x, x[a].y), make_float2(y[c].x, y[c].y), acc[a][c]);
                acc[a][c] = ffma2(make_float2(x[a].z, x[a].w), make_float2(y[c].z, y[c].w), acc[a][c]);
            }
    }
#pragma unroll
    for (int a = 0; a < RA; ++a)
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

// acc[a][x] += sum_j P[ty + TY a][j] B[j][col x] over the 64 rows of B
template <int D, int RA, int TY>
__device__ __forceinline__ void add_product(float (&acc)[RA][kCols<D>], const float *P, const float *B, int ty, int tx) {
    constexpr int NC = kCols<D>;
#pragma unroll 4
    for (int j = 0; j < kT; j += 4) {
        float4 p[RA];
#pragma unroll
        for (int a = 0; a < RA; ++a) p[a] = *reinterpret_cast<const float4 *>(P + (ty + TY * a) * kPP + j);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float v[NC];
            load_cols<D>(v, B + (j + u) * kPitch<D>, tx);
#pragma unroll
            for (int a = 0; a < RA; ++a) axpy2<NC>(acc[a], u == 0 ? p[a].x : u == 1 ? p[a].y : u == 2 ? p[a].z : p[a].w, v);
        }
    }
}

// Stores the rows, scaled, and returns whether any element of this thread's row
// a was not finite, as bit a.
template <int D, int RA, int TY>
__device__ __forceinline__ uint32_t store_rows(float *dst, const float (&acc)[RA][kCols<D>], const float (&f)[RA], int64_t r0,
                                               int64_t rows, int heads, int h, int ty, int tx) {
    uint32_t bad = 0;
#pragma unroll
    for (int a = 0; a < RA; ++a) {
        const int64_t row = r0 + ty + TY * a;
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

// Calls redo(a, half) for every row (ty + TY a of the warp's half) of which a
// thread found an element that is not finite; the warp together, after its stores.
template <int RA, int TY, typename F> __device__ __forceinline__ void each_bad_row(uint32_t bad, F redo) {
    if (!__any_sync(SGA_FULL_MASK, bad != 0)) return;
    __syncwarp();
#pragma unroll
    for (int a = 0; a < RA; ++a) {
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

// What each of a thread's rows sees: queries of a key row, or keys of a
// query row.  Rows past the last see nothing.
template <int RA, int TY>
__device__ __forceinline__ void intervals(const SeqArgs &a, bool keys, int64_t r0, int ty, int64_t (&lo)[RA], int64_t (&hi)[RA]) {
#pragma unroll
    for (int i = 0; i < RA; ++i) {
        const int64_t row = r0 + ty + TY * i;
        lo[i] = hi[i] = 0;
        if (row < a.rows) {
            const int2 se = __ldg(a.range + row);
            lo[i] = keys && a.causal ? row : se.x;
            hi[i] = !keys && a.causal ? row + 1 : se.y;
        }
    }
}
template <int RA>
__device__ __forceinline__ void in_tile(const int64_t (&lo)[RA], const int64_t (&hi)[RA], int64_t t0, int (&l)[RA], int (&h)[RA]) {
#pragma unroll
    for (int i = 0; i < RA; ++i) {
        l[i] = (int)max((int64_t)0, min((int64_t)kT, lo[i] - t0));
        h[i] = (int)max((int64_t)0, min((int64_t)kT, hi[i] - t0));
    }
}

// What the rows of this half of the warp came from (seq_rows.cuh).
__device__ __forceinline__ seq::Span span_of(const SeqArgs &a, const SeqTile &t, int64_t lo, int64_t hi, int half) {
    return seq::Span{__shfl_sync(SGA_FULL_MASK, lo, 16 * half), __shfl_sync(SGA_FULL_MASK, hi, 16 * half), (int64_t)t.t0 * kT,
                     min(a.rows, (int64_t)t.t1 * kT)};
}

// Unit u of a pass: TY RA rows (from `row` of a tile) of one head.
template <int RA, int TY> struct Unit {
    uint32_t tile;
    int head, row;
    __device__ __forceinline__ Unit(uint32_t u, int heads) {
        constexpr uint32_t S = kT / (TY * RA);
        tile = u / (S * heads);
        head = (int)(u / S % heads);
        row = (int)(u % S) * TY * RA;
    }
};
// The unit of a block: longest first, one an SM; where all of them fit two an
// SM, the shortest beside the longest (1024 rows, 8 heads of 64, causal: 68 ->
// 62 us).
__device__ __forceinline__ uint32_t unit_of_block(const SeqArgs &a) {
    const uint32_t b = blockIdx.x, n = gridDim.x, m = (uint32_t)a.num_sms;
    return b >= m && n <= 2 * m ? n - 1 - (b - m) : b;
}

// ---- forward ------------------------------------------------------------------

template <int D, int RA, int TY, int MB> __global__ void __launch_bounds__(16 * TY, MB) seq_fwd_f32_kernel(const SeqArgs a) {
    extern __shared__ __align__(16) float sm[];
    wait_previous();
    float *sQ = sm, *sK = sQ + kOwnFloats<D, RA, TY>, *sV = sK + kTileFloats<D>, *sP = sV + kTileFloats<D>;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const Unit<RA, TY> u(unit_of_block(a), a.H);
    const SeqTile t = a.qtiles[u.tile];
    const int h = u.head, hk = h / (a.H / a.Hkv);
    const int64_t q0 = (int64_t)t.tile * kT + u.row;
    const float scale2 = a.scale * kLog2e;
    load_tile<D, TY, TY * RA>(sQ, a.Q, q0, a.rows, a.H, h);
    load_tile<D, TY>(sK, a.K, (int64_t)t.t0 * kT, a.rows, a.Hkv, hk);
    tc::cp_commit();
    load_tile<D, TY>(sV, a.V, (int64_t)t.t0 * kT, a.rows, a.Hkv, hk);
    tc::cp_commit();
    int64_t lo[RA], hi[RA];
    intervals<RA, TY>(a, false, q0, ty, lo, hi);
    float m[RA], l[RA], acc[RA][kCols<D>];
#pragma unroll
    for (int i = 0; i < RA; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int x = 0; x < kCols<D>; ++x) acc[i][x] = 0.f;
    }
    for (int kt = t.t0; kt < t.t1; ++kt) {
        const int64_t k0 = (int64_t)kt * kT;
        const bool full = kt >= t.f0 && kt < t.f1;
        int kl[RA], kh[RA];
        in_tile(lo, hi, k0, kl, kh);
        tc::cp_wait<1>();   // this K (V may be on its way)
        __syncthreads();
        float s[RA][4];
        dot_tiles<D, RA, TY>(s, sQ, sK, ty, tx);
        __syncthreads();
        if (kt + 1 < t.t1) load_tile<D, TY>(sK, a.K, k0 + kT, a.rows, a.Hkv, hk);   // beside the softmax and P V
        tc::cp_commit();
#pragma unroll
        for (int i = 0; i < RA; ++i) {
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
                sP[(ty + TY * i) * kPP + tx + 16 * c] = p;
                sum += p;
            }
            l[i] = l[i] * al + half_sum(sum);
            m[i] = mn;
#pragma unroll
            for (int x = 0; x < kCols<D>; ++x) acc[i][x] *= al;
        }
        tc::cp_wait<1>();   // this V
        __syncthreads();
        add_product<D, RA, TY>(acc, sP, sV, ty, tx);
        __syncthreads();
        if (kt + 1 < t.t1) load_tile<D, TY>(sV, a.V, k0 + kT, a.rows, a.Hkv, hk);   // beside the next scores
        tc::cp_commit();
    }
    float inv[RA];
#pragma unroll
    for (int i = 0; i < RA; ++i) {
        inv[i] = 1.f / l[i];
        const int64_t row = q0 + ty + TY * i;
        if (tx == 0 && row < a.rows) a.lse_w[row * a.H + h] = (m[i] + log2f(l[i])) * kLn2;
    }
    uint32_t bad = store_rows<D, RA, TY>(static_cast<float *>(a.out_w), acc, inv, q0, a.rows, a.H, h, ty, tx);
#pragma unroll
    for (int i = 0; i < RA; ++i)
        if (l[i] != l[i]) bad &= ~(1u << i);   // NaN whatever the masked rows hold
    each_bad_row<RA, TY>(bad, [&](int i, int half) {
        seq::out_row_alone<float, D>(a, q0 + (ty & ~1) + half + TY * i, h, hk, span_of(a, t, lo[i], hi[i], half));
    });
}

// ---- backward -------------------------------------------------------------------

template <int D, int RA, int TY> __device__ __forceinline__ void dq_pass(const SeqArgs &a, float *sm, uint32_t unit) {
    float *sQ = sm, *sG = sQ + kOwnFloats<D, RA, TY>, *sV = sG + kOwnFloats<D, RA, TY>, *sP = sV + kTileFloats<D>,
          *sK = sP + kScoreFloats<RA, TY>;   // two K tiles
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const Unit<RA, TY> u(unit, a.H);
    const SeqTile t = a.qtiles[u.tile];
    const int h = u.head, hk = h / (a.H / a.Hkv);
    const int64_t q0 = (int64_t)t.tile * kT + u.row;
    const float scale2 = a.scale * kLog2e;
    load_tile<D, TY, TY * RA>(sQ, a.Q, q0, a.rows, a.H, h);
    load_tile<D, TY, TY * RA>(sG, a.dOut, q0, a.rows, a.H, h);
    load_tile<D, TY>(sK, a.K, (int64_t)t.t0 * kT, a.rows, a.Hkv, hk);
    load_tile<D, TY>(sV, a.V, (int64_t)t.t0 * kT, a.rows, a.Hkv, hk);
    tc::cp_commit();
    int64_t lo[RA], hi[RA];
    intervals<RA, TY>(a, false, q0, ty, lo, hi);
    float ls[RA], dl[RA], acc[RA][kCols<D>];
#pragma unroll
    for (int i = 0; i < RA; ++i) {
        const int64_t r = (int64_t)h * a.rows_pad + q0 + ty + TY * i;
        ls[i] = a.ws_nlse[r];
        dl[i] = a.ws_ndelta[r];
#pragma unroll
        for (int x = 0; x < kCols<D>; ++x) acc[i][x] = 0.f;
    }
    for (int kt = t.t0; kt < t.t1; ++kt) {
        const int64_t k0 = (int64_t)kt * kT;
        const bool full = kt >= t.f0 && kt < t.f1;
        float *sKi = sK + (kt - t.t0) % 2 * kTileFloats<D>, *sKn = sK + (kt - t.t0 + 1) % 2 * kTileFloats<D>;
        int kl[RA], kh[RA];
        in_tile(lo, hi, k0, kl, kh);
        tc::cp_wait<0>();
        __syncthreads();   // this K and V; the last dS K is done with the other K and with dS
        if (kt + 1 < t.t1) load_tile<D, TY>(sKn, a.K, k0 + kT, a.rows, a.Hkv, hk);
        float s[RA][4], g[RA][4];
        dot_tiles<D, RA, TY>(g, sG, sV, ty, tx);
        __syncthreads();
        if (kt + 1 < t.t1) load_tile<D, TY>(sV, a.V, k0 + kT, a.rows, a.Hkv, hk);
        tc::cp_commit();
        dot_tiles<D, RA, TY>(s, sQ, sKi, ty, tx);
#pragma unroll
        for (int i = 0; i < RA; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int j = tx + 16 * c;
                const bool on = full || (j >= kl[i] && j < kh[i]);
                sP[(ty + TY * i) * kPP + j] = on ? fast_exp2(fmaf(s[i][c], scale2, ls[i])) * (g[i][c] + dl[i]) : 0.f;
            }
        __syncthreads();
        add_product<D, RA, TY>(acc, sP, sKi, ty, tx);
    }
    float f[RA];
#pragma unroll
    for (int i = 0; i < RA; ++i) f[i] = a.scale;
    const uint32_t bad = store_rows<D, RA, TY>(static_cast<float *>(a.dQ), acc, f, q0, a.rows, a.H, h, ty, tx);
    each_bad_row<RA, TY>(bad, [&](int i, int half) {
        seq::query_row_alone<float, D>(a, q0 + (ty & ~1) + half + TY * i, h, span_of(a, t, lo[i], hi[i], half), ~0u);
    });
}

template <int D, int RA, int TY> __device__ __forceinline__ void dkdv_pass(const SeqArgs &a, float *sm, uint32_t unit) {
    float *sK = sm, *sV = sK + kOwnFloats<D, RA, TY>, *sP = sV + kOwnFloats<D, RA, TY>,
          *sD = sP + (kTwoScores<TY> ? kScoreFloats<RA, TY> : 0),   // dS^T: over P^T where there is no room for both
          *sS = sD + kScoreFloats<RA, TY>;                          // two pairs of Q and dOut tiles
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const Unit<RA, TY> u(unit, a.Hkv);
    const SeqTile t = a.ktiles[u.tile];
    const int hk = u.head, grp = a.H / a.Hkv;
    const int64_t k0 = (int64_t)t.tile * kT + u.row;
    const float scale2 = a.scale * kLog2e;
    const int nt = t.t1 - t.t0, n = nt * grp;   // steps: (head of the group, query tile)
    auto fetch = [&](int i) {
        float *dst = sS + i % 2 * 2 * kTileFloats<D>;
        const int64_t q0 = (int64_t)(t.t0 + i % nt) * kT;
        load_tile<D, TY>(dst, a.Q, q0, a.rows, a.H, hk * grp + i / nt);
        load_tile<D, TY>(dst + kTileFloats<D>, a.dOut, q0, a.rows, a.H, hk * grp + i / nt);
    };
    load_tile<D, TY, TY * RA>(sK, a.K, k0, a.rows, a.Hkv, hk);
    load_tile<D, TY, TY * RA>(sV, a.V, k0, a.rows, a.Hkv, hk);
    fetch(0);
    tc::cp_commit();
    int64_t lo[RA], hi[RA];
    intervals<RA, TY>(a, true, k0, ty, lo, hi);
    float dk[RA][kCols<D>], dv[RA][kCols<D>];
#pragma unroll
    for (int i = 0; i < RA; ++i)
#pragma unroll
        for (int x = 0; x < kCols<D>; ++x) dk[i][x] = dv[i][x] = 0.f;
    for (int step = 0; step < n; ++step) {
        const float *sQ = sS + step % 2 * 2 * kTileFloats<D>, *sG = sQ + kTileFloats<D>;
        const int qt = t.t0 + step % nt;
        const int64_t q0 = (int64_t)qt * kT;
        const bool full = qt >= t.f0 && qt < t.f1;
        int ql[RA], qh[RA];
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
        float s[RA][4], g[RA][4];
        dot_tiles<D, RA, TY>(s, sK, sQ, ty, tx);
        dot_tiles<D, RA, TY>(g, sV, sG, ty, tx);
#pragma unroll
        for (int i = 0; i < RA; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int j = tx + 16 * c;
                const bool on = full || (j >= ql[i] && j < qh[i]);
                const float p = on ? fast_exp2(fmaf(s[i][c], scale2, ls[c])) : 0.f;
                sP[(ty + TY * i) * kPP + j] = p;
                g[i][c] = on ? p * (g[i][c] + dl[c]) : 0.f;
                if (kTwoScores<TY>) sD[(ty + TY * i) * kPP + j] = g[i][c];
            }
        __syncthreads();
        add_product<D, RA, TY>(dv, sP, sG, ty, tx);
        if (!kTwoScores<TY>) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RA; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) sD[(ty + TY * i) * kPP + tx + 16 * c] = g[i][c];
            __syncthreads();
        }
        add_product<D, RA, TY>(dk, sD, sQ, ty, tx);
    }
    float one[RA], f[RA];
#pragma unroll
    for (int i = 0; i < RA; ++i) {
        one[i] = 1.f;
        f[i] = a.scale;
    }
    const uint32_t bad_v = store_rows<D, RA, TY>(static_cast<float *>(a.dV), dv, one, k0, a.rows, a.Hkv, hk, ty, tx);
    const uint32_t bad_k = store_rows<D, RA, TY>(static_cast<float *>(a.dK), dk, f, k0, a.rows, a.Hkv, hk, ty, tx);
    for (int x = 0; x < 2; ++x)
        each_bad_row<RA, TY>(x ? bad_k : bad_v, [&](int i, int half) {
            seq::key_row_alone<float, D>(a, x == 1, k0 + (ty & ~1) + half + TY * i, hk, span_of(a, t, lo[i], hi[i], half), ~0u);
        });
}

// Both passes in one launch, the dK/dV units (the longer ones) first.
template <int D, int RA, int TY, int MB> __global__ void __launch_bounds__(16 * TY, MB) seq_bwd_f32_kernel(const SeqArgs a) {
    extern __shared__ __align__(16) float sm[];
    wait_previous();
    const uint32_t kv = (uint32_t)a.n_tiles * a.Hkv * (kT / (TY * RA));
    if (blockIdx.x < kv) dkdv_pass<D, RA, TY>(a, sm, blockIdx.x);
    else dq_pass<D, RA, TY>(a, sm, blockIdx.x - kv);
}

// Row terms: D / EL lanes of 16 bytes a (row, head), four of them in flight.
// Rows behind the last sequence (to the end of its tile) get -lse = -inf, so
// that their weights are zero, and Delta = 0.
constexpr int kTerms = 4;
template <typename T, int D> __global__ void __launch_bounds__(256) seq_row_terms_kernel(const SeqArgs a) {
    let_next_start();
    wait_previous();
    constexpr int EL = Elt<T>::EL, L = D / EL, G = 256 / L;   // G items of a block at a time
    const int sub = threadIdx.x % L;
    const int64_t live = a.rows * a.H, n = a.rows_pad * a.H, g0 = (int64_t)blockIdx.x * (G * kTerms) + threadIdx.x / L;
    uint4 x[kTerms], y[kTerms];
    float lse[kTerms];
#pragma unroll
    for (int k = 0; k < kTerms; ++k) {
        const int64_t g = g0 + k * G;
        x[k] = y[k] = make_uint4(0, 0, 0, 0);
        lse[k] = INFINITY;
        if (g < live) {   // (an item's elements follow the one's before)
            x[k] = ldg16(static_cast<const T *>(a.out) + g * D + sub * EL);
            y[k] = ldg16(static_cast<const T *>(a.dOut) + g * D + sub * EL);
            if (sub == 0) lse[k] = __ldg(a.lse + g) * kLog2e;
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
            // (a 64-bit division takes longer than the rest of an item)
            const int64_t row = n <= UINT32_MAX ? (int64_t)((uint32_t)g / (uint32_t)a.H) : g / a.H;
            const int64_t at = (g - row * a.H) * a.rows_pad + row;
            a.ws_nlse[at] = -lse[k];
            a.ws_ndelta[at] = g < live ? -d : 0.f;
        }
    }
}

template <int D, int RA, int TY, int MB> cudaError_t launch_fwd(const SeqArgs &a, cudaStream_t s) {
    constexpr size_t smem = sizeof(float) * (kOwnFloats<D, RA, TY> + 2 * kTileFloats<D> + kScoreFloats<RA, TY>);
    if (cudaError_t e = allow_smem<seq_fwd_f32_kernel<D, RA, TY, MB>>(smem); e != cudaSuccess) return e;
    note_launch(SGA_KERN_SEQ_FWD, s, false);
    const cudaError_t e = launch_early(seq_fwd_f32_kernel<D, RA, TY, MB>, dim3((unsigned)((int64_t)a.n_tiles * a.H * (kT / (TY * RA)))), dim3(16 * TY), smem, s, a);
    note_launch(SGA_KERN_SEQ_FWD, s, true);
    return e;
}

template <int D, int RA, int TY, int MB> cudaError_t launch_bwd(const SeqArgs &a, cudaStream_t s) {
    constexpr size_t kv = sizeof(float) * (2 * kOwnFloats<D, RA, TY> + 4 * kTileFloats<D> + (kTwoScores<TY> ? 2 : 1) * kScoreFloats<RA, TY>);
    constexpr size_t q = sizeof(float) * (2 * kOwnFloats<D, RA, TY> + 3 * kTileFloats<D> + kScoreFloats<RA, TY>);
    constexpr size_t smem = kv > q ? kv : q;
    static_assert(smem <= 227 * 1024, "shared memory");
    cudaError_t e = allow_smem<seq_bwd_f32_kernel<D, RA, TY, MB>>(smem);
    if (e == cudaSuccess) e = seq_row_terms<float>(a, D, s);
    if (e != cudaSuccess) return e;
    note_launch(SGA_KERN_SEQ_BWD, s, false);
    e = launch_early(seq_bwd_f32_kernel<D, RA, TY, MB>, dim3((unsigned)((int64_t)a.n_tiles * (a.Hkv + a.H) * (kT / (TY * RA)))),
                      dim3(16 * TY), smem, s, a);
    note_launch(SGA_KERN_SEQ_BWD, s, true);
    return e;
}

template <typename T, int D> cudaError_t launch_terms(const SeqArgs &a, cudaStream_t s) {
    constexpr int per = kTerms * 256 / (D / Elt<T>::EL);   // items of a block
    note_launch(SGA_KERN_SEQ_BWD_ROWS, s, false);
    const cudaError_t e = launch_early(seq_row_terms_kernel<T, D>, dim3((unsigned)((a.rows_pad * a.H + per - 1) / per)), dim3(256), 0, s, a);
    note_launch(SGA_KERN_SEQ_BWD_ROWS, s, true);
    return e;
}

}  // namespace

template <typename T> cudaError_t seq_row_terms(const SeqArgs &a, int D, cudaStream_t s) {
    return D == 32 ? launch_terms<T, 32>(a, s) : D == 64 ? launch_terms<T, 64>(a, s) : launch_terms<T, 128>(a, s);
}
template cudaError_t seq_row_terms<float>(const SeqArgs &, int, cudaStream_t);
template cudaError_t seq_row_terms<__nv_bfloat16>(const SeqArgs &, int, cudaStream_t);

// Owner tiles of 32 rows (4 x 8); of 16 (2 x 8) where 32 would leave SMs without
// a block (us a call, launches apart): 512 rows, 4 heads (64 units of 32),
// forward D = 32, 64, 128: 16 rows 18.7, 24.8, 37.1, 32 rows 24.8, 33.0, 47.4;
// 1024 rows, 8 heads (256), D = 64: 117 : 84.  Backward, 256 rows, 4 heads (64):
// 16.6, 22.8, 33.2 : 18.9, 27.1, 41.3.  In the forward four blocks an SM fit in
// 128 registers a thread with a few spills, against three: 2048 rows, 8 heads
// (512 units), D = 32 174 : 213, D = 64 275 : 309; fewer units do not need them
// (256, D = 64, causal 64 : 62).  In the backward D = 32 is faster with two blocks
// an SM while they are enough (1024 rows, 4 heads 81 : 102, 8 heads 140 : 124), and
// D = 128, whose tiles leave room for one block an SM, with 64 rows and 256
// threads from there on (1024 rows, 8 heads 400 : 484; 512 rows, 8 heads, causal
// 117 : 74).
cudaError_t seq_fwd_f32(const SeqArgs &a, int D, cudaStream_t s) {
    const int64_t units = 2 * (int64_t)a.n_tiles * a.H;
    if ((D == 128 ? 2 : 1) * units <= a.num_sms)
        return D == 32 ? launch_fwd<32, 2, 8, 3>(a, s) : D == 64 ? launch_fwd<64, 2, 8, 3>(a, s) : launch_fwd<128, 2, 8, 2>(a, s);
    const bool many = units > 3 * (int64_t)a.num_sms;
    if (D == 32) return many ? launch_fwd<32, 4, 8, 4>(a, s) : launch_fwd<32, 4, 8, 3>(a, s);
    if (D == 64) return many ? launch_fwd<64, 4, 8, 4>(a, s) : launch_fwd<64, 4, 8, 3>(a, s);
    return launch_fwd<128, 4, 8, 2>(a, s);
}
cudaError_t seq_bwd_f32(const SeqArgs &a, int D, cudaStream_t s) {
    const int64_t units = 2 * (int64_t)a.n_tiles * (a.H + a.Hkv);
    if ((D == 128 ? 2 : 1) * units <= a.num_sms)
        return D == 32 ? launch_bwd<32, 2, 8, 3>(a, s) : D == 64 ? launch_bwd<64, 2, 8, 2>(a, s) : launch_bwd<128, 2, 8, 1>(a, s);
    const bool many = units > 2 * (int64_t)a.num_sms;
    if (D == 32) return many ? launch_bwd<32, 4, 8, 3>(a, s) : launch_bwd<32, 4, 8, 2>(a, s);
    if (D == 64) return launch_bwd<64, 4, 8, 2>(a, s);
    return many ? launch_bwd<128, 4, 16, 1>(a, s) : launch_bwd<128, 4, 8, 1>(a, s);
}

}  // namespace sga
