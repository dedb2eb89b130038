// Layer norm over the rows of X [N, C], forward and backward.
//   mean = sum x / C,  var = sum (x - mean)^2 / C,  rstd = 1 / sqrt(var + eps)
//   xhat = (x - mean) rstd,  y = xhat w + b
//   g = dy w,  dx = rstd (g - sum(g) / C - xhat sum(g xhat) / C)
//   dw = sum over rows dy xhat,  db = sum over rows dy
//
// Bound by DRAM: the forward reads x and writes y, the backward reads x and dy
// and writes dx, each once.  A row is held in the registers of a group of
// threads (4 to 32 lanes, or a whole block), so the variance is taken about
// the mean without a second read.  Groups walk the rows with a fixed stride and
// keep the columns' weights, and in the backward their sums of dw and db, in
// registers; a block's groups are then added in a fixed order through shared
// memory, and a second kernel adds the blocks in order: no atomics, bitwise
// reproducible.  Statistics and sums are fp32.
#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"
#include "tc.cuh"

namespace cg = cooperative_groups;

namespace sga {

void set_cuda_error(cudaError_t e);   // (api.cu)

namespace {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

sga_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return SGA_OK;
    set_cuda_error(e);
    return SGA_ECUDA;
}

struct NormArgs {
    const void *X, *w, *b, *dY;
    void *Y, *dX;
    float *mean, *rstd;
    const float *mean_in, *rstd_in;
    float *part;             // [blocks][2][C] sums of dw, db
    int64_t N;
    int C;
    float eps;
};

// EL consecutive elements as they lie in memory: 16-byte loads where EL covers
// 16 bytes (or several), one load of EL elements otherwise.
template <typename T, int EL> struct Raw {
    static constexpr int B = EL * (int)sizeof(T);
    static_assert(B % 16 == 0 || B == 8 || B == 4 || B == 2, "group");
    uint32_t u[B >= 4 ? B / 4 : 1];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (B >= 4 ? B / 4 : 1); ++i) u[i] = 0;
    }
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (B % 16 == 0) {
#pragma unroll
            for (int i = 0; i < B / 16; ++i) {
                const uint4 q = reinterpret_cast<const uint4 *>(p)[i];
                u[4 * i] = q.x;
                u[4 * i + 1] = q.y;
                u[4 * i + 2] = q.z;
                u[4 * i + 3] = q.w;
            }
        } else if constexpr (B == 8) {
            const uint2 q = *reinterpret_cast<const uint2 *>(p);
            u[0] = q.x;
            u[1] = q.y;
        } else if constexpr (B == 4) {
            u[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            u[0] = *reinterpret_cast<const uint16_t *>(p);
        }
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(u[i]);
        else return __uint_as_float((i & 1) ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16);   // (bf16: the top half of fp32)
    }
};

template <typename T, int EL> __device__ __forceinline__ void store_el(T *p, const float (&x)[EL]) {
    constexpr int CH = Elt<T>::EL;
    if constexpr (EL % CH == 0) {
#pragma unroll
        for (int c = 0; c < EL; c += CH) *reinterpret_cast<uint4 *>(p + c) = pack<T>(x + c);
    } else if constexpr (EL == 2 && sizeof(T) == 2) {
        *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(x[0], x[1]);
    } else {
        static_assert(EL == 1, "group");
        *p = from_f32<T>(x[0]);
    }
}

// Sum over the TPR threads of a row.  TPR > 32: the whole block is one row;
// `red` holds a slot per warp and is free to be reused after the next call.
template <int TPR, int K> __device__ __forceinline__ void row_sum(float (&v)[K], float (*red)[32]) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = group_sum<(TPR < 32 ? TPR : 32)>(v[k]);
    if constexpr (TPR > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) red[k][threadIdx.x >> 5] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = 0.f;
#pragma unroll
            for (int i = 0; i < TPR / 32; ++i) v[k] += red[k][i];
        }
    }
}

template <typename TX, typename TW, int EL, int TPR, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_fwd_kernel(const NormArgs a) {
    __shared__ float red[1][32];
    let_next_start();
    wait_previous();
    constexpr int GPB = THREADS / TPR;
    const int sub = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int nvec = a.C / EL;
    const TX *X = static_cast<const TX *>(a.X);
    const TW *w = static_cast<const TW *>(a.w), *b = static_cast<const TW *>(a.b);
    const float inv = 1.f / (float)a.C;
    Raw<TW, EL> wr[NV], br[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = v * TPR + sub;
        wr[v].zero();
        br[v].zero();
        if (c < nvec && w) wr[v].load(w + c * EL);
        if (c < nvec && b) br[v].load(b + c * EL);
    }
    const int64_t step = (int64_t)gridDim.x * GPB;
    Raw<TX, EL> x[NV];   // a round ahead: the next row's loads are in flight while a row is summed
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = v * TPR + sub;
            x[v].zero();
            if (row < a.N && c < nvec) x[v].load(X + row * a.C + c * EL);
        }
    };
    fetch((int64_t)blockIdx.x * GPB + grp);
    // every group of a warp runs the same number of rounds: the sums are warp-wide calls
    for (int64_t r0 = (int64_t)blockIdx.x * GPB; r0 < a.N; r0 += step) {
        const int64_t row = r0 + grp;
        float f[NV][EL], s[1] = {0.f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < EL; ++i) {
                f[v][i] = x[v].at(i);
                s[0] += f[v][i];
            }
        fetch(row + step);
        row_sum<TPR, 1>(s, red);
        const float mean = s[0] * inv;
        s[0] = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < EL; ++i) {
                f[v][i] -= mean;
                if (v * TPR + sub < nvec) s[0] = fmaf(f[v][i], f[v][i], s[0]);
            }
        row_sum<TPR, 1>(s, red);
        const float rstd = rsqrtf(s[0] * inv + a.eps);
        if (row >= a.N) continue;
        if (sub == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        TX *Y = static_cast<TX *>(a.Y) + row * a.C;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = v * TPR + sub;
            if (c >= nvec) continue;
            float y[EL];
#pragma unroll
            for (int i = 0; i < EL; ++i) y[i] = w ? fmaf(f[v][i] * rstd, wr[v].at(i), br[v].at(i)) : f[v][i] * rstd;
            store_el<TX, EL>(Y + c * EL, y);
        }
    }
}

// The sums of a block's groups, added one after the other in shared memory
// (acc_sm: [2][C]), to the block's row of partials.
template <int EL, int TPR, int NV, int THREADS>
__device__ __forceinline__ void block_sums(const NormArgs &a, float *acc_sm, const float (&dw)[NV][EL], const float (&db)[NV][EL]) {
    const int sub = threadIdx.x % TPR, grp = threadIdx.x / TPR, nvec = a.C / EL;
    for (int q = 0; q < THREADS / TPR; ++q) {
        __syncthreads();
        if (grp == q)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = v * TPR + sub;
                if (c >= nvec) continue;
#pragma unroll
                for (int i = 0; i < EL; ++i) {
                    float *p = acc_sm + c * EL + i, *z = p + a.C;
                    *p = (q ? *p : 0.f) + dw[v][i];
                    *z = (q ? *z : 0.f) + db[v][i];
                }
            }
    }
    __syncthreads();
    float *out = a.part + (int64_t)blockIdx.x * 2 * a.C;
    for (int i = threadIdx.x; i < 2 * a.C; i += THREADS) out[i] = acc_sm[i];
}

template <typename TX, typename TW, int EL, int TPR, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_bwd_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    extern __shared__ float acc_sm[];   // [2][C] sums of the block's groups
    let_next_start();
    wait_previous();
    constexpr int GPB = THREADS / TPR;
    const int sub = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int nvec = a.C / EL;
    const TX *X = static_cast<const TX *>(a.X), *dY = static_cast<const TX *>(a.dY);
    const TW *w = static_cast<const TW *>(a.w);
    const float inv = 1.f / (float)a.C;
    Raw<TW, EL> wr[NV];
    float dw[NV][EL], db[NV][EL];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = v * TPR + sub;
        wr[v].zero();
#pragma unroll
        for (int i = 0; i < EL; ++i) dw[v][i] = db[v][i] = 0.f;
        if (c < nvec && w) wr[v].load(w + c * EL);
    }
    const int64_t step = (int64_t)gridDim.x * GPB;
    Raw<TX, EL> xr[NV], gr[NV];   // a round ahead, as in the forward
    float mean_r = 0.f, rstd_r = 0.f;
    auto fetch = [&](int64_t row) {
        const bool in = row < a.N;
        mean_r = in ? a.mean_in[row] : 0.f;
        rstd_r = in ? a.rstd_in[row] : 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = v * TPR + sub;
            xr[v].zero();
            gr[v].zero();
            if (in && c < nvec) {
                xr[v].load(X + row * a.C + c * EL);
                gr[v].load(dY + row * a.C + c * EL);
            }
        }
    };
    fetch((int64_t)blockIdx.x * GPB + grp);
    for (int64_t r0 = (int64_t)blockIdx.x * GPB; r0 < a.N; r0 += step) {
        const int64_t row = r0 + grp;
        const float mean = mean_r, rstd = rstd_r;
        float x[NV][EL], g[NV][EL], s[2] = {0.f, 0.f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const bool on = row < a.N && v * TPR + sub < nvec;
#pragma unroll
            for (int i = 0; i < EL; ++i) {
                x[v][i] = (xr[v].at(i) - mean) * rstd;   // xhat
                g[v][i] = gr[v].at(i);
                if (!on) continue;
                db[v][i] += g[v][i];
                dw[v][i] = fmaf(g[v][i], x[v][i], dw[v][i]);
                if (w) g[v][i] *= wr[v].at(i);
                s[0] += g[v][i];
                s[1] = fmaf(g[v][i], x[v][i], s[1]);
            }
        }
        fetch(row + step);
        row_sum<TPR, 2>(s, red);
        if (row >= a.N) continue;
        const float c1 = s[0] * inv, c2 = s[1] * inv;
        TX *dX = static_cast<TX *>(a.dX) + row * a.C;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = v * TPR + sub;
            if (c >= nvec) continue;
            float o[EL];
#pragma unroll
            for (int i = 0; i < EL; ++i) o[i] = rstd * (g[v][i] - c1 - x[v][i] * c2);
            store_el<TX, EL>(dX + c * EL, o);
        }
    }
    if (!a.part) return;
    block_sums<EL, TPR, NV, THREADS>(a, acc_sm, dw, db);
}

// The backward pass for rows of whole 16-byte vectors that a warp can hold: the
// same sums, but each thread copies its vectors of the next STAGES - 1 rows into
// its own slots of shared memory (cp.async; nothing is shared, so there is no
// barrier).  The loads in flight are then not bound by registers: 169343 x 512
// bf16 takes 87 us, with a row ahead in registers 97 (128 threads, 16 warps an SM).
constexpr int kRingThreads = 128, kRingStages = 6;

template <typename TX, typename TW, int TPR, int NV>
__global__ void __launch_bounds__(kRingThreads, 4) norm_bwd_ring_kernel(const NormArgs a) {
    constexpr int EL = Elt<TX>::EL, GPB = kRingThreads / TPR;
    let_next_start();
    wait_previous();
    extern __shared__ __align__(16) unsigned char ring_sm[];   // [stage][vector][x, dy][thread] 16 bytes; then [2][C] sums
    const int sub = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int nvec = a.C / EL;
    const TX *X = static_cast<const TX *>(a.X), *dY = static_cast<const TX *>(a.dY);
    const TW *w = static_cast<const TW *>(a.w);
    const float inv = 1.f / (float)a.C;
    Raw<TW, EL> wr[NV];
    float dw[NV][EL], db[NV][EL];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = v * TPR + sub;
        wr[v].zero();
#pragma unroll
        for (int i = 0; i < EL; ++i) dw[v][i] = db[v][i] = 0.f;
        if (c < nvec && w) wr[v].load(w + c * EL);
    }
    const int64_t step = (int64_t)gridDim.x * GPB, first = (int64_t)blockIdx.x * GPB + grp;
    uint4 *slots = reinterpret_cast<uint4 *>(ring_sm) + threadIdx.x;
    const uint32_t slot0 = tc::smem_u32(slots);
    auto slot = [](int s, int v, int y) { return ((s * NV + v) * 2 + y) * kRingThreads; };
    auto fetch = [&](int64_t row, int s) {
        const bool in = row < a.N;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = v * TPR + sub;
            const bool ok = in && c < nvec;
            const int64_t at = ok ? row * a.C + c * EL : 0;
            tc::cp16(slot0 + slot(s, v, 0) * 16, X + at, ok);
            tc::cp16(slot0 + slot(s, v, 1) * 16, dY + at, ok);
        }
        tc::cp_commit();
    };
#pragma unroll
    for (int s = 0; s < kRingStages - 1; ++s) fetch(first + s * step, s);
    float mean_r = first < a.N ? a.mean_in[first] : 0.f, rstd_r = first < a.N ? a.rstd_in[first] : 0.f;
    int s = 0;
    // every group of a warp runs the same number of rounds: the sums are warp-wide calls
    for (int64_t r0 = (int64_t)blockIdx.x * GPB; r0 < a.N; r0 += step) {
        const int64_t row = r0 + grp, next = row + step;
        const float mean = mean_r, rstd = rstd_r;
        mean_r = next < a.N ? a.mean_in[next] : 0.f;
        rstd_r = next < a.N ? a.rstd_in[next] : 0.f;
        tc::cp_wait<kRingStages - 2>();
        float x[NV][EL], g[NV][EL], sum[2] = {0.f, 0.f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            unpack<TX>(slots[slot(s, v, 0)], x[v]);
            unpack<TX>(slots[slot(s, v, 1)], g[v]);
            const bool on = row < a.N && v * TPR + sub < nvec;
#pragma unroll
            for (int i = 0; i < EL; ++i) {
                x[v][i] = (x[v][i] - mean) * rstd;   // xhat
                if (!on) continue;
                db[v][i] += g[v][i];
                dw[v][i] = fmaf(g[v][i], x[v][i], dw[v][i]);
                if (w) g[v][i] *= wr[v].at(i);
                sum[0] += g[v][i];
                sum[1] = fmaf(g[v][i], x[v][i], sum[1]);
            }
        }
        // the slot read a round ago
        fetch(row + (kRingStages - 1) * step, s == 0 ? kRingStages - 1 : s - 1);
        s = s + 1 == kRingStages ? 0 : s + 1;
        row_sum<TPR, 2>(sum, nullptr);
        if (row >= a.N) continue;
        const float c1 = sum[0] * inv, c2 = sum[1] * inv;
        TX *dX = static_cast<TX *>(a.dX) + row * a.C;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = v * TPR + sub;
            if (c >= nvec) continue;
            float o[EL];
#pragma unroll
            for (int i = 0; i < EL; ++i) o[i] = rstd * (g[v][i] - c1 - x[v][i] * c2);
            store_el<TX, EL>(dX + c * EL, o);
        }
    }
    tc::cp_wait<0>();
    if (!a.part) return;
    float *acc_sm = reinterpret_cast<float *>(ring_sm);   // (all slots are read)
    block_sums<EL, TPR, NV, kRingThreads>(a, acc_sm, dw, db);
}

// Rows too wide for registers: CL blocks of TH threads a row (more than one: a
// cluster), x read again (from L2) in each step, EL elements a load and U loads of
// a thread in flight.  256 threads to 16384 columns, 1024 to 65536, then clusters
// of eight: a row that is one block's work is read at what one SM can.  1 row of
// 2^20 fp32: 32 us forward, 39 backward (one block of 256 threads, a load at a
// time: 896 and 1430).
template <int CL> struct RowCluster {
    float (*slots)[2][8];   // [which sum][value][rank], in every block's shared memory
    __device__ __forceinline__ static int rank() { return CL > 1 ? (int)cg::this_cluster().block_rank() : 0; }
    // every block of the row runs, so that its shared memory may be written
    __device__ __forceinline__ static void start() {
        if constexpr (CL > 1) cg::this_cluster().sync();
    }
    // Adds the blocks' sums, in the order of their ranks.  `which` alternates: a slot
    // is written again only after the barrier of the sum in between, to which a
    // block comes after it has read the slot.
    template <int K> __device__ __forceinline__ void add(float (&v)[K], int which) const {
        if constexpr (CL > 1) {
            cg::cluster_group row = cg::this_cluster();
            if (threadIdx.x < CL)
#pragma unroll
                for (int k = 0; k < K; ++k) *row.map_shared_rank(&slots[which][k][rank()], threadIdx.x) = v[k];
            row.sync();
#pragma unroll
            for (int k = 0; k < K; ++k) {
                v[k] = 0.f;
#pragma unroll
                for (int i = 0; i < CL; ++i) v[k] += slots[which][k][i];
            }
        }
    }
};

template <typename TX, typename TW, int EL, int TH, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(TH) norm_fwd_wide_kernel(const NormArgs a) {
    constexpr int U = EL == 8 ? 2 : EL == 4 ? 4 : 8, STEP = TH * EL;
    __shared__ float red[1][32], slots[2][2][8];
    let_next_start();
    wait_previous();
    const TX *X = static_cast<const TX *>(a.X);
    const TW *w = static_cast<const TW *>(a.w), *b = static_cast<const TW *>(a.b);
    const float inv = 1.f / (float)a.C;
    const RowCluster<CL> row_blocks{slots};
    const int share = (a.C / EL + CL - 1) / CL * EL, first = row_blocks.rank() * share, last = min(a.C, first + share);   // the block's columns
    row_blocks.start();
    for (int64_t row = blockIdx.x / CL; row < a.N; row += gridDim.x / CL) {
        const TX *x = X + row * a.C;
        TX *y = static_cast<TX *>(a.Y) + row * a.C;
        auto each = [&](auto f) {   // f(elements, column) over the thread's columns
            for (int c0 = first + threadIdx.x * EL; c0 < last; c0 += U * STEP) {
                Raw<TX, EL> r[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + u * STEP < last) r[u].load(x + c0 + u * STEP);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + u * STEP < last) f(r[u], c0 + u * STEP);
            }
        };
        float s[1] = {0.f};
        each([&](const Raw<TX, EL> &r, int) {
#pragma unroll
            for (int i = 0; i < EL; ++i) s[0] += r.at(i);
        });
        row_sum<TH, 1>(s, red);
        row_blocks.add(s, 0);
        const float mean = s[0] * inv;
        s[0] = 0.f;
        each([&](const Raw<TX, EL> &r, int) {
#pragma unroll
            for (int i = 0; i < EL; ++i) {
                const float d = r.at(i) - mean;
                s[0] = fmaf(d, d, s[0]);
            }
        });
        row_sum<TH, 1>(s, red);
        row_blocks.add(s, 1);
        const float rstd = rsqrtf(s[0] * inv + a.eps);
        each([&](const Raw<TX, EL> &r, int c) {
            Raw<TW, EL> wr, br;
            br.zero();
            if (w) wr.load(w + c);
            if (b) br.load(b + c);
            float o[EL];
#pragma unroll
            for (int i = 0; i < EL; ++i) o[i] = fmaf((r.at(i) - mean) * rstd, w ? wr.at(i) : 1.f, br.at(i));
            store_el<TX, EL>(y + c, o);
        });
        if (threadIdx.x == 0 && first == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
    }
}

template <typename TX, typename TW, int EL, int TH, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(TH) norm_bwd_wide_kernel(const NormArgs a) {
    constexpr int U = EL == 8 ? 1 : EL == 4 ? 2 : 4, STEP = TH * EL;
    __shared__ float red[2][32], slots[2][2][8];
    let_next_start();
    wait_previous();
    const TW *w = static_cast<const TW *>(a.w);
    const float inv = 1.f / (float)a.C;
    const RowCluster<CL> row_blocks{slots};
    const int share = (a.C / EL + CL - 1) / CL * EL, first = row_blocks.rank() * share, last = min(a.C, first + share);   // the block's columns
    row_blocks.start();
    int which = 0;
    for (int64_t row = blockIdx.x / CL; row < a.N; row += gridDim.x / CL) {
        const TX *x = static_cast<const TX *>(a.X) + row * a.C, *dy = static_cast<const TX *>(a.dY) + row * a.C;
        TX *dx = static_cast<TX *>(a.dX) + row * a.C;
        const float mean = a.mean_in[row], rstd = a.rstd_in[row];
        auto each = [&](auto f) {   // f(xhat, g, column) over the thread's columns
            for (int c0 = first + threadIdx.x * EL; c0 < last; c0 += U * STEP) {
                Raw<TX, EL> xr[U], gr[U];
                Raw<TW, EL> wr[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + u * STEP < last) {
                        xr[u].load(x + c0 + u * STEP);
                        gr[u].load(dy + c0 + u * STEP);
                        if (w) wr[u].load(w + c0 + u * STEP);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + u * STEP < last) {
                        float h[EL], g[EL];
#pragma unroll
                        for (int i = 0; i < EL; ++i) {
                            h[i] = (xr[u].at(i) - mean) * rstd;
                            g[i] = gr[u].at(i) * (w ? wr[u].at(i) : 1.f);
                        }
                        f(h, g, c0 + u * STEP);
                    }
            }
        };
        float s[2] = {0.f, 0.f};
        each([&](const float (&h)[EL], const float (&g)[EL], int) {
#pragma unroll
            for (int i = 0; i < EL; ++i) {
                s[0] += g[i];
                s[1] = fmaf(g[i], h[i], s[1]);
            }
        });
        row_sum<TH, 2>(s, red);
        row_blocks.add(s, which);
        which ^= 1;
        const float c1 = s[0] * inv, c2 = s[1] * inv;
        each([&](const float (&h)[EL], const float (&g)[EL], int c) {
            float o[EL];
#pragma unroll
            for (int i = 0; i < EL; ++i) o[i] = rstd * (g[i] - c1 - h[i] * c2);
            store_el<TX, EL>(dx + c, o);
        });
    }
}

// Column sums of wide rows: a thread per column over the rows of a slab.
template <typename TX> __global__ void __launch_bounds__(256) norm_cols_wide_kernel(const NormArgs a, int64_t slab) {
    let_next_start();
    wait_previous();
    const int c = blockIdx.x * 256 + threadIdx.x;
    const int64_t r0 = (int64_t)blockIdx.y * slab, r1 = min(a.N, r0 + slab);
    if (c >= a.C) return;
    float dw = 0.f, db = 0.f;
    for (int64_t r = r0; r < r1; ++r) {
        const float dy = to_f32<TX>(static_cast<const TX *>(a.dY)[r * a.C + c]);
        const float xh = (to_f32<TX>(static_cast<const TX *>(a.X)[r * a.C + c]) - a.mean_in[r]) * a.rstd_in[r];
        dw = fmaf(dy, xh, dw);
        db += dy;
    }
    float *out = a.part + (int64_t)blockIdx.y * 2 * a.C;
    out[c] = dw;
    out[a.C + c] = db;
}

// dw, db from the blocks' sums: 32 columns a block; its 32 warps take every
// 32nd partial, four in flight, and are added in order.
template <typename TW> __global__ void __launch_bounds__(1024) norm_reduce_kernel(const float *__restrict__ part, int blocks,
                                                                                  int C, TW *dw, TW *db) {
    __shared__ float sm[32][33];
    wait_previous();
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane, n = 2 * (int64_t)C;   // column of [dw | db]
    float s = 0.f;
    if (i < n)
        for (int b = wp; b < blocks; b += 128) {
            float v[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) v[z] = b + 32 * z < blocks ? part[(b + 32 * z) * n + i] : 0.f;
            s += (v[0] + v[1]) + (v[2] + v[3]);
        }
    sm[wp][lane] = s;
    __syncthreads();
    s = group_sum<32>(sm[lane][wp]);   // warp wp: column wp of the block
    const int64_t c = (int64_t)blockIdx.x * 32 + wp;
    if (lane == 0 && c < n) {
        if (c < C) dw[c] = from_f32<TW>(s);
        else if (db) db[c - C] = from_f32<TW>(s);
    }
}

// The same from few blocks: a thread per column.
template <typename TW> __global__ void __launch_bounds__(256) norm_reduce_few_kernel(const float *__restrict__ part, int blocks,
                                                                                     int C, TW *dw, TW *db) {
    wait_previous();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = 2 * (int64_t)C;
    if (i >= n) return;
    float s = 0.f;
    for (int b = 0; b < blocks; ++b) s += part[b * n + i];
    if (i < C) dw[i] = from_f32<TW>(s);
    else if (db) db[i - C] = from_f32<TW>(s);
}

// Blocks of the backward pass, each with a row of sums: four an SM.
constexpr int kNormBlocksPerSm = 4;
int64_t bwd_blocks(int sms) { return (int64_t)sms * kNormBlocksPerSm; }

template <typename TX, typename TW, int EL, int TPR, int NV>
cudaError_t launch_fwd(const NormArgs &a, cudaStream_t s) {
    constexpr int TH = TPR > 128 ? TPR : 128;
    constexpr int GPB = TH / TPR;
    const int64_t need = (a.N + GPB - 1) / GPB;
    const unsigned grid = (unsigned)std::min<int64_t>(need, (int64_t)device_sms() * 32);
    note_launch(SGA_KERN_NORM_FWD, s, false);
    const cudaError_t e = launch_early(norm_fwd_kernel<TX, TW, EL, TPR, NV, TH>, dim3(grid), dim3(TH), 0, s, a);
    note_launch(SGA_KERN_NORM_FWD, s, true);
    return e;
}

template <typename TX, typename TW, int EL, int TPR, int NV>
cudaError_t launch_bwd(const NormArgs &a, int &blocks, cudaStream_t s) {
    constexpr int TH = TPR > 128 ? TPR : 128;
    constexpr int GPB = TH / TPR;
    const size_t smem = a.part ? sizeof(float) * 2 * a.C : 0;
    if (cudaError_t e = allow_smem<norm_bwd_kernel<TX, TW, EL, TPR, NV, TH>>(smem); e != cudaSuccess) return e;
    // as many blocks as are resident at once: a few more would run alone (4099 x
    // 301 fp32: 8.4 us with three an SM, 12.6 with four, of which three fit)
    static std::atomic<int> per_sm[kMaxDevices];
    cudaError_t asked = cudaSuccess;
    const int fit = per_device(per_sm, [&] {
        int n = 0;
        asked = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, norm_bwd_kernel<TX, TW, EL, TPR, NV, TH>, TH,
                                                              sizeof(float) * 2 * 4096);
        return asked == cudaSuccess ? std::max(1, std::min(n, kNormBlocksPerSm)) : 0;
    });
    if (asked != cudaSuccess) return asked;
    blocks = (int)std::min<int64_t>((a.N + GPB - 1) / GPB, (int64_t)device_sms() * fit);
    note_launch(SGA_KERN_NORM_BWD, s, false);
    const cudaError_t e = launch_early(norm_bwd_kernel<TX, TW, EL, TPR, NV, TH>, dim3((unsigned)blocks), dim3(TH), smem, s, a);
    note_launch(SGA_KERN_NORM_BWD, s, true);
    return e;
}

template <typename TX, typename TW, int TPR, int NV> cudaError_t launch_bwd_ring(const NormArgs &a, int &blocks, cudaStream_t s) {
    constexpr int GPB = kRingThreads / TPR;
    blocks = (int)std::min<int64_t>((a.N + GPB - 1) / GPB, bwd_blocks(device_sms()));
    const size_t ring = (size_t)kRingStages * NV * 2 * 16 * kRingThreads, sums = sizeof(float) * 2 * a.C;
    const size_t smem = std::max(ring, sums);
    if (cudaError_t e = allow_smem<norm_bwd_ring_kernel<TX, TW, TPR, NV>>(smem); e != cudaSuccess) return e;
    note_launch(SGA_KERN_NORM_BWD, s, false);
    const cudaError_t e = launch_early(norm_bwd_ring_kernel<TX, TW, TPR, NV>, dim3((unsigned)blocks), dim3(kRingThreads), smem, s, a);
    note_launch(SGA_KERN_NORM_BWD, s, true);
    return e;
}

// The wide kernels by width: 256 threads a row, 1024, eight blocks of 1024.
cudaError_t launch_wide(const NormArgs &a, cudaStream_t s, void (*narrow)(NormArgs), void (*wide)(NormArgs), void (*cluster)(NormArgs)) {
    const int64_t sms = device_sms();
    if (a.C <= 16384) return launch_early(narrow, dim3((unsigned)std::min(a.N, sms * 8)), dim3(256), 0, s, a);
    if (a.C <= 65536) return launch_early(wide, dim3((unsigned)std::min(a.N, sms * 2)), dim3(1024), 0, s, a);
    return launch_early(cluster, dim3((unsigned)std::min(a.N, sms / 4) * 8), dim3(1024), 0, s, a);
}

// Threads of a row by its number of 16-byte vectors (or of elements, where the
// width or an address is no multiple of 16 bytes).  Two vectors a thread where
// a warp can hold the row: of 1048576 x 256 bf16, 170 us (6.3 TB/s) with two,
// 189 with four, 193 with one; blocks of 128 threads, 32 an SM (16 to 64 the
// same, 8 15% slower).
template <typename TX, typename TW> cudaError_t norm_fwd_t(const NormArgs &a, bool vec, bool pairs, cudaStream_t s) {
    constexpr int EL = Elt<TX>::EL, P = sizeof(TX) == 2 ? 2 : 1;   // P: two bf16, one float
    const int nv = a.C / EL;
    if (vec && nv <= 8) return launch_fwd<TX, TW, EL, 4, 2>(a, s);
    if (vec && nv <= 16) return launch_fwd<TX, TW, EL, 8, 2>(a, s);
    if (vec && nv <= 32) return launch_fwd<TX, TW, EL, 16, 2>(a, s);
    if (vec && nv <= 64) return launch_fwd<TX, TW, EL, 32, 2>(a, s);
    if (vec && nv <= 128) return launch_fwd<TX, TW, EL, 32, 4>(a, s);
    if (vec && nv <= 1024) return launch_fwd<TX, TW, EL, 256, 4>(a, s);
    if (pairs && a.C <= 64) return launch_fwd<TX, TW, P, 8, 8 / P>(a, s);
    if (pairs && a.C <= 512) return launch_fwd<TX, TW, P, 32, 16 / P>(a, s);
    if (pairs && a.C <= 4096) return launch_fwd<TX, TW, P, 256, 16 / P>(a, s);
    if constexpr (P == 2) {   // an odd width, or bf16 rows off a 4-byte boundary
        if (a.C <= 64) return launch_fwd<TX, TW, 1, 16, 4>(a, s);
        if (a.C <= 512) return launch_fwd<TX, TW, 1, 32, 16>(a, s);
        if (a.C <= 4096) return launch_fwd<TX, TW, 1, 256, 16>(a, s);
    }
    note_launch(SGA_KERN_NORM_FWD, s, false);
    const cudaError_t e = launch_wide(
        a, s, vec ? norm_fwd_wide_kernel<TX, TW, EL, 256, 1> : norm_fwd_wide_kernel<TX, TW, 1, 256, 1>,
        vec ? norm_fwd_wide_kernel<TX, TW, EL, 1024, 1> : norm_fwd_wide_kernel<TX, TW, 1, 1024, 1>,
        vec ? norm_fwd_wide_kernel<TX, TW, EL, 1024, 8> : norm_fwd_wide_kernel<TX, TW, 1, 1024, 8>);
    note_launch(SGA_KERN_NORM_FWD, s, true);
    return e;
}

template <typename TX, typename TW> cudaError_t norm_bwd_t(const NormArgs &a, bool vec, bool pairs, TW *dw, TW *db, cudaStream_t s) {
    constexpr int EL = Elt<TX>::EL, P = sizeof(TX) == 2 ? 2 : 1;   // P: two bf16, one float
    const int nv = a.C / EL;
    int blocks = 0;
    cudaError_t e;
    if (vec && nv <= 8) e = launch_bwd_ring<TX, TW, 4, 2>(a, blocks, s);
    else if (vec && nv <= 16) e = launch_bwd_ring<TX, TW, 8, 2>(a, blocks, s);
    else if (vec && nv <= 32) e = launch_bwd_ring<TX, TW, 16, 2>(a, blocks, s);
    else if (vec && nv <= 64) e = launch_bwd_ring<TX, TW, 32, 2>(a, blocks, s);
    else if (vec && nv <= 512) e = launch_bwd<TX, TW, EL, 256, 2>(a, blocks, s);
    else if (pairs && a.C <= 64) e = launch_bwd<TX, TW, P, 8, 8 / P>(a, blocks, s);
    else if (pairs && a.C <= 512) e = launch_bwd<TX, TW, P, 32, 16 / P>(a, blocks, s);
    else if (pairs && a.C <= 4096) e = launch_bwd<TX, TW, P, 256, 16 / P>(a, blocks, s);
    else if (a.C <= 64) e = launch_bwd<TX, TW, 1, 16, 4>(a, blocks, s);
    else if (a.C <= 512) e = launch_bwd<TX, TW, 1, 32, 16>(a, blocks, s);
    else if (a.C <= 4096) e = launch_bwd<TX, TW, 1, 256, 16>(a, blocks, s);
    else {
        note_launch(SGA_KERN_NORM_BWD, s, false);
        e = launch_wide(a, s, vec ? norm_bwd_wide_kernel<TX, TW, EL, 256, 1> : norm_bwd_wide_kernel<TX, TW, 1, 256, 1>,
                        vec ? norm_bwd_wide_kernel<TX, TW, EL, 1024, 1> : norm_bwd_wide_kernel<TX, TW, 1, 1024, 1>,
                        vec ? norm_bwd_wide_kernel<TX, TW, EL, 1024, 8> : norm_bwd_wide_kernel<TX, TW, 1, 1024, 8>);
        note_launch(SGA_KERN_NORM_BWD, s, true);
        if (e != cudaSuccess || !a.part) return e;
        const int64_t want = std::min<int64_t>(bwd_blocks(device_sms()), (a.N + 15) / 16);
        const int64_t slab = (a.N + want - 1) / want;
        blocks = (int)((a.N + slab - 1) / slab);
        note_launch(SGA_KERN_NORM_BWD, s, false);
        e = launch_early(norm_cols_wide_kernel<TX>, dim3((unsigned)((a.C + 255) / 256), (unsigned)blocks), dim3(256), 0, s, a, slab);
        note_launch(SGA_KERN_NORM_BWD, s, true);
    }
    if (e != cudaSuccess || !a.part) return e;
    note_launch(SGA_KERN_NORM_REDUCE, s, false);
    const int64_t sums = 2 * (int64_t)a.C;
    // (wide rows have few blocks of sums and many columns)
    if (a.C > 4096 && blocks <= 32)
        e = launch_early(norm_reduce_few_kernel<TW>, dim3((unsigned)((sums + 255) / 256)), dim3(256), 0, s,
                         static_cast<const float *>(a.part), blocks, a.C, dw, db);
    else
        e = launch_early(norm_reduce_kernel<TW>, dim3((unsigned)((sums + 31) / 32)), dim3(1024), 0, s,
                         static_cast<const float *>(a.part), blocks, a.C, dw, db);
    note_launch(SGA_KERN_NORM_REDUCE, s, true);
    return e;
}

sga_status check_norm(int64_t N, int64_t C, sga_dtype dt, sga_dtype wdt) {
    if (N < 0 || C < 1) return SGA_EINVAL;
    if (dt != SGA_F32 && dt != SGA_BF16) return SGA_EUNSUPPORTED;
    if (wdt != SGA_F32 && wdt != dt) return SGA_EUNSUPPORTED;
    if (C > (1 << 20)) return SGA_EUNSUPPORTED;
    return SGA_OK;
}
size_t size_of(sga_dtype dt) { return dt == SGA_F32 ? 4 : 2; }

}  // namespace
}  // namespace sga

using namespace sga;

extern "C" {

sga_status layer_norm_fwd(const void *X, const void *weight, const void *bias, int64_t N, int64_t C, float eps,
                          sga_dtype dt, sga_dtype wdt, void *out, float *mean, float *rstd, void *stream) {
    sga_status st = check_norm(N, C, dt, wdt);
    if (st != SGA_OK) return st;
    if (!(eps >= 0.f) || !(eps < INFINITY) || (bias && !weight)) return SGA_EINVAL;
    if (N == 0) return SGA_OK;
    const size_t e = size_of(dt), we = size_of(wdt);
    if (!X || !out || !mean || !rstd || !aligned(X, e) || !aligned(out, e) || !aligned(mean, 4) || !aligned(rstd, 4) ||
        !aligned(weight, we) || !aligned(bias, we))
        return SGA_EINVAL;
    NormArgs a{};
    a.X = X;
    a.w = weight;
    a.b = bias;
    a.Y = out;
    a.mean = mean;
    a.rstd = rstd;
    a.N = N;
    a.C = (int)C;
    a.eps = eps;
    // rows on 16-byte boundaries are moved 16 bytes at a time, bf16 rows of an even width two elements at a time
    auto fits = [&](size_t row, size_t w) {
        return C * e % row == 0 && aligned(X, row) && aligned(out, row) && aligned(weight, w) && aligned(bias, w);
    };
    const bool vec = fits(16, 16), pairs = fits(4, dt == SGA_F32 ? 4 : 2 * we);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dt == SGA_F32) return status_of(norm_fwd_t<float, float>(a, vec, pairs, s));
    if (wdt == SGA_F32) return status_of(norm_fwd_t<__nv_bfloat16, float>(a, vec, pairs, s));
    return status_of(norm_fwd_t<__nv_bfloat16, __nv_bfloat16>(a, vec, pairs, s));
}

size_t sga_norm_bwd_workspace_bytes(int64_t N, int64_t C) {
    if (N <= 0 || C <= 0) return 0;
    const int64_t most = C > 4096 ? (N + 15) / 16 : N;   // (wide rows: slabs of at least 16)
    return (size_t)std::min<int64_t>(bwd_blocks(device_sms()), most) * 2 * (size_t)C * sizeof(float);
}

sga_status layer_norm_bwd(const void *X, const void *weight, const float *mean, const float *rstd, const void *dOut,
                          int64_t N, int64_t C, sga_dtype dt, sga_dtype wdt, void *dX, void *dweight, void *dbias,
                          void *workspace, size_t workspace_bytes, void *stream) {
    sga_status st = check_norm(N, C, dt, wdt);
    if (st != SGA_OK) return st;
    if ((dweight || dbias) && !weight) return SGA_EINVAL;
    if (dbias && !dweight) return SGA_EINVAL;
    const size_t e = size_of(dt), we = size_of(wdt);
    if (!aligned(weight, we) || !aligned(dweight, we) || !aligned(dbias, we)) return SGA_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) {   // an empty sum
        cudaError_t ce = cudaSuccess;
        if (dweight) ce = cudaMemsetAsync(dweight, 0, C * we, s);
        if (ce == cudaSuccess && dbias) ce = cudaMemsetAsync(dbias, 0, C * we, s);
        return status_of(ce);
    }
    if (!X || !dOut || !dX || !mean || !rstd || !aligned(X, e) || !aligned(dOut, e) || !aligned(dX, e) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return SGA_EINVAL;
    if (dweight) {
        if (!workspace || !aligned(workspace, 16)) return SGA_EINVAL;
        if (workspace_bytes < sga_norm_bwd_workspace_bytes(N, C)) return SGA_EWORKSPACE;
    }
    NormArgs a{};
    a.X = X;
    a.w = weight;
    a.dY = dOut;
    a.dX = dX;
    a.mean_in = mean;
    a.rstd_in = rstd;
    a.part = dweight ? static_cast<float *>(workspace) : nullptr;
    a.N = N;
    a.C = (int)C;
    auto fits = [&](size_t row, size_t w) {
        return C * e % row == 0 && aligned(X, row) && aligned(dOut, row) && aligned(dX, row) && aligned(weight, w);
    };
    const bool vec = fits(16, 16), pairs = fits(4, dt == SGA_F32 ? 4 : 2 * we);
    if (dt == SGA_F32)
        return status_of(norm_bwd_t<float, float>(a, vec, pairs, static_cast<float *>(dweight), static_cast<float *>(dbias), s));
    if (wdt == SGA_F32)
        return status_of(norm_bwd_t<__nv_bfloat16, float>(a, vec, pairs, static_cast<float *>(dweight),
                                                          static_cast<float *>(dbias), s));
    return status_of(norm_bwd_t<__nv_bfloat16, __nv_bfloat16>(a, vec, pairs, static_cast<__nv_bfloat16 *>(dweight),
                                                              static_cast<__nv_bfloat16 *>(dbias), s));
}

}  // extern "C"
