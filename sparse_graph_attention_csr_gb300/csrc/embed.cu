// Embedding lookup with scaling, and its gradient by sorted tokens, or without a
// sort into few rows.
//   forward:  out_t = scale table[id_t]
//   backward: dTable_v = scale sum over the tokens t with id_t = v of dOut_t
//
// Both are bound by DRAM (rows read once, rows written once).  The gradient
// sorts (id, token) pairs, stably, so that the tokens of a row lie together in
// token order, and sums them in fixed chunks of the sorted list, one warp a
// chunk: every warp has the same number of tokens however uneven their
// frequencies are.  A row whose tokens lie inside one chunk is written from
// there; where a row crosses chunks, each chunk leaves an fp32 partial, and a
// block adds the row's partials in chunk order.  No float atomics: the sums'
// order is fixed and results are bitwise reproducible.
#include <algorithm>
#include <type_traits>

#include <cooperative_groups.h>

#include "common.cuh"
#include "tc.cuh"

namespace cg = cooperative_groups;

namespace sga {

void set_cuda_error(cudaError_t e);   // (api.cu)

namespace {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t round256(size_t b) { return (b + 255) & ~size_t(255); }

sga_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return SGA_OK;
    set_cuda_error(e);
    return SGA_ECUDA;
}

// Bit kErrIndexRange: an id outside [0, V) since the last read, per device.
__device__ int32_t g_embed_err;

__device__ __forceinline__ int64_t id_at(const void *ids, int64_t t, bool wide) {
    return wide ? __ldg(static_cast<const long long *>(ids) + t) : (int64_t)__ldg(static_cast<const int *>(ids) + t);
}

// One element group: 16 bytes (VEC) or one element.
template <typename T, bool VEC> constexpr int kEl = VEC ? Elt<T>::EL : 1;
template <typename T, bool VEC> __device__ __forceinline__ void load_g(const T *p, float *x) {
    if constexpr (VEC) unpack<T>(ldg16_stream(p), x);
    else x[0] = to_f32<T>(__ldg(p));
}
template <typename T, bool VEC> __device__ __forceinline__ void store_g(T *p, const float *x) {
    if constexpr (VEC) __stcs(reinterpret_cast<uint4 *>(p), pack<T>(x));
    else *p = from_f32<T>(x[0]);
}

// ---- forward ------------------------------------------------------------------

// A warp takes 32 >> sh tokens at a time (1 << sh lanes each); U groups of a
// lane's row are loaded before any is stored.  Where there are few tokens, their
// columns are spread over gridDim.y blocks (1 of 2^20 bf16: 5.5 us, 297 by one warp).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const void *__restrict__ ids, bool wide, const T *__restrict__ table,
                                                        int64_t N, int64_t V, int C, float scale, int sh, T *out) {
    constexpr int EL = kEl<T, VEC>, U = 4;
    let_next_start();
    wait_previous();
    const int n = C / EL, lanes = 1 << sh, sub = threadIdx.x & (lanes - 1);
    const int64_t step = ((int64_t)gridDim.x * blockDim.x) >> sh;
    for (int64_t t = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> sh; t < N; t += step) {
        const int64_t id = id_at(ids, t, wide);
        const bool ok = id >= 0 && id < V;
        if (!ok && sub == 0 && blockIdx.y == 0) atomicOr(&g_embed_err, kErrIndexRange);
        const T *src = table + (ok ? id : 0) * C;
        T *dst = out + t * C;
        for (int c0 = sub + (int)blockIdx.y * U * lanes; c0 < n; c0 += U * lanes * (int)gridDim.y) {
            float x[U][EL];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * lanes;
#pragma unroll
                for (int i = 0; i < EL; ++i) x[u][i] = 0.f;
                if (c < n && ok) load_g<T, VEC>(src + (int64_t)c * EL, x[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * lanes;
                if (c >= n) continue;
#pragma unroll
                for (int i = 0; i < EL; ++i) x[u][i] *= scale;
                store_g<T, VEC>(dst + (int64_t)c * EL, x[u]);
            }
        }
    }
}

// ---- backward -----------------------------------------------------------------
//
// One cooperative launch (at most a block per SM, grid barriers between the steps):
//   sort: least significant digit first, digits of at most 8 bits.  A warp owns
//     a run of consecutive tokens and counts their digits in shared memory; a
//     block adds its warps' counts per digit, then each block all blocks', and
//     every warp places its tokens in order (equal digits of 32
//     tokens ranked by lane), so the sort is stable.  Counts are whole numbers:
//     the order in which they are added does not matter.
//   sums: groups of lanes over chunks of the sorted list, as described above;
//   joins: a warp per chunk whose last row runs on; rows of more than kLongRow
//     chunks by the whole block.
// The table's rows without a token are zeroed in the first step, whose latency
// hides the stores.

constexpr int kSortThreads = 1024, kSortWarps = 32;
constexpr int kDigits = 256;
constexpr int kLongRow = 8;
constexpr int kJoinCols = 4096;   // columns that a warp joins (wider rows: several warps)

struct GradArgs {
    const void *ids, *dOut;
    void *dTable;
    int32_t *key[2], *tok[2];   // ping-pong buffers of the sort
    int32_t *hist;              // [digit][block] counts
    float *part;                // [chunks][2][C]: the row that runs on from the chunk before, the row that runs on
    int64_t N, V, chunks, padding;
    int wide, L, C, bits, passes, gshift, few;
    float scale;
};

// Sort key of a token: its id, or V (last, never summed) for the padding id
// and for an id outside the table.
__device__ __forceinline__ int32_t key_of(const GradArgs &a, int64_t t) {
    int64_t id = id_at(a.ids, t, a.wide);
    if (id < 0 || id >= a.V) {
        atomicOr(&g_embed_err, kErrIndexRange);
        id = a.V;
    }
    return (int32_t)(id == a.padding ? a.V : id);
}

__device__ void sort_tokens(const GradArgs &a, int32_t (*cnt)[kDigits], int32_t *scan) {
    cg::grid_group grid = cg::this_grid();
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, B = gridDim.x;
    const int64_t per = (a.N + B - 1) / B, per_w = (per + kSortWarps - 1) / kSortWarps;
    const int64_t b0 = blockIdx.x * per, b1 = min(a.N, b0 + per);
    const int64_t w0 = min(b1, b0 + wp * per_w), w1 = min(b1, w0 + per_w);
    for (int p = 0; p < a.passes; ++p) {
        const int shift = p * a.bits;
        const int32_t mask = (1 << a.bits) - 1;
        const int32_t *kin = a.key[p & 1], *vin = a.tok[p & 1];
        int32_t *kout = a.key[(p + 1) & 1], *vout = a.tok[(p + 1) & 1];
        for (int d = lane; d < kDigits; d += 32) cnt[wp][d] = 0;
        __syncwarp();
        for (int64_t e = w0 + lane; e < w1; e += 128) {   // four keys of a lane in flight
            int32_t k[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) k[z] = e + 32 * z < w1 ? (p ? __ldcg(kin + e + 32 * z) : key_of(a, e + 32 * z)) : -1;
#pragma unroll
            for (int z = 0; z < 4; ++z)
                if (k[z] >= 0) atomicAdd(&cnt[wp][(k[z] >> shift) & mask], 1);
        }
        __syncthreads();
        if (threadIdx.x < kDigits) {
            int32_t run = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                const int32_t c = cnt[w][threadIdx.x];
                cnt[w][threadIdx.x] = run;
                run += c;
            }
            a.hist[(int64_t)threadIdx.x * B + blockIdx.x] = run;
        }
        grid.sync();
        // every block adds the counts itself (40 loads a lane in flight at once, cheaper
        // than a further step with its barrier): of a digit, all blocks' and the earlier blocks'
        {
            constexpr int DW = kDigits / kSortWarps;
            int32_t all[DW], before[DW];
#pragma unroll
            for (int k = 0; k < DW; ++k) all[k] = before[k] = 0;
            const int32_t *h = a.hist + (int64_t)(wp * DW) * B;
            for (int i0 = 0; i0 < B; i0 += 160) {
                int32_t c[5][DW];
#pragma unroll
                for (int z = 0; z < 5; ++z)
#pragma unroll
                    for (int k = 0; k < DW; ++k) {
                        const int i = i0 + 32 * z + lane;
                        c[z][k] = i < B ? __ldcg(h + k * B + i) : 0;
                    }
#pragma unroll
                for (int z = 0; z < 5; ++z)
#pragma unroll
                    for (int k = 0; k < DW; ++k) {
                        all[k] += c[z][k];
                        before[k] += i0 + 32 * z + lane < (int)blockIdx.x ? c[z][k] : 0;
                    }
            }
#pragma unroll
            for (int k = 0; k < DW; ++k) {
                const int32_t t = __reduce_add_sync(SGA_FULL_MASK, all[k]), q = __reduce_add_sync(SGA_FULL_MASK, before[k]);
                if (lane == 0) {
                    scan[kSortWarps + wp * DW + k] = t;
                    scan[kSortWarps + kDigits + wp * DW + k] = q;
                }
            }
        }
        __syncthreads();
        // first position of every digit: exclusive sums over the digits' totals
        int32_t first = 0;
        if (threadIdx.x < kDigits) {
            const int32_t c = scan[kSortWarps + threadIdx.x];
            int32_t x = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t y = __shfl_up_sync(SGA_FULL_MASK, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) scan[wp] = x;
            first = x - c;
        }
        __syncthreads();
        if (threadIdx.x < kDigits) {
            for (int w = 0; w < wp; ++w) first += scan[w];
            scan[kSortWarps + kDigits + threadIdx.x] += first;
        }
        __syncthreads();
        for (int d = lane; d < kDigits; d += 32) cnt[wp][d] += scan[kSortWarps + kDigits + d];
        __syncwarp();
        for (int64_t e0 = w0; e0 < w1; e0 += 128) {
            int32_t k[4], v[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int64_t e = e0 + 32 * z + lane;
                k[z] = e < w1 ? (p ? __ldcg(kin + e) : key_of(a, e)) : -1;
                v[z] = e < w1 ? (p ? __ldcg(vin + e) : (int32_t)e) : 0;
            }
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                if (e0 + 32 * z >= w1) break;
                const bool valid = k[z] >= 0;
                const int d = valid ? (k[z] >> shift) & mask : kDigits;
                const unsigned peers = __match_any_sync(SGA_FULL_MASK, d);
                const int rank = __popc(peers & ((1u << lane) - 1u));
                int32_t pos = 0;
                if (valid) pos = cnt[wp][d] + rank;
                __syncwarp();
                if (valid) {
                    kout[pos] = k[z];
                    vout[pos] = v[z];
                    if (rank == 0) cnt[wp][d] = pos + __popc(peers);
                }
                __syncwarp();
            }
        }
        grid.sync();
    }
}

// A group of 1 << gshift lanes per (chunk of L sorted tokens, slab of U groups
// of columns a lane).
template <typename T, bool VEC, int U> __device__ __forceinline__ void sum_chunks(const GradArgs &a) {
    constexpr int EL = kEl<T, VEC>;
    const int32_t *key = a.key[a.passes & 1], *tok = a.tok[a.passes & 1];
    const int lanes = 1 << a.gshift, sub = threadIdx.x & (lanes - 1), n = a.C / EL, step = lanes * U;
    const int slabs = (n + step - 1) / step;
    const T *dOut = static_cast<const T *>(a.dOut);
    T *dTable = static_cast<T *>(a.dTable);
    const int64_t items = a.chunks * slabs, groups = ((int64_t)gridDim.x * kSortThreads) >> a.gshift;
    // neighbouring chunks on different SMs: the hot rows' chunks, alike in cost, are spread
    for (int64_t it = (((int64_t)threadIdx.x >> a.gshift) * gridDim.x) + blockIdx.x; it < items; it += groups) {
        const int64_t chunk = it / slabs;
        const int g0 = (int)(it % slabs) * step + sub;
        const int64_t k0 = chunk * a.L, k1 = min(a.N, k0 + a.L);
        float acc[U][EL];
        int32_t cur = __ldcg(key + k0);
        bool joined = k0 > 0 && __ldcg(key + k0 - 1) == cur;   // the first run continues one of the chunk before
        auto clear = [&] {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < EL; ++i) acc[u][i] = 0.f;
        };
        auto flush = [&](bool goes_on) {
            if (cur >= a.V) return;
            if (joined || goes_on) {
                float *p = a.part + ((chunk * 2) + (joined ? 0 : 1)) * a.C;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (g0 + lanes * u < n)
#pragma unroll
                        for (int i = 0; i < EL; ++i) p[(g0 + lanes * u) * EL + i] = acc[u][i];
            } else {
                T *o = dTable + (int64_t)cur * a.C;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (g0 + lanes * u < n) {
                        float y[EL];
#pragma unroll
                        for (int i = 0; i < EL; ++i) y[i] = acc[u][i] * a.scale;
                        store_g<T, VEC>(o + (int64_t)(g0 + lanes * u) * EL, y);
                    }
            }
        };
        clear();
        for (int64_t q = k0; q < k1; q += 4) {   // L is a multiple of four, the lists are padded to one
            const int4 kk = __ldcg(reinterpret_cast<const int4 *>(key + q)), tt = __ldcg(reinterpret_cast<const int4 *>(tok + q));
            const int32_t ks[4] = {kk.x, kk.y, kk.z, kk.w}, ts[4] = {tt.x, tt.y, tt.z, tt.w};
            uint4 raw[4][U];
#pragma unroll
            for (int z = 0; z < 4; ++z)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    raw[z][u] = make_uint4(0, 0, 0, 0);
                    if (q + z < k1 && ks[z] < a.V && g0 + lanes * u < n) {
                        const T *p = dOut + (int64_t)ts[z] * a.C + (int64_t)(g0 + lanes * u) * EL;
                        if constexpr (VEC) raw[z][u] = ldg16_stream(p);
                        else raw[z][u].x = __float_as_uint(to_f32<T>(__ldg(p)));
                    }
                }
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                if (q + z >= k1) break;
                if (ks[z] != cur) {
                    flush(false);
                    clear();
                    cur = ks[z];
                    joined = false;
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float x[EL];
                    if constexpr (VEC) unpack<T>(raw[z][u], x);
                    else x[0] = __uint_as_float(raw[z][u].x);
#pragma unroll
                    for (int i = 0; i < EL; ++i) acc[u][i] += x[i];
                }
            }
        }
        flush(k1 < a.N && __ldcg(key + k1) == cur);
    }
}

// Whether chunk c0's last row begins in it and runs on (the warp together): its
// id and the last chunk that begins with it, found 32 chunks at a time.
__device__ __forceinline__ bool runs_on(const GradArgs &a, const int32_t *key, int64_t c0, int32_t &cur, int64_t &cl) {
    const int lane = threadIdx.x & 31;
    const int64_t kl = (c0 + 1) * a.L - 1;   // the chunk's last token
    if (c0 >= a.chunks || kl + 1 >= a.N) return false;
    const int64_t at = lane == 0 ? kl : lane == 1 ? kl + 1 : c0 > 0 ? c0 * a.L - 1 : kl;
    const int32_t k = lane < 3 ? __ldcg(key + at) : 0;
    cur = __shfl_sync(SGA_FULL_MASK, k, 0);
    const int32_t next = __shfl_sync(SGA_FULL_MASK, k, 1), prev = __shfl_sync(SGA_FULL_MASK, k, 2);
    if (cur >= a.V || next != cur || (c0 > 0 && prev == cur)) return false;   // (prev: the row began in an earlier chunk)
    auto more = [&](int64_t stride) {   // chunks cl + stride, cl + 2 stride, .. that begin with the row: how many of 32
        const int64_t c = cl + (lane + 1) * stride;
        return __popc(__ballot_sync(SGA_FULL_MASK, c < a.chunks && __ldcg(key + (c < a.chunks ? c * a.L : 0)) == cur));
    };
    cl = c0 + 1;   // (it begins with token kl + 1)
    int n = more(1);
    cl += n;
    if (n == 32) {
        while ((n = more(32)) > 0) cl += 32 * (int64_t)n;
        cl += more(1);
    }
    return true;
}

// W consecutive columns of the partials.
template <int W> struct Cols {
    float x[W];
    __device__ __forceinline__ void load(const float *p) {
        if constexpr (W == 4) {
            const float4 q = __ldcg(reinterpret_cast<const float4 *>(p));
            x[0] = q.x;
            x[1] = q.y;
            x[2] = q.z;
            x[3] = q.w;
        } else {
            x[0] = __ldcg(p);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = 0.f;
    }
    __device__ __forceinline__ void add(const Cols &o) {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] += o.x[i];
    }
    template <typename T> __device__ __forceinline__ void store(T *o, float scale) const {
#pragma unroll
        for (int i = 0; i < W; ++i) o[i] = from_f32<T>(x[i] * scale);
    }
};

// The partials of the chunks [b, e) (slot 0) at column `col`, M of them in flight.
template <int W, int M> __device__ __forceinline__ Cols<W> columns_of(const GradArgs &a, int64_t b, int64_t e, int col) {
    Cols<W> s;
    s.zero();
    for (int64_t c = b; c < e; c += M) {
        Cols<W> v[M];
#pragma unroll
        for (int z = 0; z < M; ++z) {
            v[z].zero();
            if (c + z < e) v[z].load(a.part + (c + z) * 2 * a.C + col);
        }
#pragma unroll
        for (int z = 0; z < M; ++z) s.add(v[z]);
    }
    return s;
}

// sm: kSortWarps * 32 * W floats.
template <typename T, int W> __device__ __forceinline__ void join_rows(const GradArgs &a, float *sm, int64_t (*who)[4]) {
    const int32_t *key = a.key[a.passes & 1];
    T *dTable = static_cast<T *>(a.dTable);
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int64_t slabs = (a.C + kJoinCols - 1) / kJoinCols, items = a.chunks * slabs;   // (chunk, columns)
    // a block's items are apart: the hot rows, which begin close together, go to different blocks
    for (int64_t base = 0; base < items; base += (int64_t)gridDim.x * kSortWarps) {
        const int64_t it = base + (int64_t)wp * gridDim.x + blockIdx.x, c0 = it / slabs;   // (past the last chunk: nothing runs on)
        const int k0 = (int)(it % slabs) * kJoinCols, k1 = min(a.C, k0 + kJoinCols);
        int32_t cur = 0;
        int64_t cl = 0;
        const bool on = runs_on(a, key, c0, cur, cl);
        const bool lng = on && cl - c0 > kLongRow;
        if (lane == 0) {
            who[wp][0] = lng ? cl : -1;
            who[wp][1] = c0;
            who[wp][2] = cur;
            who[wp][3] = k0;
        }
        const bool any = __syncthreads_or(lng);
        if (on && !lng)
            for (int col = k0 + lane * W; col < k1; col += 32 * W) {
                Cols<W> s;
                s.load(a.part + (c0 * 2 + 1) * a.C + col);
                s.add(columns_of<W, kLongRow / 2>(a, c0 + 1, cl + 1, col));
                s.store(dTable + (int64_t)cur * a.C + col, a.scale);
            }
        if (!any) continue;
        // long rows by the whole block: a warp per 32 W columns and share of the chunks
        const int cols = min(kSortWarps, (a.C + 32 * W - 1) / (32 * W)), shares = kSortWarps / cols, slab = wp % cols,
                  share = wp / cols;
        for (int w = 0; w < kSortWarps; ++w) {
            const int64_t l = who[w][0];
            if (l < 0) continue;   // (the same for the whole block)
            const int64_t f = who[w][1], id = who[w][2], per = (l - f + shares - 1) / shares;
            const int last = min(a.C, (int)who[w][3] + kJoinCols);
            for (int cb = (int)who[w][3]; cb < last; cb += 32 * W * cols) {
                const int col = cb + (slab * 32 + lane) * W;
                Cols<W> s;
                s.zero();
                if (col < last && share < shares) {
                    s = columns_of<W, 8>(a, min(l + 1, f + 1 + share * per), min(l + 1, f + 1 + (share + 1) * per), col);
                    if (share == 0) {
                        Cols<W> v;
                        v.load(a.part + (f * 2 + 1) * a.C + col);
                        s.add(v);
                    }
                }
#pragma unroll
                for (int i = 0; i < W; ++i) sm[(wp * 32 + lane) * W + i] = s.x[i];
                __syncthreads();
                if (share == 0 && col < last) {
                    for (int q = 1; q < shares; ++q)
#pragma unroll
                        for (int i = 0; i < W; ++i) s.x[i] += sm[((q * cols + slab) * 32 + lane) * W + i];
                    s.store(dTable + id * a.C + col, a.scale);
                }
                __syncthreads();
            }
        }
        __syncthreads();
    }
}

template <typename T, bool VEC> __global__ void __launch_bounds__(kSortThreads, 1) embed_grad_kernel(const GradArgs a) {
    __shared__ int32_t cnt[kSortWarps][kDigits];
    __shared__ int32_t scan[kSortWarps + 2 * kDigits];
    __shared__ int64_t who[kSortWarps][4];
    const int64_t t0 = (int64_t)blockIdx.x * kSortThreads + threadIdx.x, nt = (int64_t)gridDim.x * kSortThreads;
    if constexpr (VEC) {
        for (int64_t i = t0; i < a.V * a.C / Elt<T>::EL; i += nt)
            reinterpret_cast<uint4 *>(a.dTable)[i] = make_uint4(0, 0, 0, 0);
    } else {
        for (int64_t i = t0; i < a.V * a.C; i += nt) static_cast<T *>(a.dTable)[i] = from_f32<T>(0.f);
    }
    sort_tokens(a, cnt, scan);
    sum_chunks<T, VEC, VEC ? 1 : 4>(a);
    cg::this_grid().sync();
    static_assert(sizeof cnt >= kSortWarps * 32 * 4 * sizeof(float), "joins");
    if (a.C % 4 == 0) join_rows<T, 4>(a, reinterpret_cast<float *>(cnt), who);
    else join_rows<T, 1>(a, reinterpret_cast<float *>(cnt), who);
}

// Few rows (atom or edge types) and few tokens: no sort.  A block takes consecutive
// tokens; each of its warps owns every 32nd row, finds the rows' tokens by votes
// over the block's ids and adds them in order, so that nothing is shared.  Of 16
// rows and fewer, 32 / R warps share the rows that are alike modulo R and take a
// part of the columns each; blocks that are fewer than the SMs share their columns
// with gridDim.y others (1000 x 4096 bf16 into 1 row: 18.5 us, 197 by one warp a
// block).  Then the blocks' sums are added.  STAGED: the block's part of dOut, which
// is contiguous, is copied to shared memory while the ids are listed, so that a warp
// with a frequent row does not wait for memory batch after batch. 30011 tokens x 100
// into 119 rows, id i with a weight of 1 / i: fp32 14.4 us a call (2.5 more from
// memory, 28 sorted), bf16 13.6 (8.5 more from memory).  At the ends of its range it
// is still the faster one: 70000 x 100 into 256 rows 21 us (257 rows, sorted: fp32
// 42, bf16 46), 76000 x 100 into 119 rows fp32 25, bf16 20 (80000, sorted: 36, 40);
// past them a block's lists would have to be walked again.
constexpr int kFewRows = 256, kFewTokens = 512;   // rows; tokens of a block
constexpr size_t kStage = 220 * 1024;             // shared memory beside the lists

// SHARED: 16 rows and fewer.
template <typename T, bool VEC, bool STAGED, bool SHARED>
__global__ void __launch_bounds__(kSortThreads, 1) embed_grad_few_kernel(const GradArgs a, int64_t per) {
    constexpr int EL = kEl<T, VEC>, M = VEC ? 8 : 4, U = VEC ? 1 : 4;   // M tokens in flight, of U groups each
    __shared__ int32_t id[kFewTokens];
    __shared__ uint16_t found[kFewTokens], sorted[kFewTokens];   // the warps' tokens in order, and by row: token | row / 32 << 9
    __shared__ int32_t count[kSortWarps];
    extern __shared__ __align__(16) unsigned char stage[];
    static_assert(kFewTokens <= 512 && kFewRows <= 32 * 128, "list entries");
    let_next_start();
    wait_previous();
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, V = (int)a.V, n = a.C / EL;
    // the warp's rows (own, own + R, ..) and columns (groups [n0, n1), every parts-th 32 U of them)
    const int rsh = !SHARED ? 5 : V > 1 ? 32 - __clz(V - 1) : 0, R = 1 << rsh, own = wp & (R - 1), part_of = wp >> rsh, parts = kSortWarps >> rsh;
    int n0 = 0, n1 = n;
    if constexpr (!STAGED) {
        const int rounds = (n + 32 * U - 1) / (32 * U), share = (rounds + (int)gridDim.y - 1) / (int)gridDim.y * 32 * U;
        n0 = (int)blockIdx.y * share;
        n1 = min(n, n0 + share);
    }
    const int64_t t0 = min(a.N, blockIdx.x * per);
    const int cnt = (int)min(per, a.N - t0);
    const T *dOut = static_cast<const T *>(a.dOut) + t0 * a.C;
    if constexpr (STAGED) {   // (the part begins on 16 bytes: `per` is a multiple of 8)
        const int all = cnt * a.C, whole = all / Elt<T>::EL;
        for (int i = threadIdx.x; i < whole; i += kSortThreads)
            tc::cp16(tc::smem_u32(stage) + 16 * i, dOut + (int64_t)i * Elt<T>::EL, true);
        tc::cp_commit();
        for (int i = whole * Elt<T>::EL + threadIdx.x; i < all; i += kSortThreads)
            reinterpret_cast<T *>(stage)[i] = dOut[i];
    }
    for (int i = threadIdx.x; i < kFewTokens; i += kSortThreads) id[i] = i < cnt ? key_of(a, t0 + i) : V;
    __syncthreads();
    float *part = a.part + ((int64_t)blockIdx.x * V + own) * a.C;   // the warp's first row; the next is R rows on
    const uint32_t below = (1u << lane) - 1u;
    auto mine = [&](int b) { return (id[b + lane] & (R - 1)) == own && id[b + lane] < V; };
    int total = 0;
    for (int b = 0; b < cnt; b += 32) total += __popc(__ballot_sync(SGA_FULL_MASK, mine(b)));
    if (lane == 0) count[wp] = total;
    __syncthreads();
    const int base = __reduce_add_sync(SGA_FULL_MASK, lane < own ? count[lane] : 0);
    uint16_t *f = found + base, *list = sorted + base;
    if (part_of == 0) {   // (the parts read what the first one lists)
        for (int b = 0, at = 0; b < cnt; b += 32) {
            const bool on = mine(b);
            const uint32_t who = __ballot_sync(SGA_FULL_MASK, on);
            if (on) f[at + __popc(who & below)] = (uint16_t)((b + lane) | (id[b + lane] >> rsh) << 9);
            at += __popc(who);
        }
        __syncwarp();
        for (int q = 0, at = 0; own + R * q < V; ++q) {
            const int before = at;
            for (int b = 0; b < total; b += 32) {
                const int e = b + lane < total ? f[b + lane] : -1;
                const uint32_t who = __ballot_sync(SGA_FULL_MASK, e >> 9 == q);
                if (e >> 9 == q) list[at + __popc(who & below)] = (uint16_t)e;
                at += __popc(who);
            }
            if (at == before)   // a row without a token here
                for (int c = n0 * EL + lane; c < n1 * EL; c += 32) part[(int64_t)R * q * a.C + c] = 0.f;
        }
    }
    if constexpr (STAGED) {
        tc::cp_wait<0>();
        dOut = reinterpret_cast<const T *>(stage);
    }
    __syncthreads();
    for (int g0 = n0 + part_of * 32 * U + lane; g0 - lane < n1; g0 += 32 * U * parts) {
        float acc[U][EL];
        int cur = -1;
        auto flush = [&] {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < EL; ++i) {
                    if (cur >= 0 && g0 + 32 * u < n1) part[(int64_t)R * cur * a.C + (g0 + 32 * u) * EL + i] = acc[u][i];
                    acc[u][i] = 0.f;
                }
        };
        flush();
        for (int k = 0; k < total; k += M) {
            uint4 raw[M][U];
            int row[M];
#pragma unroll
            for (int z = 0; z < M; ++z) {
                const int e = k + z < total ? list[k + z] : -1;
                row[z] = e >> 9;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    raw[z][u] = make_uint4(0, 0, 0, 0);
                    if (e < 0 || g0 + 32 * u >= n1) continue;
                    const T *p = dOut + (int64_t)(e & 511) * a.C + (int64_t)(g0 + 32 * u) * EL;
                    if constexpr (VEC) raw[z][u] = STAGED ? *reinterpret_cast<const uint4 *>(p) : ldg16_stream(p);
                    else raw[z][u].x = __float_as_uint(to_f32<T>(STAGED ? *p : __ldg(p)));
                }
            }
#pragma unroll
            for (int z = 0; z < M; ++z) {
                if (row[z] < 0) break;
                if (row[z] != cur) {
                    flush();
                    cur = row[z];
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float x[EL];
                    if constexpr (VEC) unpack<T>(raw[z][u], x);
                    else x[0] = __uint_as_float(raw[z][u].x);
#pragma unroll
                    for (int i = 0; i < EL; ++i) acc[u][i] += x[i];
                }
            }
        }
        flush();
    }
}

// The blocks' sums of every row: a warp per W columns of a row, its lanes take
// every 32nd block's.
template <typename T, int W> __global__ void __launch_bounds__(256) embed_add_few_kernel(const GradArgs a, int B) {
    let_next_start();
    wait_previous();
    const int lane = threadIdx.x & 31;
    const int64_t stride = a.V * a.C, it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (it >= stride / W) return;
    Cols<W> s;
    s.zero();
    for (int b0 = 0; b0 < B; b0 += 160) {
        Cols<W> x[5];
#pragma unroll
        for (int z = 0; z < 5; ++z) {
            x[z].zero();
            const int b = b0 + 32 * z + lane;
            if (b < B) x[z].load(a.part + b * stride + it * W);
        }
#pragma unroll
        for (int z = 0; z < 5; ++z) s.add(x[z]);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) s.x[i] = group_sum<32>(s.x[i]);
    if (lane == 0) s.store(static_cast<T *>(a.dTable) + it * W, a.scale);
}

// The same of few blocks: a thread per W columns, whatever their number.
template <typename T, int W> __global__ void __launch_bounds__(256) embed_add_fewer_kernel(const GradArgs a, int B) {
    let_next_start();
    wait_previous();
    const int64_t stride = a.V * a.C, it = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (it >= stride / W) return;
    Cols<W> s;
    s.zero();
    for (int b0 = 0; b0 < B; b0 += 4) {
        Cols<W> x[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            x[z].zero();
            if (b0 + z < B) x[z].load(a.part + (b0 + z) * stride + it * W);
        }
#pragma unroll
        for (int z = 0; z < 4; ++z) s.add(x[z]);
    }
    s.store(static_cast<T *>(a.dTable) + it * W, a.scale);
}

// Blocks of the gradient's launch: one an SM, fewer where that leaves them under
// 256 tokens and 16384 elements of the table, which the same blocks zero (100
// tokens into 50257 x 512 bf16: 34 us, 804 with a block a 256 tokens alone).
int grad_blocks(int64_t N, int64_t V, int64_t C, int sms) {
    return (int)std::min<int64_t>(sms, std::max<int64_t>((N + 255) / 256, (V * C + 16383) / 16384));
}

// Sorted tokens of a chunk: an equal share of the resident warps, at least 16.
int chunk_len(int64_t N, int sms) {
    const int64_t per = (N + (int64_t)sms * kSortWarps - 1) / ((int64_t)sms * kSortWarps);
    return (int)std::max<int64_t>(16, (per + 3) / 4 * 4);
}

// Tokens of a block where the gradient goes without the sort (0: it is sorted):
// a block an SM, but as many tokens as rows, so that the blocks' sums are no
// more than the tokens, and at least 128; a multiple of 8.
int few_tokens(int64_t N, int64_t V, int sms) {
    const int64_t per = (std::max<int64_t>(std::max<int64_t>(128, V), (N + sms - 1) / sms) + 7) / 8 * 8;
    return V > 0 && V <= kFewRows && V <= N && per <= kFewTokens ? (int)per : 0;
}

int bits_of(int64_t v) {
    int b = 1;
    while ((v >> b) != 0) ++b;
    return b;
}

struct Layout {
    size_t key[2], tok[2], hist, part, bytes;
};
Layout layout(int64_t N, int64_t V, int64_t C, int sms) {
    Layout l{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += round256(bytes);
        return at;
    };
    if (const int per = few_tokens(N, V, sms)) {
        l.part = take((size_t)((N + per - 1) / per) * V * C * 4);
        l.bytes = off;
        return l;
    }
    for (int i = 0; i < 2; ++i) {
        l.key[i] = take((size_t)N * 4 + 16);
        l.tok[i] = take((size_t)N * 4 + 16);
    }
    l.hist = take((size_t)kDigits * grad_blocks(N, V, C, sms) * 4);
    const int L = chunk_len(N, sms);
    l.part = take((size_t)((N + L - 1) / L) * 2 * C * 4);
    l.bytes = off;
    return l;
}

template <typename T, bool VEC> cudaError_t grad_t(GradArgs a, int blocks, cudaStream_t s) {
    const int n = a.C / kEl<T, VEC>;
    a.gshift = 0;
    while (a.gshift < 5 && (1 << a.gshift) < n) ++a.gshift;
    if (a.few) {
        blocks = (int)((a.N + a.few - 1) / a.few);
        note_launch(SGA_KERN_EMBED_BWD, s, false);
        const int64_t per = a.few;
        const size_t bytes = (size_t)per * a.C * sizeof(T);
        cudaError_t le;
        constexpr int kShared = 16;
        if (bytes <= kStage && aligned(a.dOut, 16)) {
            auto launch = [&]<bool SHARED>() {
                if (cudaError_t e = allow_smem<embed_grad_few_kernel<T, VEC, true, SHARED>>(kStage); e != cudaSuccess) return e;
                return launch_early(embed_grad_few_kernel<T, VEC, true, SHARED>, dim3((unsigned)blocks), dim3(kSortThreads), bytes, s, a, per);
            };
            le = a.V <= kShared ? launch.template operator()<true>() : launch.template operator()<false>();
        } else {
            const int64_t rounds = (n + (VEC ? 31 : 127)) / (VEC ? 32 : 128);
            const dim3 grid((unsigned)blocks, (unsigned)std::max<int64_t>(1, std::min<int64_t>(rounds, device_sms() / blocks)));
            le = launch_early(a.V <= kShared ? embed_grad_few_kernel<T, VEC, false, true> : embed_grad_few_kernel<T, VEC, false, false>, grid,
                              dim3(kSortThreads), 0, s, a, per);
        }
        note_launch(SGA_KERN_EMBED_BWD, s, true);
        if (le != cudaSuccess) return le;
        const int64_t items = a.V * a.C / (a.C % 4 == 0 ? 4 : 1);
        note_launch(SGA_KERN_EMBED_ADD, s, false);
        cudaError_t e;
        if (blocks <= 16)
            e = launch_early(a.C % 4 == 0 ? embed_add_fewer_kernel<T, 4> : embed_add_fewer_kernel<T, 1>,
                             dim3((unsigned)((items + 255) / 256)), dim3(256), 0, s, a, blocks);
        else
            e = launch_early(a.C % 4 == 0 ? embed_add_few_kernel<T, 4> : embed_add_few_kernel<T, 1>, dim3((unsigned)((items + 7) / 8)),
                             dim3(256), 0, s, a, blocks);
        note_launch(SGA_KERN_EMBED_ADD, s, true);
        return e;
    }
    void *args[] = {&a};
    note_launch(SGA_KERN_EMBED_BWD, s, false);
    (void)cudaLaunchCooperativeKernel(reinterpret_cast<const void *>(embed_grad_kernel<T, VEC>), dim3(blocks),
                                      dim3(kSortThreads), args, 0, s);
    note_launch(SGA_KERN_EMBED_BWD, s, true);
    return cudaGetLastError();
}

sga_status check_embed(int64_t N, int64_t V, int64_t C, sga_dtype dt, int id_bytes) {
    if (N < 0 || V < 0 || C < 1 || (id_bytes != 4 && id_bytes != 8)) return SGA_EINVAL;
    if (dt != SGA_F32 && dt != SGA_BF16) return SGA_EUNSUPPORTED;
    if (N >= INT32_MAX || V >= INT32_MAX || C > (1 << 20)) return SGA_EUNSUPPORTED;
    return SGA_OK;
}
size_t size_of(sga_dtype dt) { return dt == SGA_F32 ? 4 : 2; }

template <typename T, bool VEC>
cudaError_t fwd_t(const void *ids, bool wide, const void *table, int64_t N, int64_t V, int C, float scale, void *out,
                  cudaStream_t s) {
    const int n = C / kEl<T, VEC>;
    int sh = 0;
    while (sh < 5 && (4 << sh) < n) ++sh;   // four groups a lane
    const int64_t blocks = ((N << sh) + 255) / 256;
    const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)device_sms() * 32);
    const int64_t rounds = (n + (4 << sh) - 1) / (4 << sh);   // of a lane over its row
    const unsigned slabs = (unsigned)std::max<int64_t>(1, std::min<int64_t>(rounds, device_sms() * 4 / (int64_t)grid));
    note_launch(SGA_KERN_EMBED_FWD, s, false);
    const cudaError_t e = launch_early(embed_fwd_kernel<T, VEC>, dim3(grid, slabs), dim3(256), 0, s, ids, wide,
                                       static_cast<const T *>(table), N, V, C, scale, sh, static_cast<T *>(out));
    note_launch(SGA_KERN_EMBED_FWD, s, true);
    return e;
}

}  // namespace
}  // namespace sga

using namespace sga;

extern "C" {

sga_status embed_fwd(const void *ids, int id_bytes, const void *table, int64_t N, int64_t V, int64_t C, float scale,
                     sga_dtype dt, void *out, void *stream) {
    sga_status st = check_embed(N, V, C, dt, id_bytes);
    if (st != SGA_OK) return st;
    if (N == 0) return SGA_OK;
    const size_t e = size_of(dt);
    if (!ids || !aligned(ids, id_bytes) || (V > 0 && !table) || !aligned(table, e) || !out || !aligned(out, e))
        return SGA_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = (C * e) % 16 == 0 && aligned(table, 16) && aligned(out, 16), wide = id_bytes == 8;
    if (dt == SGA_F32)
        return status_of(vec ? fwd_t<float, true>(ids, wide, table, N, V, (int)C, scale, out, s)
                             : fwd_t<float, false>(ids, wide, table, N, V, (int)C, scale, out, s));
    return status_of(vec ? fwd_t<__nv_bfloat16, true>(ids, wide, table, N, V, (int)C, scale, out, s)
                         : fwd_t<__nv_bfloat16, false>(ids, wide, table, N, V, (int)C, scale, out, s));
}

size_t sga_embed_bwd_workspace_bytes(int64_t N, int64_t V, int64_t C) {
    return N <= 0 || V < 0 || C <= 0 || N >= INT32_MAX ? 0 : layout(N, V, C, device_sms()).bytes;
}

sga_status embed_bwd(const void *ids, int id_bytes, const void *dOut, int64_t N, int64_t V, int64_t C, float scale,
                     int64_t padding_idx, sga_dtype dt, void *dTable, void *workspace, size_t workspace_bytes,
                     void *stream) {
    sga_status st = check_embed(N, V, C, dt, id_bytes);
    if (st != SGA_OK) return st;
    const size_t e = size_of(dt);
    if (V > 0 && (!dTable || !aligned(dTable, e))) return SGA_EINVAL;
    if (N > 0 && (!ids || !aligned(ids, id_bytes) || !dOut || !aligned(dOut, e))) return SGA_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) return status_of(V > 0 ? cudaMemsetAsync(dTable, 0, (size_t)V * C * e, s) : cudaSuccess);
    const int sms = device_sms();
    const Layout l = layout(N, V, C, sms);
    if (!workspace || !aligned(workspace, 256)) return SGA_EINVAL;
    if (workspace_bytes < l.bytes) return SGA_EWORKSPACE;
    char *ws = static_cast<char *>(workspace);
    GradArgs a{};
    a.ids = ids;
    a.wide = id_bytes == 8;
    a.dOut = dOut;
    a.dTable = dTable;
    for (int i = 0; i < 2; ++i) {
        a.key[i] = reinterpret_cast<int32_t *>(ws + l.key[i]);
        a.tok[i] = reinterpret_cast<int32_t *>(ws + l.tok[i]);
    }
    a.hist = reinterpret_cast<int32_t *>(ws + l.hist);
    a.part = reinterpret_cast<float *>(ws + l.part);
    a.N = N;
    a.V = V;
    a.C = (int)C;
    a.L = chunk_len(N, sms);
    a.chunks = (N + a.L - 1) / a.L;
    a.padding = padding_idx;
    a.few = few_tokens(N, V, sms);
    a.scale = scale;
    const int bits = bits_of(V);
    a.passes = (bits + 7) / 8;
    a.bits = (bits + a.passes - 1) / a.passes;
    const bool vec = (C * e) % 16 == 0 && aligned(dOut, 16) && aligned(dTable, 16);
    const int blocks = grad_blocks(N, V, C, sms);
    if (dt == SGA_F32) return status_of(vec ? grad_t<float, true>(a, blocks, s) : grad_t<float, false>(a, blocks, s));
    return status_of(vec ? grad_t<__nv_bfloat16, true>(a, blocks, s) : grad_t<__nv_bfloat16, false>(a, blocks, s));
}

sga_status sga_embed_read_device_error(void *stream, int32_t *code) {
    if (!code) return SGA_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    void *p = nullptr;
    int32_t v = 0;
    cudaError_t e = cudaGetSymbolAddress(&p, g_embed_err);
    if (e == cudaSuccess) e = cudaMemcpyAsync(&v, p, sizeof v, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = cudaMemsetAsync(p, 0, sizeof v, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return status_of(e);
    *code = v;
    return v ? SGA_EDEVICE_CHECK : SGA_OK;
}

}  // extern "C"
