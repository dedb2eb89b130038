// Embedding lookup with scaling, and its gradient by sorted tokens.
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

#include "common.cuh"
#include "plan.h"

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

int sm_count() {
    int dev = 0, n = 1;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

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
// lane's row are loaded before any is stored.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const void *__restrict__ ids, bool wide, const T *__restrict__ table,
                                                        int64_t N, int64_t V, int C, float scale, int sh, T *out) {
    constexpr int EL = kEl<T, VEC>, U = 4;
    const int n = C / EL, lanes = 1 << sh, sub = threadIdx.x & (lanes - 1);
    const int64_t step = ((int64_t)gridDim.x * blockDim.x) >> sh;
    for (int64_t t = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> sh; t < N; t += step) {
        const int64_t id = id_at(ids, t, wide);
        const bool ok = id >= 0 && id < V;
        if (!ok && sub == 0) atomicOr(&g_embed_err, kErrIndexRange);
        const T *src = table + (ok ? id : 0) * C;
        T *dst = out + t * C;
        for (int c0 = sub; c0 < n; c0 += U * lanes) {
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

// Sort key of a token: its id, or V (last, never summed) for the padding id
// and for an id outside the table.
__global__ void embed_keys_kernel(const void *__restrict__ ids, bool wide, int64_t N, int64_t V, int64_t padding,
                                  int32_t *__restrict__ key, int32_t *__restrict__ val) {
    for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < N; t += (int64_t)gridDim.x * blockDim.x) {
        int64_t id = id_at(ids, t, wide);
        if (id < 0 || id >= V) {
            atomicOr(&g_embed_err, kErrIndexRange);
            id = V;
        }
        if (id == padding) id = V;
        key[t] = (int32_t)id;
        val[t] = (int32_t)t;
    }
}

struct SumArgs {
    const int32_t *key, *tok;   // sorted
    const void *dOut;
    void *dTable;
    float *part;                // [chunks][2][C]: the row that runs on from the chunk before, the row that runs on
    int64_t N, V, chunks;
    int L, C;
    float scale;
};

// A warp per (chunk of L sorted tokens, slab of 32 * U groups of columns).
template <typename T, bool VEC, int U> __global__ void __launch_bounds__(256) embed_sum_kernel(const SumArgs a, int slabs) {
    constexpr int EL = kEl<T, VEC>;
    const int64_t w = (((int64_t)blockIdx.x * 256) + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int64_t chunk = w / slabs;
    if (chunk >= a.chunks) return;
    const int g0 = (int)(w % slabs) * 32 * U + lane, n = a.C / EL;
    const T *dOut = static_cast<const T *>(a.dOut);
    T *dTable = static_cast<T *>(a.dTable);
    const int64_t k0 = chunk * a.L, k1 = min(a.N, k0 + a.L);
    float acc[U][EL];
    int32_t cur = __ldg(a.key + k0);
    // the first run continues one of the chunk before
    bool joined = k0 > 0 && __ldg(a.key + k0 - 1) == cur;
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
                if (g0 + 32 * u < n)
#pragma unroll
                    for (int i = 0; i < EL; ++i) p[(g0 + 32 * u) * EL + i] = acc[u][i];
        } else {
            T *o = dTable + (int64_t)cur * a.C;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (g0 + 32 * u < n) {
#pragma unroll
                    for (int i = 0; i < EL; ++i) acc[u][i] *= a.scale;
                    store_g<T, VEC>(o + (int64_t)(g0 + 32 * u) * EL, acc[u]);
                }
        }
    };
    clear();
    for (int64_t kb = k0; kb < k1; kb += 32) {
        const int m = (int)min((int64_t)32, k1 - kb);
        const int32_t key = lane < m ? __ldg(a.key + kb + lane) : 0, tok = lane < m ? __ldg(a.tok + kb + lane) : 0;
        for (int q = 0; q < m; q += 4) {
            float x[4][U][EL];
            int32_t kk[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                kk[z] = __shfl_sync(SGA_FULL_MASK, key, (q + z) & 31);
                const int64_t t = __shfl_sync(SGA_FULL_MASK, tok, (q + z) & 31);
                const bool on = q + z < m && kk[z] < a.V;
#pragma unroll
                for (int u = 0; u < U; ++u) {
#pragma unroll
                    for (int i = 0; i < EL; ++i) x[z][u][i] = 0.f;
                    if (on && g0 + 32 * u < n) load_g<T, VEC>(dOut + t * a.C + (int64_t)(g0 + 32 * u) * EL, x[z][u]);
                }
            }
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                if (q + z >= m) break;
                if (kk[z] != cur) {
                    flush(false);
                    clear();
                    cur = kk[z];
                    joined = false;
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < EL; ++i) acc[u][i] += x[z][u][i];
            }
        }
    }
    flush(k1 < a.N && __ldg(a.key + k1) == cur);
}

// A block per chunk whose last row runs on into the next chunk, and 32 columns:
// the row's partials in chunk order, eight warps over a contiguous eighth each.
template <typename T> __global__ void __launch_bounds__(256) embed_join_kernel(const SumArgs a) {
    __shared__ float sm[8][32];
    const int64_t c0 = blockIdx.x;
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int64_t kl = (c0 + 1) * a.L - 1;   // the chunk's last token
    if (kl + 1 >= a.N) return;
    const int32_t cur = __ldg(a.key + kl);
    if (cur >= a.V || __ldg(a.key + kl + 1) != cur) return;
    if (c0 > 0 && __ldg(a.key + c0 * a.L - 1) == cur) return;   // the row began in an earlier chunk
    // one past the row's last token
    int64_t lo = kl + 1, hi = a.N;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (__ldg(a.key + mid) == cur) lo = mid + 1;
        else hi = mid;
    }
    const int64_t cl = (lo - 1) / a.L;       // the row's last chunk
    const int64_t n = cl - c0, per = (n + 7) / 8;
    const int col = blockIdx.y * 32 + lane;
    float s = 0.f;
    if (col < a.C) {
        const int64_t b = c0 + 1 + wp * per, e = min(cl + 1, b + per);
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (wp == 0) v[0] = a.part[(c0 * 2 + 1) * a.C + col];
        int64_t c = b;
        for (; c + 4 <= e; c += 4)
#pragma unroll
            for (int z = 0; z < 4; ++z) v[z] += a.part[(c + z) * 2 * a.C + col];
        for (; c < e; ++c) v[0] += a.part[c * 2 * a.C + col];
        s = (v[0] + v[1]) + (v[2] + v[3]);
    }
    sm[wp][lane] = s;
    __syncthreads();
    if (wp == 0 && col < a.C) {
        s = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += sm[q][lane];
        static_cast<T *>(a.dTable)[(int64_t)cur * a.C + col] = from_f32<T>(s * a.scale);
    }
}

// Sorted tokens of a chunk: an equal share of the resident warps, at least 16.
int chunk_len(int64_t N, int sms) {
    const int64_t per = (N + (int64_t)sms * 32 - 1) / ((int64_t)sms * 32);
    return (int)std::max<int64_t>(16, (per + 15) / 16 * 16);
}

int bits_of(int64_t v) {
    int b = 1;
    while ((v >> b) != 0) ++b;
    return b;
}

struct Layout {
    size_t key[2], val[2], hist, scan, part, total;
};
Layout layout(int64_t N, int64_t C, int sms) {
    Layout l{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += round256(bytes);
        return at;
    };
    for (int i = 0; i < 2; ++i) {
        l.key[i] = take((size_t)N * 4);
        l.val[i] = take((size_t)N * 4);
    }
    const int64_t h = radix_hist_elems(N);
    l.hist = take((size_t)h * 4);
    l.scan = take((size_t)scan_tmp_elems(h) * 4);
    const int L = chunk_len(N, sms);
    l.part = take((size_t)((N + L - 1) / L) * 2 * C * 4);
    l.total = off;
    return l;
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
    const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)sm_count() * 32);
    note_launch(SGA_KERN_EMBED_FWD, s, false);
    embed_fwd_kernel<T, VEC><<<grid, 256, 0, s>>>(ids, wide, static_cast<const T *>(table), N, V, C, scale, sh,
                                                  static_cast<T *>(out));
    note_launch(SGA_KERN_EMBED_FWD, s, true);
    return cudaGetLastError();
}

template <typename T, bool VEC> cudaError_t sum_t(const SumArgs &a, cudaStream_t s) {
    const int n = a.C / kEl<T, VEC>;
    const int U = n <= 32 ? 1 : 2;
    const int slabs = (n + 32 * U - 1) / (32 * U);
    const unsigned grid = (unsigned)((a.chunks * slabs + 7) / 8);
    note_launch(SGA_KERN_EMBED_SUM, s, false);
    if (U == 1) embed_sum_kernel<T, VEC, 1><<<grid, 256, 0, s>>>(a, slabs);
    else embed_sum_kernel<T, VEC, 2><<<grid, 256, 0, s>>>(a, slabs);
    note_launch(SGA_KERN_EMBED_SUM, s, true);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.chunks < 2) return e;
    note_launch(SGA_KERN_EMBED_JOIN, s, false);
    embed_join_kernel<T><<<dim3((unsigned)(a.chunks - 1), (unsigned)((a.C + 31) / 32)), 256, 0, s>>>(a);
    note_launch(SGA_KERN_EMBED_JOIN, s, true);
    return cudaGetLastError();
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

size_t sga_embed_bwd_workspace_bytes(int64_t N, int64_t C) {
    return N <= 0 || C <= 0 || N >= INT32_MAX ? 0 : layout(N, C, sm_count()).total;
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
    const int sms = sm_count();
    const Layout l = layout(std::max<int64_t>(N, 1), C, sms);
    if (N > 0) {
        if (!workspace || !aligned(workspace, 256)) return SGA_EINVAL;
        if (workspace_bytes < l.total) return SGA_EWORKSPACE;
    }
    // rows without a token
    cudaError_t ce = V > 0 ? cudaMemsetAsync(dTable, 0, (size_t)V * C * e, s) : cudaSuccess;
    if (ce != cudaSuccess || N == 0) return status_of(ce);
    auto at = [&](size_t off) { return reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + off); };
    int32_t *ka = at(l.key[0]), *kb = at(l.key[1]), *va = at(l.val[0]), *vb = at(l.val[1]);
    note_launch(SGA_KERN_EMBED_SORT, s, false);
    embed_keys_kernel<<<(unsigned)std::min<int64_t>((N + 255) / 256, sms * 8), 256, 0, s>>>(ids, id_bytes == 8, N, V,
                                                                                          padding_idx, ka, va);
    ce = cudaGetLastError();
    if (ce == cudaSuccess) ce = radix_sort_pairs(&ka, &va, &kb, &vb, N, bits_of(V), at(l.hist), at(l.scan), s);
    note_launch(SGA_KERN_EMBED_SORT, s, true);
    if (ce != cudaSuccess || V == 0) return status_of(ce);
    SumArgs a{};
    a.key = ka;
    a.tok = va;
    a.dOut = dOut;
    a.dTable = dTable;
    a.part = reinterpret_cast<float *>(at(l.part));
    a.N = N;
    a.V = V;
    a.C = (int)C;
    a.L = chunk_len(N, sms);
    a.chunks = (N + a.L - 1) / a.L;
    a.scale = scale;
    const bool vec = (C * e) % 16 == 0 && aligned(dOut, 16) && aligned(dTable, 16);
    if (dt == SGA_F32) return status_of(vec ? sum_t<float, true>(a, s) : sum_t<float, false>(a, s));
    return status_of(vec ? sum_t<__nv_bfloat16, true>(a, s) : sum_t<__nv_bfloat16, false>(a, s));
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
