// Plans of packed-sequence attention (host side) and its C entry points.
#include <algorithm>
#include <new>
#include <vector>

#include "seq.h"

namespace sga {

void set_cuda_error(cudaError_t e);   // (api.cu)

namespace {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

sga_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return SGA_OK;
    set_cuda_error(e);
    return SGA_ECUDA;
}

bool supported(int64_t B, int H, int Hkv, int D, sga_dtype dt) {
    return (dt == SGA_F32 || dt == SGA_BF16) && (D == 32 || D == 64 || D == 128) && H >= 1 && Hkv >= 1 &&
           H % Hkv == 0 && (int64_t)H * D <= 16384 && B < INT32_MAX;
}

// (s, e) of every packed row: binary search of the sequence that holds it.
__global__ void range_kernel(const int32_t *__restrict__ ptr, int64_t B, int64_t rows, int2 *__restrict__ range) {
    const int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (r >= rows) return;
    int64_t lo = 0, hi = B;   // ptr[lo] <= r < ptr[hi]
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (__ldg(ptr + mid) <= r) lo = mid;
        else hi = mid;
    }
    range[r] = make_int2(__ldg(ptr + lo), __ldg(ptr + lo + 1));
}

// What the tiles of a batch see: its sequences and the plan's mask.
struct Mask {
    const std::vector<int32_t> &ptr;
    int64_t rows;
    int TR;
    bool causal;
    int64_t window, sinks;   // window 0: none
};

void longest_first(std::vector<SeqTile> &all) {
    std::stable_sort(all.begin(), all.end(), [](const SeqTile &a, const SeqTile &b) {
        return (a.t1 - a.t0) + (a.g1 - a.g0) > (b.t1 - b.t0) + (b.g1 - b.g0);
    });
}

// The tile lists, sorted by the number of tiles, longest first (ties in row
// order), so that the last blocks to start are the short ones.
//
// Tiles of queries and the key tiles they see.
std::vector<SeqTile> query_tiles(const Mask &m) {
    const int64_t n = (m.rows + m.TR - 1) / m.TR, TR = m.TR;
    std::vector<SeqTile> all(n);
    size_t s = 0;   // sequence of the tile's first row
    for (int64_t i = 0; i < n; ++i) {
        const int64_t r0 = i * TR, r1 = std::min(m.rows, r0 + TR) - 1;   // first and last row
        while (m.ptr[s + 1] <= r0) ++s;
        size_t z = s;
        while (m.ptr[z + 1] <= r1) ++z;
        const int64_t s0 = m.ptr[s], e0 = m.ptr[s + 1], s1 = m.ptr[z], e1 = m.ptr[z + 1];
        // intervals of the first and the last row: both ends grow with the row
        int64_t lo0 = s0, lo1 = s1, hi0 = m.causal ? r0 + 1 : e0, hi1 = m.causal ? r1 + 1 : e1;
        SeqTile t{};
        if (m.window) {
            lo0 = std::max(s0, r0 - m.window + 1);
            lo1 = std::max(s1, r1 - m.window + 1);
            hi0 = std::min(hi0, r0 + m.window);
            hi1 = std::min(hi1, r1 + m.window);
            // the sinks of the first row's sequence lie before its window, or touch
            // it; those of a sequence that begins in the tile lie in what its rows
            // see, or reach past it (the tile's last such sequence's the farthest)
            const int64_t b0 = std::min(s0 + m.sinks, m.causal ? std::min(hi1, e0) : e0), b1 = std::min(s1 + m.sinks, m.causal ? hi1 : e1);
            hi1 = std::max(hi1, std::max(b0, b1));
            if (b0 > s0 && (b0 + TR - 1) / TR >= lo0 / TR) {
                lo0 = s0;
            } else if (b0 > s0) {
                t.g0 = (int32_t)(s0 / TR);
                t.g1 = (int32_t)((b0 + TR - 1) / TR);
            }
        }
        t.tile = (int32_t)i;
        t.t0 = (int32_t)(lo0 / TR);
        t.t1 = (int32_t)((hi1 + TR - 1) / TR);
        t.f0 = (int32_t)((lo1 + TR - 1) / TR);
        t.f1 = (int32_t)(hi0 / TR);
        if (t.f1 <= t.f0) t.f0 = t.f1 = t.t0;
        all[i] = t;
    }
    longest_first(all);
    return all;
}

// Tiles of keys and the query tiles that see them.
std::vector<SeqTile> key_tiles(const Mask &m) {
    const int64_t n = (m.rows + m.TR - 1) / m.TR, TR = m.TR;
    std::vector<SeqTile> all(n);
    size_t s = 0;
    for (int64_t i = 0; i < n; ++i) {
        const int64_t r0 = i * TR, r1 = std::min(m.rows, r0 + TR) - 1;
        while (m.ptr[s + 1] <= r0) ++s;
        size_t z = s;
        while (m.ptr[z + 1] <= r1) ++z;
        // the least and the greatest of the rows' interval ends; the beginnings grow with the row
        const int64_t s0 = m.ptr[s], s1 = m.ptr[z];
        int64_t lo0 = m.causal ? r0 : s0, lo1 = m.causal ? r1 : s1, hi0 = m.ptr[s + 1], hi1 = m.ptr[z + 1];
        if (m.window) {
            if (r0 - s0 >= m.sinks) lo0 = std::max(lo0, r0 - m.window + 1);
            if (r1 - s1 >= m.sinks) lo1 = std::max(lo1, r1 - m.window + 1);
            hi0 = INT64_MAX;
            hi1 = 0;
            for (size_t q = s; q <= z; ++q) {   // the tile's share [a, b) of each sequence
                const int64_t b = m.ptr[q + 1], a = std::max<int64_t>(m.ptr[q], r0), e = std::min(b, r1 + 1), far = m.ptr[q] + m.sinks;
                if (a >= e) continue;
                if (a < far) {
                    hi0 = std::min(hi0, b);
                    hi1 = std::max(hi1, b);
                }
                if (e > far) {   // (rows max(a, far) .. e - 1 are no sinks)
                    hi0 = std::min(hi0, std::min(b, std::max(a, far) + m.window));
                    hi1 = std::max(hi1, std::min(b, e - 1 + m.window));
                }
            }
        }
        SeqTile t{};
        t.tile = (int32_t)i;
        t.t0 = (int32_t)(lo0 / TR);
        t.t1 = (int32_t)((hi1 + TR - 1) / TR);
        t.f0 = (int32_t)((lo1 + TR - 1) / TR);
        t.f1 = (int32_t)(hi0 / TR);
        if (t.f1 <= t.f0) t.f0 = t.f1 = t.t0;
        all[i] = t;
    }
    longest_first(all);
    return all;
}

// Cuts the walks of key tiles that are twice as long as a window's or more (the sinks'
// of long sequences, which one block would walk alone while the others are long done)
// into parts of about a window's length, or of an eighth of an SM's share of all walks,
// where that is more: fewer parts are fewer sums to join.  3428 rows of four sequences,
// 4/2 heads of 32, fp32, window 129, a sink: backward 128 us with parts of 16 tiles at
// least, 72 without the sink.
std::vector<SeqJoin> cut_walks(const Mask &m, std::vector<SeqTile> &keys, int64_t sm_heads, int &n_parts) {
    std::vector<SeqJoin> joins;
    n_parts = 0;
    if (!m.window) return joins;
    int64_t all = 0;
    for (const SeqTile &t : keys) all += t.t1 - t.t0;
    const int64_t span = (m.window + m.TR - 1) / m.TR * (m.causal ? 1 : 2) + 1, most = std::max(span, all / (8 * std::max<int64_t>(1, sm_heads)));
    std::vector<SeqTile> out;
    for (const SeqTile &t : keys) {
        const int64_t n = t.t1 - t.t0;
        if (n < 2 * most) {
            out.push_back(t);
            continue;
        }
        const int64_t k = (n + most - 1) / most;
        joins.push_back({t.tile, t.t0, t.t1, n_parts + 1, (int32_t)k});
        for (int64_t i = 0; i < k; ++i) {
            SeqTile c = t;
            c.t0 = (int32_t)(t.t0 + n * i / k);
            c.t1 = (int32_t)(t.t0 + n * (i + 1) / k);
            c.part = ++n_parts;
            out.push_back(c);
        }
    }
    keys = std::move(out);
    longest_first(keys);
    return joins;
}

// Neighbouring tiles by twos, by the key tiles that a pair walks; a missing
// second tile lies past the rows and sees nothing.
std::vector<SeqTile> pair_list(std::vector<SeqTile> all) {
    std::sort(all.begin(), all.end(), [](const SeqTile &a, const SeqTile &b) { return a.tile < b.tile; });
    if (all.size() % 2) {
        SeqTile t = all.back();
        ++t.tile;
        t.t1 = t.f0 = t.f1 = t.t0;
        t.g0 = t.g1 = 0;
        all.push_back(t);
    }
    std::vector<int32_t> order(all.size() / 2);
    for (size_t i = 0; i < order.size(); ++i) order[i] = (int32_t)i;
    auto cost = [&](int32_t i) {
        return std::max(all[2 * i].t1, all[2 * i + 1].t1) - std::min(all[2 * i].t0, all[2 * i + 1].t0) +
               std::max(all[2 * i].g1 - all[2 * i].g0, all[2 * i + 1].g1 - all[2 * i + 1].g0);
    };
    std::stable_sort(order.begin(), order.end(), [&](int32_t a, int32_t b) { return cost(a) > cost(b); });
    std::vector<SeqTile> out;
    out.reserve(all.size());
    for (int32_t i : order) {
        out.push_back(all[2 * i]);
        out.push_back(all[2 * i + 1]);
    }
    return out;
}

void seq_free(sga_seq_plan *p) {
    free_device(p->d_qpairs);
    free_device(p->d_range);
    free_device(p->d_qtiles);
    free_device(p->d_ktiles);
    free_device(p->d_joins);
    free_device(p->d_err);
}

template <typename P> cudaError_t dev_alloc(sga_seq_plan *p, P **out, size_t count) {
    const size_t bytes = std::max<size_t>(count, 1) * sizeof(P);
    cudaError_t e = cudaMalloc(reinterpret_cast<void **>(out), bytes);
    if (e == cudaSuccess) p->device_bytes += (int64_t)bytes;
    return e;
}

cudaError_t seq_build(sga_seq_plan *p, const std::vector<int32_t> &ptr, const int32_t *d_ptr, cudaStream_t s) {
    const Mask mask{ptr, p->rows, p->tile_rows, p->causal != 0, p->window, p->sinks};
    const std::vector<SeqTile> q = query_tiles(mask);
    std::vector<SeqTile> k = key_tiles(mask);
    const std::vector<SeqJoin> joins = cut_walks(mask, k, p->num_sms / p->Hkv, p->n_parts);
    const bool pairs = p->dt == SGA_BF16 && p->H / p->Hkv % 2 != 0;
    const std::vector<SeqTile> qp = pairs ? pair_list(q) : std::vector<SeqTile>();
    p->n_tiles = (int)q.size();
    p->n_ktiles = (int)k.size();
    p->n_joins = (int)joins.size();
    cudaError_t e = dev_alloc(p, &p->d_range, (size_t)p->rows);
    if (e == cudaSuccess) e = dev_alloc(p, &p->d_qtiles, q.size());
    if (e == cudaSuccess) e = dev_alloc(p, &p->d_ktiles, k.size());
    if (e == cudaSuccess && pairs) e = dev_alloc(p, &p->d_qpairs, qp.size());
    if (e == cudaSuccess && !joins.empty()) e = dev_alloc(p, &p->d_joins, joins.size());
    if (e == cudaSuccess) e = dev_alloc(p, &p->d_err, 1);
    if (e == cudaSuccess) e = cudaMemsetAsync(p->d_err, 0, sizeof(int32_t), s);
    if (e == cudaSuccess && p->rows > 0) {
        range_kernel<<<(unsigned)((p->rows + 255) / 256), 256, 0, s>>>(d_ptr, p->B, p->rows, p->d_range);
        e = cudaGetLastError();
        if (e == cudaSuccess)
            e = cudaMemcpyAsync(p->d_qtiles, q.data(), q.size() * sizeof(SeqTile), cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess && pairs)
            e = cudaMemcpyAsync(p->d_qpairs, qp.data(), qp.size() * sizeof(SeqTile), cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess)
            e = cudaMemcpyAsync(p->d_ktiles, k.data(), k.size() * sizeof(SeqTile), cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess && !joins.empty())
            e = cudaMemcpyAsync(p->d_joins, joins.data(), joins.size() * sizeof(SeqJoin), cudaMemcpyHostToDevice, s);
    }
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return e;
}

sga_status check_seq(const sga_seq_plan *p, int64_t T, float scale, std::initializer_list<const void *> ps) {
    if (!p) return SGA_EINVAL;
    if (T < p->rows) return SGA_EINVAL;
    if (!(scale > 0.f) || !(scale * kLog2e < INFINITY)) return SGA_EINVAL;   // (scores are held in units of log2)
    if (p->rows == 0) return SGA_OK;
    for (const void *q : ps)
        if (!q || !aligned(q, 16)) return SGA_EINVAL;
    return SGA_OK;
}

SeqArgs seq_args(const sga_seq_plan *p, float scale) {
    SeqArgs a{};
    a.range = p->d_range;
    a.qtiles = p->d_qtiles;
    a.ktiles = p->d_ktiles;
    a.qpairs = p->d_qpairs;
    a.rows = p->rows;
    a.rows_pad = seq_rows_pad(p->rows);
    a.H = p->H;
    a.Hkv = p->Hkv;
    a.causal = p->causal;
    a.n_tiles = p->n_tiles;
    a.n_ktiles = p->n_ktiles;
    a.joins = p->d_joins;
    a.n_joins = p->n_joins;
    a.window = p->window;
    a.sinks = p->sinks;
    a.num_sms = p->num_sms;
    a.scale = scale;
    a.d_err = p->d_err;
    return a;
}

// -lse and -Delta (a multiple of 512 bytes)
size_t terms_bytes(const sga_seq_plan *p) { return (size_t)2 * p->H * (size_t)seq_rows_pad(p->rows) * sizeof(float); }

// The call's device must be the plan's (its memory and the tensors' live
// there).  Setting it binds the device's context to a thread that has made no
// runtime call yet (an autograd worker): the tensor-map encoder needs one.
sga_status on_device(const sga_seq_plan *p) {
    static thread_local int bound = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev != p->device) return SGA_EINVAL;
    if (e == cudaSuccess && bound != dev && (e = cudaSetDevice(dev)) == cudaSuccess) bound = dev;
    return status_of(e);
}

}  // namespace
}  // namespace sga

using namespace sga;

extern "C" {

sga_status sga_seq_plan_create(const int32_t *seq_ptr, int64_t B, int H, int Hkv, int D, sga_dtype dt, int causal,
                               void *stream, sga_seq_plan **out) {
    return sga_seq_plan_create_windowed(seq_ptr, B, H, Hkv, D, dt, causal, 0, 0, stream, out);
}

sga_status sga_seq_plan_create_windowed(const int32_t *seq_ptr, int64_t B, int H, int Hkv, int D, sga_dtype dt, int causal,
                                        int64_t window, int64_t sinks, void *stream, sga_seq_plan **out) {
    if (!out) return SGA_EINVAL;
    *out = nullptr;
    if (!seq_ptr || !aligned(seq_ptr, 4) || B < 0) return SGA_EINVAL;
    if (causal != 0 && causal != 1) return SGA_EINVAL;
    if (window < 0 || sinks < 0 || (sinks > 0 && window == 0)) return SGA_EINVAL;
    if (!supported(B, H, Hkv, D, dt)) return SGA_EUNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    sga_seq_plan *p = nullptr;
    try {
        std::vector<int32_t> ptr((size_t)B + 1);
        cudaError_t e = cudaMemcpyAsync(ptr.data(), seq_ptr, ptr.size() * sizeof(int32_t), cudaMemcpyDeviceToHost, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
        if (e != cudaSuccess) return status_of(e);
        if (ptr[0] != 0) return SGA_EINVAL;
        for (int64_t i = 0; i < B; ++i)
            if (ptr[i + 1] < ptr[i]) return SGA_EINVAL;
        // the row index of a tile's end stays an int32
        if (ptr[B] > INT32_MAX - 256) return SGA_EUNSUPPORTED;
        p = new sga_seq_plan();
        p->B = B;
        p->rows = ptr[B];
        p->H = H;
        p->Hkv = Hkv;
        p->D = D;
        p->dt = dt;
        p->causal = causal;
        p->tile_rows = dt == SGA_BF16 ? 128 : 64;
        int32_t longest = 0;
        for (int64_t i = 0; i < B; ++i) longest = std::max(longest, ptr[i + 1] - ptr[i]);
        if (window > 0 && std::max(window, sinks) < longest) {   // (otherwise every pair of a sequence is near, or its key a sink)
            p->window = (int)window;
            p->sinks = (int)sinks;
        }
        e = cudaGetDevice(&p->device);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&p->num_sms, cudaDevAttrMultiProcessorCount, p->device);
        if (e == cudaSuccess) e = seq_build(p, ptr, seq_ptr, s);
        if (e != cudaSuccess) {
            seq_free(p);
            delete p;
            return status_of(e);
        }
    } catch (const std::bad_alloc &) {   // host memory
        if (p) {
            seq_free(p);
            delete p;
        }
        return SGA_EINVAL;
    }
    *out = p;
    return SGA_OK;
}

void sga_seq_plan_destroy(sga_seq_plan *p) {
    if (!p) return;
    seq_free(p);
    delete p;
}

int64_t sga_seq_plan_rows(const sga_seq_plan *p) { return p ? p->rows : 0; }

size_t sga_seq_bwd_workspace_bytes(const sga_seq_plan *p) {
    return p ? terms_bytes(p) + (size_t)p->n_parts * p->Hkv * 2 * p->tile_rows * p->D * sizeof(float) : 0;
}

sga_status sga_seq_read_device_error(const sga_seq_plan *p, void *stream, int32_t *code) {
    if (!p || !code) return SGA_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int32_t v = 0;
    cudaError_t e = cudaMemcpyAsync(&v, p->d_err, sizeof(int32_t), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = cudaMemsetAsync(p->d_err, 0, sizeof(int32_t), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return status_of(e);
    *code = v;
    return v ? SGA_EDEVICE_CHECK : SGA_OK;
}

sga_status seq_attn_fwd(const sga_seq_plan *p, const void *Q, const void *K, const void *V, int64_t T, float scale,
                        void *out, float *lse, void *stream) {
    sga_status st = check_seq(p, T, scale, {Q, K, V, out, lse});
    if (st != SGA_OK) return st;
    if (p->rows == 0) return SGA_OK;
    if ((st = on_device(p)) != SGA_OK) return st;
    SeqArgs a = seq_args(p, scale);
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.out_w = out;
    a.lse_w = lse;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->window) return status_of(p->dt == SGA_F32 ? seq_fwd_f32<true>(a, p->D, s) : seq_fwd_bf16<true>(a, p->D, s));
    return status_of(p->dt == SGA_F32 ? seq_fwd_f32<false>(a, p->D, s) : seq_fwd_bf16<false>(a, p->D, s));
}

sga_status seq_attn_bwd(const sga_seq_plan *p, const void *Q, const void *K, const void *V, const void *out,
                        const float *lse, const void *dOut, int64_t T, float scale, void *dQ, void *dK, void *dV,
                        void *workspace, size_t workspace_bytes, void *stream) {
    sga_status st = check_seq(p, T, scale, {Q, K, V, out, lse, dOut, dQ, dK, dV});
    if (st != SGA_OK) return st;
    if (p->rows == 0) return SGA_OK;
    if (!workspace || !aligned(workspace, 256)) return SGA_EINVAL;
    if (workspace_bytes < sga_seq_bwd_workspace_bytes(p)) return SGA_EWORKSPACE;
    if ((st = on_device(p)) != SGA_OK) return st;
    SeqArgs a = seq_args(p, scale);
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.out = out;
    a.lse = lse;
    a.dOut = dOut;
    a.dQ = dQ;
    a.dK = dK;
    a.dV = dV;
    a.ws_nlse = static_cast<float *>(workspace);
    a.ws_ndelta = a.ws_nlse + (size_t)p->H * a.rows_pad;
    a.ws_part = reinterpret_cast<float *>(static_cast<char *>(workspace) + terms_bytes(p));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->window) return status_of(p->dt == SGA_F32 ? seq_bwd_f32<true>(a, p->D, s) : seq_bwd_bf16<true>(a, p->D, s));
    return status_of(p->dt == SGA_F32 ? seq_bwd_f32<false>(a, p->D, s) : seq_bwd_bf16<false>(a, p->D, s));
}

}  // extern "C"
