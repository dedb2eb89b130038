// The gated feed-forward product, forward and backward: its entry points, the
// layout of operands that the tensor cores cannot read as they are, and the
// gradients of the two projections.  The products are in ff_gemm.cuh.
//
// Bound by the tensor cores: 4 T F M operations forward, 8 T F M backward.  The
// forward keeps G and U (rounded to the tensors' type), from which the backward
// forms dG and dU in one pass over memory: computing them again would be half a
// forward more.
#include "ff_gemm.cuh"

namespace sga {

void set_cuda_error(cudaError_t e);   // (api.cu)

namespace {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t round256(size_t b) { return (b + 255) & ~size_t(255); }
int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }

sga_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return SGA_OK;
    set_cuda_error(e);
    return SGA_ECUDA;
}

// Eight elements of a row as one bf16, or as the three that add up to each: every
// part is the rest's rounding to bf16, and the third holds what is left exactly (24
// bits, unless below 2^-133).  A value that bf16 would round to infinity is cut off
// instead; infinities and NaN stay in the first part alone.
template <bool F32> __device__ __forceinline__ void store_parts(__nv_bfloat16 *dst, int64_t part, const float *x) {
    if constexpr (!F32) {
        *reinterpret_cast<uint4 *>(dst) = pack<__nv_bfloat16>(x);
    } else {
        float h[8], m[8], l[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[i] = __bfloat162float(__float2bfloat16_rn(x[i]));
            const bool fine = fabsf(x[i]) < INFINITY;
            if (fine && !(fabsf(h[i]) < INFINITY)) h[i] = __uint_as_float(__float_as_uint(x[i]) & 0xffff0000u);
            const float r = fine ? x[i] - h[i] : 0.f;
            m[i] = __bfloat162float(__float2bfloat16_rn(r));
            l[i] = r - m[i];
        }
        *reinterpret_cast<uint4 *>(dst) = pack<__nv_bfloat16>(h);
        *reinterpret_cast<uint4 *>(dst + part) = pack<__nv_bfloat16>(m);
        *reinterpret_cast<uint4 *>(dst + 2 * part) = pack<__nv_bfloat16>(l);
    }
}

// Elements c .. c + 7 of a row of `cols` (zeros past its end).  VEC: whole 16 bytes.
// (The 16 bytes around elements that begin elsewhere, moved down in registers, took
// longer than one load an element: dG and dU of 4099 x 803 fp32 22 against 17 us.)
template <typename T, bool VEC> __device__ __forceinline__ void load8(const T *row, int64_t c, int64_t cols, float *x) {
    if constexpr (VEC) {
        constexpr int EL = Elt<T>::EL;
#pragma unroll
        for (int i = 0; i < 8; i += EL) {
            const uint4 v = c + i < cols ? *reinterpret_cast<const uint4 *>(row + c + i) : make_uint4(0, 0, 0, 0);
            unpack<T>(v, x + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = c + i < cols ? to_f32<T>(row[c + i]) : 0.f;
    }
}

// Up to three matrices into operands: rows of a multiple of 16 bytes, in parts.
struct FfLay {
    const void *src[3];
    FfMatrix dst[3];
    int64_t end[3];   // groups of eight elements of the matrices so far
    int n;
};
template <typename T, bool VEC> __global__ void __launch_bounds__(256) ff_lay_kernel(const __grid_constant__ FfLay a) {
    let_next_start();
    wait_previous();
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.end[a.n - 1]; i += step) {
        const int k = i < a.end[0] ? 0 : i < a.end[1] ? 1 : 2;
        const FfMatrix &m = a.dst[k];
        const int64_t at = k ? i - a.end[k - 1] : i, per = m.ld / 8, row = at / per, c = (at - row * per) * 8;
        float x[8];
        load8<T, VEC>(static_cast<const T *>(a.src[k]) + row * m.cols, c, m.cols, x);
        store_parts<sizeof(T) == 4>(const_cast<__nv_bfloat16 *>(m.p) + row * m.ld + c, m.part_elems(), x);
    }
}

// dG and dU as operands.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) ff_slopes_kernel(const T *G, const T *U, const T *dOut, int act, FfMatrix dg, FfMatrix du) {
    let_next_start();
    wait_previous();
    const int64_t per = dg.ld / 8, n = dg.rows * per, step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
        const int64_t row = i / per, c = (i - row * per) * 8, at = row * dg.cols;
        float g[8], u[8], d[8];
        load8<T, VEC>(G + at, c, dg.cols, g);
        load8<T, VEC>(U + at, c, dg.cols, u);
        load8<T, VEC>(dOut + at, c, dg.cols, d);
        ff_with_slope(act, [&](auto f) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float a, slope;
                f(g[k], a, slope);
                g[k] = d[k] * u[k] * slope;
                u[k] = d[k] * a;
            }
        });
        store_parts<sizeof(T) == 4>(const_cast<__nv_bfloat16 *>(dg.p) + row * dg.ld + c, dg.part_elems(), g);
        store_parts<sizeof(T) == 4>(const_cast<__nv_bfloat16 *>(du.p) + row * du.ld + c, du.part_elems(), u);
    }
}

// Where everything lies in the workspace; sizes depend on the shapes alone.
struct FfSpace {
    bool f32;
    int64_t T, F, M;
    size_t used = 0;
    char *base;
    size_t operand(int64_t rows, int64_t cols) {   // offset of a copied operand
        const size_t at = used;
        used += round256((size_t)rows * round8(cols) * 2 * (f32 ? 3 : 1));
        return at;
    }
    size_t bytes(size_t n) {
        const size_t at = used;
        used += round256(n);
        return at;
    }
    // the matrix as an operand: itself, or a copy noted in `lay`
    FfMatrix take(const void *src, int64_t rows, int64_t cols, FfLay *lay) {
        FfMatrix m;
        m.rows = rows;
        m.cols = cols;
        m.ld = round8(cols);
        if (!f32 && cols % 8 == 0) {
            m.p = static_cast<const __nv_bfloat16 *>(src);
            return m;
        }
        const size_t at = operand(rows, cols);
        if (lay) {
            m.p = reinterpret_cast<const __nv_bfloat16 *>(base + at);
            lay->src[lay->n] = src;
            lay->dst[lay->n] = m;
            lay->end[lay->n] = (lay->n ? lay->end[lay->n - 1] : 0) + rows * (m.ld / 8);
            ++lay->n;
        }
        return m;
    }
};

template <FfMode MODE> size_t partial_bytes(int64_t T, int64_t F, int64_t M, bool f32) {
    const FfPlan q = ff_plan<MODE>(T, F, M, f32);
    return q.split ? (size_t)2 * q.pairs * kTileFloats * sizeof(float) : 0;
}

cudaError_t lay_out(FfLay &a, bool f32, cudaStream_t s) {
    if (a.n == 0) return cudaSuccess;
    const int64_t groups = a.end[a.n - 1];
    bool vec = true;   // every source's rows are whole 16 bytes
    for (int i = 0; i < a.n; ++i) vec &= a.dst[i].cols % (f32 ? 4 : 8) == 0;
    for (int i = a.n; i < 3; ++i) a.end[i] = groups;
    const dim3 grid((unsigned)std::min<int64_t>((groups + 255) / 256, (int64_t)device_sms() * 32));
    note_launch(SGA_KERN_FF_LAY, s, false);
    const cudaError_t e = f32 ? launch_early(vec ? ff_lay_kernel<float, true> : ff_lay_kernel<float, false>, grid, dim3(256), 0, s, a)
                              : launch_early(ff_lay_kernel<__nv_bfloat16, false>, grid, dim3(256), 0, s, a);
    note_launch(SGA_KERN_FF_LAY, s, true);
    return e;
}

template <typename T> cudaError_t slopes(const void *G, const void *U, const void *dOut, int act, const FfMatrix &dg, const FfMatrix &du, cudaStream_t s) {
    const int64_t groups = dg.rows * (dg.ld / 8);
    const dim3 grid((unsigned)std::min<int64_t>((groups + 255) / 256, (int64_t)device_sms() * 32));
    const bool vec = dg.cols % Elt<T>::EL == 0;
    note_launch(SGA_KERN_FF_SLOPES, s, false);
    const cudaError_t e = launch_early(vec ? ff_slopes_kernel<T, true> : ff_slopes_kernel<T, false>, grid, dim3(256), 0, s, static_cast<const T *>(G),
                                       static_cast<const T *>(U), static_cast<const T *>(dOut), act, dg, du);
    note_launch(SGA_KERN_FF_SLOPES, s, true);
    return e;
}

sga_status check_ff(int64_t T, int64_t F, int64_t M, int act, sga_dtype dt) {
    if (T < 0 || F < 1 || M < 1) return SGA_EINVAL;
    if (act != SGA_ACT_SILU && act != SGA_ACT_GELU && act != SGA_ACT_RELU) return SGA_EINVAL;
    if (dt != SGA_F32 && dt != SGA_BF16) return SGA_EUNSUPPORTED;
    // coordinates and counts of tiles are 32 bits
    const int64_t most = INT32_MAX - 1024;
    if (T > most || F > (1 << 20) || M > (1 << 20)) return SGA_EUNSUPPORTED;
    if ((T / 256 + 1) * (std::max(F, M) / 128 + 1) > most || (F / 256 + 1) * (M / 128 + 2) > most) return SGA_EUNSUPPORTED;
    return SGA_OK;
}

// A thread that has made no runtime call yet (an autograd worker) has no context,
// which the tensor-map encoder needs: setting the device binds it.
cudaError_t bind_device() {
    static thread_local int bound = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && bound != dev && (e = cudaSetDevice(dev)) == cudaSuccess) bound = dev;
    return e;
}

}  // namespace
}  // namespace sga

using namespace sga;

extern "C" {

size_t sga_gated_ff_fwd_workspace_bytes(int64_t T, int64_t F, int64_t M, sga_dtype dt) {
    if (T <= 0 || check_ff(T, F, M, SGA_ACT_SILU, dt) != SGA_OK) return 0;
    FfSpace w{dt == SGA_F32, T, F, M};
    w.take(nullptr, T, F, nullptr);
    w.take(nullptr, F, M, nullptr);
    w.take(nullptr, F, M, nullptr);
    w.bytes(partial_bytes<FfMode::FWD>(T, F, M, w.f32));
    return w.used;
}

sga_status gated_ff_fwd(const void *X, const void *Wg, const void *Wu, int64_t T, int64_t F, int64_t M, int act, sga_dtype dt, void *out,
                        void *G, void *U, void *workspace, size_t workspace_bytes, void *stream) {
    sga_status st = check_ff(T, F, M, act, dt);
    if (st != SGA_OK) return st;
    if (T == 0) return SGA_OK;
    if (!G != !U) return SGA_EINVAL;
    for (const void *p : {X, Wg, Wu, static_cast<const void *>(out)})
        if (!p || !aligned(p, 16)) return SGA_EINVAL;
    if (!aligned(G, 16) || !aligned(U, 16)) return SGA_EINVAL;
    const size_t need = sga_gated_ff_fwd_workspace_bytes(T, F, M, dt);
    if (need && (!workspace || !aligned(workspace, 256))) return SGA_EINVAL;
    if (workspace_bytes < need) return SGA_EWORKSPACE;
    if ((st = status_of(bind_device())) != SGA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    FfSpace w{dt == SGA_F32, T, F, M, 0, static_cast<char *>(workspace)};
    FfLay lay{};
    FfProduct p{};
    p.x = w.take(X, T, F, &lay);
    p.wg = w.take(Wg, F, M, &lay);
    p.wu = w.take(Wu, F, M, &lay);
    p.T = T;
    p.F = F;
    p.M = M;
    p.act = act;
    p.out = out;
    p.g = G;
    p.u = U;
    p.partial = reinterpret_cast<float *>(w.base + w.used);
    cudaError_t e = lay_out(lay, w.f32, s);
    FfShares shares{}, none{};
    if (e == cudaSuccess) e = w.f32 ? ff_product<FfMode::FWD, true>(p, shares, s) : ff_product<FfMode::FWD, false>(p, shares, s);
    if (e == cudaSuccess) e = w.f32 ? ff_join<true, true>(shares, none, s) : ff_join<true, false>(shares, none, s);
    return status_of(e);
}

size_t sga_gated_ff_bwd_workspace_bytes(int64_t T, int64_t F, int64_t M, sga_dtype dt) {
    if (T <= 0 || check_ff(T, F, M, SGA_ACT_SILU, dt) != SGA_OK) return 0;
    FfSpace w{dt == SGA_F32, T, F, M};
    w.take(nullptr, T, F, nullptr);
    w.take(nullptr, F, M, nullptr);
    w.take(nullptr, F, M, nullptr);
    w.operand(T, M);
    w.operand(T, M);
    w.bytes(partial_bytes<FfMode::DX>(T, F, M, w.f32));
    w.bytes(partial_bytes<FfMode::DW>(T, F, M, w.f32));
    return w.used;
}

sga_status gated_ff_bwd(const void *X, const void *Wg, const void *Wu, const void *G, const void *U, const void *dOut, int64_t T, int64_t F,
                        int64_t M, int act, sga_dtype dt, void *dX, void *dWg, void *dWu, void *workspace, size_t workspace_bytes,
                        void *stream) {
    sga_status st = check_ff(T, F, M, act, dt);
    if (st != SGA_OK) return st;
    if (!dWg != !dWu || !aligned(dX, 16) || !aligned(dWg, 16) || !aligned(dWu, 16)) return SGA_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {   // an empty sum
        const size_t bytes = (size_t)F * M * (dt == SGA_F32 ? 4 : 2);
        cudaError_t e = cudaSuccess;
        if (dWg) e = cudaMemsetAsync(dWg, 0, bytes, s);
        if (dWu && e == cudaSuccess) e = cudaMemsetAsync(dWu, 0, bytes, s);
        return status_of(e);
    }
    for (const void *p : {X, Wg, Wu, G, U, dOut})
        if (!p || !aligned(p, 16)) return SGA_EINVAL;
    if (!workspace || !aligned(workspace, 256)) return SGA_EINVAL;
    if (workspace_bytes < sga_gated_ff_bwd_workspace_bytes(T, F, M, dt)) return SGA_EWORKSPACE;
    if (!dX && !dWg) return SGA_OK;
    if ((st = status_of(bind_device())) != SGA_OK) return st;
    FfSpace w{dt == SGA_F32, T, F, M, 0, static_cast<char *>(workspace)};
    FfLay lay{};
    FfProduct p{};
    p.x = w.take(X, T, F, dWg ? &lay : nullptr);
    p.wg = w.take(Wg, F, M, dX ? &lay : nullptr);
    p.wu = w.take(Wu, F, M, dX ? &lay : nullptr);
    p.dg = p.du = FfMatrix{nullptr, T, M, round8(M)};
    p.dg.p = reinterpret_cast<const __nv_bfloat16 *>(w.base + w.operand(T, M));
    p.du.p = reinterpret_cast<const __nv_bfloat16 *>(w.base + w.operand(T, M));
    p.T = T;
    p.F = F;
    p.M = M;
    p.act = act;
    cudaError_t e = lay_out(lay, w.f32, s);
    if (e == cudaSuccess) e = w.f32 ? slopes<float>(G, U, dOut, act, p.dg, p.du, s) : slopes<__nv_bfloat16>(G, U, dOut, act, p.dg, p.du, s);
    FfShares of_x{}, of_w{};
    if (dX && e == cudaSuccess) {
        p.out = dX;
        p.partial = reinterpret_cast<float *>(w.base + w.bytes(partial_bytes<FfMode::DX>(T, F, M, w.f32)));
        e = w.f32 ? ff_product<FfMode::DX, true>(p, of_x, s) : ff_product<FfMode::DX, false>(p, of_x, s);
    }
    if (dWg && e == cudaSuccess) {
        p.g = dWg;
        p.u = dWu;
        p.partial = reinterpret_cast<float *>(w.base + w.bytes(partial_bytes<FfMode::DW>(T, F, M, w.f32)));
        e = w.f32 ? ff_product<FfMode::DW, true>(p, of_w, s) : ff_product<FfMode::DW, false>(p, of_w, s);
    }
    if (e == cudaSuccess) e = w.f32 ? ff_join<false, true>(of_x, of_w, s) : ff_join<false, false>(of_x, of_w, s);
    return status_of(e);
}

sga_status sga_gated_ff_read_device_error(void *stream, int32_t *code) {
    if (!code) return SGA_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int32_t v = 0;
    const int32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_ff_err, sizeof v, 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbolAsync(g_ff_err, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess && v) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return status_of(e);
    *code = v;
    return v ? SGA_EDEVICE_CHECK : SGA_OK;
}

}  // extern "C"
