// dK and dV of the key tiles whose walk over the queries was cut into parts (the
// sinks of long sequences): the parts' fp32 sums added in order, a warp a row of a
// head.  Bound by reading them: 32768 rows with a window of 1024 leave 16 parts of
// 128 rows, 2 MB a key head of 128.
#include "seq_rows.cuh"

namespace sga {
namespace {

template <typename T, int D, int TR> __global__ void __launch_bounds__(256) seq_join_kernel(const SeqArgs a) {
    wait_previous();
    const int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);   // (cut tile, row, key head, dV or dK)
    const bool dk = u & 1;
    const int hk = (int)(u / 2 % a.Hkv), r = (int)(u / 2 / a.Hkv % TR);
    const int64_t j = u / 2 / a.Hkv / TR;
    if (j >= a.n_joins) return;
    const SeqJoin c = a.joins[j];
    const int64_t row = (int64_t)c.tile * TR + r;
    if (row >= a.rows) return;
    constexpr int W = D / 32;
    seq::RowFrag<float, D> sum, x;
    sum.zero();
    const int64_t step = (int64_t)a.Hkv * 2 * TR * D;
    const float *src = a.ws_part + (int64_t)(c.part - 1) * step + ((int64_t)hk * 2 + dk) * TR * D + r * D;
#pragma unroll 4
    for (int i = 0; i < c.count; ++i) {
        x.load(src + i * step, 0);
#pragma unroll
        for (int k = 0; k < W; ++k) sum.x[k] += x.x[k];
    }
    seq::RowFrag<T, D> res;
#pragma unroll
    for (int k = 0; k < W; ++k) res.x[k] = sum.x[k];
    res.store(dk ? a.dK : a.dV, (row * a.Hkv + hk) * D, dk ? a.scale : 1.f, ~0u);
    bool bad = false;
#pragma unroll
    for (int k = 0; k < W; ++k) bad |= !(fabsf(to_f32<T>(from_f32<T>(sum.x[k] * (dk ? a.scale : 1.f)))) < INFINITY);
    if (!__any_sync(SGA_FULL_MASK, bad)) return;
    seq::Span<true> sp;
    static_cast<seq::View<true> &>(sp) = seq::key_view<true>(a, row);
    sp.w0 = (int64_t)c.t0 * TR;
    sp.w1 = min(a.rows, (int64_t)c.t1 * TR);
    seq::key_row_alone<T, D, true>(a, dk, row, hk, sp, ~0u);
}

template <typename T, int D> cudaError_t launch(const SeqArgs &a, cudaStream_t s) {
    constexpr int TR = sizeof(T) == 2 ? 128 : 64;
    note_launch(SGA_KERN_SEQ_JOIN, s, false);
    const cudaError_t e = launch_early(seq_join_kernel<T, D, TR>, dim3((unsigned)(((int64_t)a.n_joins * TR * a.Hkv * 2 + 7) / 8)), dim3(256), 0, s, a);
    note_launch(SGA_KERN_SEQ_JOIN, s, true);
    return e;
}

}  // namespace

template <typename T> cudaError_t seq_join(const SeqArgs &a, int D, cudaStream_t s) {
    if (a.n_joins == 0) return cudaSuccess;
    return D == 32 ? launch<T, 32>(a, s) : D == 64 ? launch<T, 64>(a, s) : launch<T, 128>(a, s);
}
template cudaError_t seq_join<float>(const SeqArgs &, int, cudaStream_t);
template cudaError_t seq_join<__nv_bfloat16>(const SeqArgs &, int, cudaStream_t);

}  // namespace sga
