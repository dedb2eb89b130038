// Row terms of the attention backward, for both dtypes: -lse log2(e) and -Delta.
#include "seq.h"

namespace sga {
namespace {

// Row terms: D / EL lanes of 16 bytes a (row, head), two of them in flight: what is in
// flight on an SM comes from its blocks (25176 rows, 8 heads of 128, bf16: one 25.1 us,
// two 25.4, four 28.6, eight 43; 60000 rows, 4 of 64: 17.0, 17.6, 20.2, 32).  The next
// kernel's blocks take the places that are free when they may start, so they may once
// the loads are out: started before, they lay uneven over the SMs (2900 rows, 4/2 heads
// of 32, window 129, fp32: backward 72 us, now 59).
// With four in flight half as many blocks end later, and the next kernel's lie uneven
// again; the fp32 passes ask for that where their rounds come out better so.
// Rows behind the last sequence (to the end of its tile) get -lse = -inf, so
// that their weights are zero, and Delta = 0.
template <typename T, int D, int kTerms> __global__ void __launch_bounds__(256) seq_row_terms_kernel(const SeqArgs a) {
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
    let_next_start();
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

template <typename T, int D, int kTerms = 2> cudaError_t launch_terms(const SeqArgs &a, cudaStream_t s) {
    constexpr int per = kTerms * 256 / (D / Elt<T>::EL);   // items of a block
    note_launch(SGA_KERN_SEQ_BWD_ROWS, s, false);
    const cudaError_t e = launch_early(seq_row_terms_kernel<T, D, kTerms>, dim3((unsigned)((a.rows_pad * a.H + per - 1) / per)), dim3(256), 0, s, a);
    note_launch(SGA_KERN_SEQ_BWD_ROWS, s, true);
    return e;
}

}  // namespace

template <typename T> cudaError_t seq_row_terms(const SeqArgs &a, int D, cudaStream_t s, bool uneven) {
    if constexpr (sizeof(T) == 4)
        if (uneven && D < 128) return D == 32 ? launch_terms<T, 32, 4>(a, s) : launch_terms<T, 64, 4>(a, s);
    return D == 32 ? launch_terms<T, 32>(a, s) : D == 64 ? launch_terms<T, 64>(a, s) : launch_terms<T, 128>(a, s);
}
template cudaError_t seq_row_terms<float>(const SeqArgs &, int, cudaStream_t, bool);
template cudaError_t seq_row_terms<__nv_bfloat16>(const SeqArgs &, int, cudaStream_t, bool);

}  // namespace sga
