// The gated feed-forward product: what its host code and its tensor-core products
// (ff_gemm.cuh) share.
//   forward   G = X Wg, U = X Wu, out = act(G) U              X [T, F], Wg, Wu [F, M]
//   backward  dG = dOut U act'(G), dU = dOut act(G)
//             dX = dG Wg^T + dU Wu^T,  dWg = X^T dG,  dWu = X^T dU
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace sga {

enum class FfMode { FWD, DX, DW };

// A matrix [rows][cols] of bf16, rows `ld` elements apart, or in fp32 the three
// bf16 parts that make it up, one behind the other.
struct FfMatrix {
    const __nv_bfloat16 *p = nullptr;
    int64_t rows = 0, cols = 0, ld = 0;
    __host__ __device__ int64_t part_elems() const { return rows * ld; }
};

struct FfProduct {
    FfMode mode;
    bool f32;                  // operands in three parts, results in fp32
    FfMatrix x, wg, wu;        // X; the weights (DW: unused)
    FfMatrix dg, du;           // backward
    int64_t T, F, M;
    int act;
    void *out, *g, *u;         // FWD: out [T, M], and G, U unless null; DX: out = dX [T, F]; DW: g = dWg, u = dWu [F, M]
    float *partial;            // fp32 sums of tiles whose depth is shared by several CTA pairs
};

// ---- activations: 0 silu, 1 gelu (by the normal distribution function), 2 relu -------

// Phi(x), the normal distribution function: erfc's own accuracy in its tail.
__device__ __forceinline__ float ff_phi(float x) { return 0.5f * erfcf(-0.70710678118654752f * x); }

// act(g); FAST: results that are rounded to bf16
template <bool FAST> __device__ __forceinline__ float ff_act(float g, int act) {
    if (act == SGA_ACT_SILU) return FAST ? __fdividef(g, 1.f + fast_exp2(-kLog2e * g)) : g / (1.f + expf(-g));
    if (act == SGA_ACT_GELU) return g * ff_phi(g);
    return g != g ? g : fmaxf(g, 0.f);
}
// act(g) and its derivative (relu: 0 at 0)
template <bool FAST> __device__ __forceinline__ void ff_act_slope(float g, int act, float &a, float &slope) {
    if (act == SGA_ACT_SILU) {
        const float e = FAST ? fast_exp2(-kLog2e * g) : expf(-g), s = FAST ? __fdividef(1.f, 1.f + e) : 1.f / (1.f + e);
        a = g * s;
        slope = fmaf(a, 1.f - s, s);
    } else if (act == SGA_ACT_GELU) {
        const float p = ff_phi(g);
        a = g * p;
        slope = fmaf(g * 0.39894228040143268f, FAST ? fast_exp2(-0.5f * kLog2e * g * g) : expf(-0.5f * g * g), p);
    } else {
        a = g != g ? g : fmaxf(g, 0.f);
        slope = g > 0.f ? 1.f : 0.f;
    }
}

}  // namespace sga
