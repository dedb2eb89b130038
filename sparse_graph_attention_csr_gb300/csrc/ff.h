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

// Phi(x) = erfc(-x / sqrt(2)) / 2, the normal distribution function, by the Chebyshev
// fit to erfc of "Numerical Recipes" (Press et al., erfcc), whose relative error is below
// 1.2e-7 (2 units of 2^-24) everywhere.  In fp32 the exponent's rounding adds to that in
// the tail: off by 8 + 2 x^2 such units of Phi for x < 0 (emulated: 34 down to x = -4, 122
// to -8), by 6 for x > 0.  erfcf, whose chain is longer, took 20 us more of a forward of
// 4099 x 301 x 803 in fp32.
__device__ __forceinline__ float ff_phi(float x) {
    const float z = 0.70710678118654752f * fabsf(x), t = __fdividef(1.f, fmaf(0.5f, z, 1.f));
    float y = fmaf(t, 0.17087277f, -0.82215223f);
    y = fmaf(t, y, 1.48851587f);
    y = fmaf(t, y, -1.13520398f);
    y = fmaf(t, y, 0.27886807f);
    y = fmaf(t, y, -0.18628806f);
    y = fmaf(t, y, 0.09678418f);
    y = fmaf(t, y, 0.37409196f);
    y = fmaf(t, y, 1.00002368f);
    y = fmaf(t, y, -1.26551223f);
    const float q = 0.5f * t * fast_exp2(kLog2e * fmaf(-z, z, y));
    return x < 0.f ? q : 1.f - q;
}

// act(g).  Exponentials and quotients by the MUFU instructions: off by a few units of
// 2^-24, and by 1.2 more for each unit of |g| (the exponent's rounding).
__device__ __forceinline__ float ff_silu(float g) { return __fdividef(g, 1.f + fast_exp2(-kLog2e * g)); }
__device__ __forceinline__ float ff_relu(float g) { return g != g ? g : fmaxf(g, 0.f); }
// Calls f with the activation.
template <typename F> __device__ __forceinline__ void ff_with_act(int act, F f) {
    if (act == SGA_ACT_SILU) f([](float g) { return ff_silu(g); });
    else if (act == SGA_ACT_GELU) f([](float g) { return g * ff_phi(g); });
    else f([](float g) { return ff_relu(g); });
}
// Calls f with a function of g, a, slope: the activation and its derivative (relu: 0 at 0).
template <typename F> __device__ __forceinline__ void ff_with_slope(int act, F f) {
    if (act == SGA_ACT_SILU) {
        f([](float g, float &a, float &slope) {
            const float s = __fdividef(1.f, 1.f + fast_exp2(-kLog2e * g));
            a = g * s;
            slope = fmaf(a, 1.f - s, s);
        });
    } else if (act == SGA_ACT_GELU) {
        f([](float g, float &a, float &slope) {
            const float p = ff_phi(g);
            a = g * p;
            slope = fmaf(g * 0.39894228040143268f, fast_exp2(-0.5f * kLog2e * g * g), p);
        });
    } else {
        f([](float g, float &a, float &slope) {
            a = ff_relu(g);
            slope = g > 0.f ? 1.f : 0.f;
        });
    }
}

}  // namespace sga
