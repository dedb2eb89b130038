// What the tensor-core passes of packed-sequence attention share.
#pragma once

#include <cuda.h>

#include "seq_rows.cuh"
#include "tc.cuh"

namespace sga {

// TMA descriptor of a [rows][heads][D] bf16 tensor: boxes of 64 elements of one
// head x 128 rows in the 128-byte swizzle (one column atom of a K-major tile).
// Rows past the last sequence, and elements past D (D = 32: the box is wider
// than a head), read as zero.
// box_rows: 128, or 32 for a result that each warp stores its share of.
cudaError_t seq_tensor_map(CUtensorMap *m, const void *base, int64_t rows, int heads, int D, int box_rows = 128);

namespace seq {

// A head's tile of 128 rows: its column atoms, one behind the other.
template <int DA>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, int head, int row, uint64_t *mbar) {
#pragma unroll
    for (int at = 0; at < DA; ++at) tc::tma_load_3d(dst + at * 16384, map, at * 64, head, row, mbar);
}

// Results leave through shared memory and TMA where a head fills whole boxes of 64
// columns: stored by the threads that hold a row each, every 16-byte store of a warp
// would touch 32 lines.
template <int D> constexpr bool kTmaResult = D >= 64;
// 32 columns from c0 of a row of a tile, scaled, into the tile's place (K-major,
// 128-byte swizzle, as loaded).
__device__ __forceinline__ void stage_columns(uint32_t tile, int row, int c0, const float *x) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 v = pack<__nv_bfloat16>(x + 8 * q);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(tile + (c0 >> 6) * 16384 + row * 128 +
                                                                      ((((c0 & 63) / 8 + q) ^ (row & 7)) << 4)),
                     "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                     : "memory");
    }
}
// One lane: 32 rows (from tile row r, packed row `row`) of the tile's column atom to
// head `head` of the result.
__device__ __forceinline__ void store_atom(const CUtensorMap *map, uint32_t tile, int atom, int r, int head, int64_t row, int64_t rows) {
    if (row < rows) tc::tma_store_3d(map, atom * 64, head, (int)row, tile + atom * 16384 + r * 128);
}
// Barrier `id` over 64 threads, with whether any of them passed `flag`.
__device__ __forceinline__ bool pair_any(int id, bool flag) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"((uint32_t)flag), "r"(id) : "memory");
    return r != 0;
}

// Bit c of the result's word w: column 32 w + c of a tile lies in [lo, hi).
__device__ __forceinline__ uint32_t column_bits(int lo, int hi, int w) {
    const int a = max(0, min(32, lo - 32 * w)), b = max(0, min(32, hi - 32 * w));
    const uint32_t upto_b = b == 32 ? 0xffffffffu : (1u << b) - 1u, upto_a = a == 32 ? 0xffffffffu : (1u << a) - 1u;
    return upto_b & ~upto_a;
}

// The tiles that a query tile (or two of one unit) walks, in order: of windowed
// plans the sinks' (of both tiles) and then the window's, which are disjoint.
template <bool WIN> struct Walk {
    int t0, n;
    __device__ __forceinline__ Walk(const SeqTile &x, const SeqTile &y) : t0(min(x.t0, y.t0)), n(max(x.t1, y.t1) - t0) {}
    __device__ __forceinline__ int tile(int i) const { return t0 + i; }
};
template <> struct Walk<true> {
    int g0, ng, h0, nh, t0, n;
    __device__ __forceinline__ Walk(const SeqTile &x, const SeqTile &y) {
        t0 = min(x.t0, y.t0);
        // (the second tile's sinks begin no earlier than the first's)
        const int g1 = min(x.g1, t0), h1 = min(y.g1, t0);
        g0 = x.g0;
        ng = max(0, g1 - g0);
        h0 = ng > 0 ? max(y.g0, g1) : y.g0;
        nh = max(0, h1 - h0);
        n = ng + nh + max(x.t1, y.t1) - t0;
    }
    __device__ __forceinline__ int tile(int i) const { return i < ng ? g0 + i : i < ng + nh ? h0 + i - ng : t0 + i - ng - nh; }
};
// Whether the tile's own walk holds tile kt of the other side.
template <bool WIN> __device__ __forceinline__ bool walks(const SeqTile &t, int kt) {
    return (kt >= t.t0 && kt < t.t1) || (WIN && kt >= t.g0 && kt < t.g1);
}
// A tile's own walk.
template <bool WIN> __device__ __forceinline__ int own_count(const SeqTile &t) { return (WIN ? t.g1 - t.g0 : 0) + t.t1 - t.t0; }
template <bool WIN> __device__ __forceinline__ int own_tile(const SeqTile &t, int i) {
    if (WIN && i < t.g1 - t.g0) return t.g0 + i;
    return t.t0 + i - (WIN ? t.g1 - t.g0 : 0);
}

// a row's interval relative to the tile that starts at row t0
__device__ __forceinline__ int rel(int64_t x, int64_t t0) {
    return (int)max((int64_t)0, min((int64_t)128, x - t0));
}

// The columns of word w of the tile at row t0 that a row sees.
template <bool WIN> __device__ __forceinline__ uint32_t view_bits(const View<WIN> &v, int64_t t0, int w) {
    uint32_t bits = column_bits(rel(v.lo, t0), rel(v.hi, t0), w);
    if constexpr (WIN) bits |= column_bits(rel(v.slo, t0), rel(v.shi, t0), w);
    return bits;
}

}  // namespace seq
}  // namespace sga
