// What the tensor-core passes of packed-sequence attention share.
#pragma once

#include <cuda.h>

#include "seq.h"
#include "tc.cuh"

namespace sga {

// TMA descriptor of a [rows][heads][D] bf16 tensor: boxes of 64 elements of one
// head x 128 rows in the 128-byte swizzle (one column atom of a K-major tile).
// Rows past the last sequence, and elements past D (D = 32: the box is wider
// than a head), read as zero.
cudaError_t seq_tensor_map(CUtensorMap *m, const void *base, int64_t rows, int heads, int D);

namespace seq {

// A head's tile of 128 rows: its column atoms, one behind the other.
template <int DA>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, int head, int row, uint64_t *mbar) {
#pragma unroll
    for (int at = 0; at < DA; ++at) tc::tma_load_3d(dst + at * 16384, map, at * 64, head, row, mbar);
}

// Bit c of the result's word w: column 32 w + c of a tile lies in [lo, hi).
__device__ __forceinline__ uint32_t column_bits(int lo, int hi, int w) {
    const int a = max(0, min(32, lo - 32 * w)), b = max(0, min(32, hi - 32 * w));
    const uint32_t upto_b = b == 32 ? 0xffffffffu : (1u << b) - 1u, upto_a = a == 32 ? 0xffffffffu : (1u << a) - 1u;
    return upto_b & ~upto_a;
}

// a row's interval relative to the tile that starts at row t0
__device__ __forceinline__ int rel(int64_t x, int64_t t0) {
    return (int)max((int64_t)0, min((int64_t)128, x - t0));
}

}  // namespace seq
}  // namespace sga
