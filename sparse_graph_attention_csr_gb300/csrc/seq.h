// Packed-sequence attention: the plan, the arguments of its kernels and what
// they share.
//
// Sequences lie one behind the other along the rows of Q, K and V.  Row r
// belongs to the sequence [s_r, e_r) and sees the keys [s_r, causal ? r + 1 :
// e_r); seen from a key, the queries are [causal ? r : s_r, e_r).  The kernels
// cut the packed rows into tiles of 128 (64 in fp32) regardless of where
// sequences begin and end and mask each row to its own interval: a tile may
// hold many short sequences, which share its products, and a long sequence
// costs at most one tile more per row of tiles than if it began on one.
//
// With a window w and n sinks, row r of the sequence sees of those keys the ones
// less than w rows away, and the sequence's first n rows: two intervals, which
// are one while they touch.  A row tile then walks two ranges of tiles, the
// sinks' and the window's.  Seen from a key the queries stay one interval: those
// less than w rows away, or for a sink the whole of the sequence.
#pragma once

#include "common.cuh"

namespace sga {

// One row tile: the tiles [t0, t1) of the other side that hold anything it
// sees (or is seen by), and of these [f0, f1), where every pair is visible.
// Windowed plans: the tiles [g0, g1) of a query tile's sinks that lie before t0;
// and of a key tile whose walk is cut into parts, the number of the part (from 1;
// 0: not cut).
struct SeqTile {
    int32_t tile, t0, t1, f0, f1, g0, g1, part;
};

// A key tile whose walk over the query tiles [t0, t1) is cut into parts
// part .. part + count - 1, which leave fp32 sums that are joined afterwards.
struct SeqJoin {
    int32_t tile, t0, t1, part, count;
};

}  // namespace sga

struct sga_seq_plan {
    int64_t B = 0, rows = 0;          // sequences, packed rows (the last entry of seq_ptr)
    int H = 0, Hkv = 0, D = 0;
    sga_dtype dt = SGA_F32;
    int causal = 0, num_sms = 0, device = 0;
    int tile_rows = 0;                // 128 (bf16) or 64 (fp32)
    int n_tiles = 0;
    int window = 0, sinks = 0;        // window 0: none (or one that holds every sequence)
    int n_ktiles = 0;                 // entries of d_ktiles (n_tiles, but for cut walks)
    int n_parts = 0, n_joins = 0;
    // device memory of the plan
    int2 *d_range = nullptr;          // [rows] (s, e)
    sga::SeqTile *d_qtiles = nullptr; // row tiles of queries, most key tiles first
    sga::SeqTile *d_ktiles = nullptr; // row tiles of keys, most query tiles first
    sga::SeqTile *d_qpairs = nullptr; // neighbouring row tiles of queries by twos (bf16, odd head groups)
    sga::SeqJoin *d_joins = nullptr;
    int32_t *d_err = nullptr;
    int64_t device_bytes = 0;
};

namespace sga {

struct SeqArgs {
    const void *Q, *K, *V;
    const void *out;          // backward: the forward's out, lse; dOut
    const float *lse;
    const void *dOut;
    void *out_w;              // forward outputs
    float *lse_w;
    void *dQ, *dK, *dV;       // backward outputs
    float *ws_nlse, *ws_ndelta; // [H][rows_pad] -lse * log2(e) (-inf behind the last row) and -Delta
    const int2 *range;
    const SeqTile *qtiles, *ktiles, *qpairs;
    const SeqJoin *joins;
    float *ws_part;           // [n_parts][Hkv][2][tile rows][D] sums of dV, dK
    int64_t rows, rows_pad;
    int H, Hkv, causal, n_tiles, n_ktiles, n_joins, num_sms;
    int window, sinks;
    float scale;
    int32_t *d_err;
};

// rows of a head's slice of the backward's row terms: whole tiles, 512-byte aligned
inline int64_t seq_rows_pad(int64_t rows) { return (rows + 127) / 128 * 128; }

// -lse * log2(e) and -Delta of every row, head-major (seq_terms.cu); uneven: the next
// kernel's first blocks may lie unevenly over the SMs (fp32, D < 128)
template <typename T> cudaError_t seq_row_terms(const SeqArgs &a, int D, cudaStream_t s, bool uneven = false);
// the parts of cut walks added up (seq_join.cu)
template <typename T> cudaError_t seq_join(const SeqArgs &a, int D, cudaStream_t s);
// WIN: a plan with a window (a.window > 0)
template <bool WIN> cudaError_t seq_fwd_f32(const SeqArgs &a, int D, cudaStream_t s);
template <bool WIN> cudaError_t seq_bwd_f32(const SeqArgs &a, int D, cudaStream_t s);
template <bool WIN> cudaError_t seq_fwd_bf16(const SeqArgs &a, int D, cudaStream_t s);
template <bool WIN> cudaError_t seq_bwd_bf16(const SeqArgs &a, int D, cudaStream_t s);

}  // namespace sga
