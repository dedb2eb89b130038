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
#pragma once

#include "common.cuh"

namespace sga {

// One row tile: the tiles [t0, t1) of the other side that hold anything it
// sees (or is seen by), and of these [f0, f1), where every pair is visible.
struct SeqTile {
    int32_t tile, t0, t1, f0, f1, pad0, pad1, pad2;
};

}  // namespace sga

struct sga_seq_plan {
    int64_t B = 0, rows = 0;          // sequences, packed rows (the last entry of seq_ptr)
    int H = 0, Hkv = 0, D = 0;
    sga_dtype dt = SGA_F32;
    int causal = 0, num_sms = 0, device = 0;
    int tile_rows = 0;                // 128 (bf16) or 64 (fp32)
    int n_tiles = 0;
    // device memory of the plan
    int2 *d_range = nullptr;          // [rows] (s, e)
    sga::SeqTile *d_qtiles = nullptr; // row tiles of queries, most key tiles first
    sga::SeqTile *d_ktiles = nullptr; // row tiles of keys, most query tiles first
    sga::SeqTile *d_qpairs = nullptr; // neighbouring row tiles of queries by twos (bf16, odd head groups)
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
    int64_t rows, rows_pad;
    int H, Hkv, causal, n_tiles, num_sms;
    float scale;
    int32_t *d_err;
};

// rows of a head's slice of the backward's row terms: whole tiles, 512-byte aligned
inline int64_t seq_rows_pad(int64_t rows) { return (rows + 127) / 128 * 128; }

// -lse * log2(e) and -Delta of every row, head-major (seq_simt.cu)
template <typename T> cudaError_t seq_row_terms(const SeqArgs &a, int D, cudaStream_t s);
cudaError_t seq_fwd_f32(const SeqArgs &a, int D, cudaStream_t s);
cudaError_t seq_bwd_f32(const SeqArgs &a, int D, cudaStream_t s);
// (seq_fwd.cu, seq_bwd.cu)
cudaError_t seq_fwd_bf16(const SeqArgs &a, int D, cudaStream_t s);
cudaError_t seq_bwd_bf16(const SeqArgs &a, int D, cudaStream_t s);

}  // namespace sga
