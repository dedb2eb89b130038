// Products of the gated feed-forward block on the tcgen05 tensor cores, by CTA
// pairs (tc_pair.cuh): tiles of 256 x 256 (forward: 256 rows x 128 gate and the
// same 128 up columns, so that one thread has both halves of a result; dX: narrower
// ones where that covers its columns with less beside them).
//
// Persistent pairs; in each CTA
//   warp 0, one lane: TMA loads of its half of a k-block's operands (128 rows of A,
//     128 columns of B, 64 deep) into a ring, arriving at the first CTA's barriers;
//   warp 1 (first CTA): the products, into one of two accumulators of 256 columns;
//   warps 4 .. 11: move finished accumulators to registers and add them there
//     (every `depth` k-blocks), and store a tile's result, through shared memory
//     and TMA where its rows allow it.
// Operands lie in memory as the tensors do: X and dG of the dX product along their
// depth (K-major), weights of the forward and both operands of the dW product
// across it (MN-major).
//
// fp32: an operand is the sum of three bf16 parts (8 + 8 + 8 bits); of the nine
// products of parts the six that reach 2^-24 of the result are taken, smallest
// first.  The tensor core's accumulator drops what falls below its last bit, always
// towards zero, so every k-block's sum (64 deep) is added to fp32 registers: in a
// k-block only the four additions of the leading parts' products meet a sum of full
// size, and drop at most 2^-21 of it; a second k-block's smaller products would meet
// the first one's sum, 24 additions more.  Error of the norm, a k-block : two : four : a
// plain fp32 product, 8192 x 1024 x 4096, G, dW, dX: 1.1, 2.2, 2.0 : 6.0, 6.0, 5.9 :
// 14.6, 14.3, 14.3 : 5.7, 11.5, 8.1 e-7 (forward 518 : 483 : 463 us).
//
// Tiles are dealt to the pairs by whole rounds; the last, incomplete round would
// leave pairs idle, so its tiles' depth is cut into equal shares, which leave fp32
// sums that a second kernel adds in order (where that is quicker): no atomics, bitwise
// reproducible.
//
// Every wait is bounded; a timeout sets the error word and ends the role.
#pragma once

#include <algorithm>
#include <type_traits>

#include "ff.h"
#include "tc_dx.cuh"
#include "tc_pair.cuh"

namespace sga {

cudaError_t bf16_tensor_map(CUtensorMap *m, const __nv_bfloat16 *base, int64_t rows, int64_t cols, int64_t row_elems,
                            uint32_t box_cols, uint32_t box_rows);   // (tc_dx.cu)

namespace {

// Bit kErrMmaTimeout: a wait gave up since the last read, per device.
__device__ int32_t g_ff_err;

constexpr int kFfThreads = 384;
// Registers a thread at launch and after the split: an epilogue thread holds 128
// sums.  The shares add up to the launch's total.
constexpr int kFfLaunch = 168, kFfCtrl = 56, kFfEpi = 224;
static_assert(kFfCtrl + 2 * kFfEpi <= 3 * kFfLaunch, "register split");

template <FfMode MODE, bool F32> struct FfCfg {
    static constexpr int PARTS = F32 ? 3 : 1;
    static constexpr uint32_t TB = 128 * 128;                // a CTA's share of an operand's k-block, 128 x 64 bf16
    static constexpr uint32_t STAGE = 2 * PARTS * TB;
    static constexpr int NST = F32 ? 2 : 6;
    static constexpr uint32_t OUT0 = NST * STAGE;            // staging of results: 32 rows x 64 bf16 a warp
    static constexpr uint32_t BYTES = OUT0 + 8 * 4096;
    static constexpr bool A_MN = MODE == FfMode::DW, B_MN = MODE != FfMode::DX;
    static constexpr int BN = MODE == FfMode::FWD ? 128 : 256;   // columns of a result that a tile covers (DX: at most)
};
constexpr int kTileFloats = 256 * 256;

struct FfParams {
    CUtensorMap ta[2][3], tb[2][3];   // [segment (DX) or operand][part]
    CUtensorMap to[3];                // results: FWD out, G, U; DX dX; DW dWg, dWu
    void *out[3];
    float *partial;
    int64_t rows, cols;               // of a result
    int tiles_m, tiles_n;             // tiles
    int width;                        // columns of a result that a tile covers
    int kb, kb_seg;                   // k-blocks of a tile; of a segment
    int depth;                        // k-blocks between two moves to registers
    int pairs, whole;                 // pairs of the grid; tiles dealt whole
    int act, tma_out;
};

// Tile t's row and column of tiles: eight rows of tiles at a time, column by column,
// so that what the pairs load at one time is near square.
__host__ __device__ __forceinline__ void ff_tile(int t, int tiles_m, int tiles_n, int &m, int &n) {
    const int per = 8 * tiles_n, g = t / per, rest = t - g * per, rows = tiles_m - 8 * g < 8 ? tiles_m - 8 * g : 8;
    n = rest / rows;
    m = 8 * g + rest - n * rows;
}

// A pair's units: whole tiles pair, pair + pairs, ... of the first `whole`, then its
// share of the others' k-blocks, laid end to end; a share is no longer than a tile is
// deep, so it lies in one tile or two.
struct FfUnit {
    int tile, k0, k1, slot;   // k-blocks [k0, k1); slot of the partial sums, or -1 for a whole tile
};
struct FfUnits {
    int pair, pairs, kb, full, tile, k0, k1, next;   // the share: [k0, k1) of `tile`, [0, next) of the one behind it
    __host__ __device__ FfUnits(int tiles, int whole, int depth, int n_pairs, int which) : pair(which), pairs(n_pairs), kb(depth) {
        full = pair < whole ? (whole - 1 - pair) / pairs + 1 : 0;
        const int64_t all = (int64_t)(tiles - whole) * kb, b = all * pair / pairs, e = all * (pair + 1) / pairs;
        const int t = (int)(b / kb);
        tile = whole + t;
        k0 = (int)(b - (int64_t)t * kb);
        k1 = (int)(e - b) < kb - k0 ? k0 + (int)(e - b) : kb;
        next = (int)(e - b) - (k1 - k0);
    }
    // the i-th; false past the last
    __host__ __device__ __forceinline__ bool get(int i, FfUnit &u) const {
        if (i < full) {
            u = {pair + i * pairs, 0, kb, -1};
            return true;
        }
        if (i == full && k0 < k1) {
            u = {tile, k0, k1, 2 * pair};
            return true;
        }
        if (i == full + 1 && next > 0) {
            u = {tile + 1, 0, next, 2 * pair + 1};
            return true;
        }
        return false;
    }
};

// 32 x 32 floats of a warp (a row a lane) to rows of `ld` floats from dst, of which
// `rows` and `cols` are there, through the warp's staging: whole rows at a time (a row
// a lane, as they lie in the registers, would be 32 places a store).  vec: rows begin on
// 16 bytes, and cols is a multiple of 4.
__device__ __forceinline__ void ff_store_block(uint32_t stage, const float *x, float *dst, int64_t ld, int rows, int cols, bool vec) {
    const int lane = threadIdx.x & 31;
    __syncwarp();   // (what was staged before has been read)
#pragma unroll
    for (int c = 0; c < 8; ++c)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + ((c ^ (lane & 7)) << 4)), "f"(x[4 * c]),
                     "f"(x[4 * c + 1]), "f"(x[4 * c + 2]), "f"(x[4 * c + 3])
                     : "memory");
    __syncwarp();
    if (vec) {
        const int c = lane & 7;
#pragma unroll
        for (int q = 0; q < 32; q += 4) {
            const int r = q + (lane >> 3);
            float y[4];
            tc::lds128(stage + r * 128 + ((c ^ (r & 7)) << 4), y);
            if (r < rows && 4 * c < cols) *reinterpret_cast<float4 *>(dst + r * ld + 4 * c) = make_float4(y[0], y[1], y[2], y[3]);
        }
    } else {
#pragma unroll 8
        for (int r = 0; r < 32; ++r) {
            float y;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(y) : "r"(stage + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4));
            if (r < rows && lane < cols) dst[r * ld + lane] = y;
        }
    }
}

template <FfMode MODE, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFfThreads, 1) ff_gemm_kernel(const __grid_constant__ FfParams p) {
    using C = FfCfg<MODE, F32>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[C::NST], empty[C::NST][C::PARTS], tfull[2], tempty[2];
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
    const uint32_t sbase = tc::smem_u32(smem), rank = tc::cluster_rank();
    const FfUnits units(p.tiles_m * p.tiles_n, p.whole, p.kb, p.pairs, blockIdx.x >> 1);
    const int width = MODE == FfMode::DX ? p.width : C::BN;

    if (tid == 32) {
        for (int i = 0; i < C::NST; ++i) {
            tc::mbar_init(&full[i], 1);
            for (int q = 0; q < C::PARTS; ++q) tc::mbar_init(&empty[i][q], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&tfull[i], 1);
            tc::mbar_init(&tempty[i], 16);   // the epilogue warps of both CTAs
        }
    }
    if (warp == 2 && lane == 0) {   // (while the previous kernel ends)
        for (int i = 0; i < 2; ++i)
            for (int q = 0; q < C::PARTS; ++q) {
                if (i == 0 || MODE == FfMode::DX) tc::prefetch_map(&p.ta[i][q]);
                tc::prefetch_map(&p.tb[i][q]);
            }
    }
    wait_previous();
    tc::cluster_sync();   // both CTAs run, their barriers initialised
    if (warp == 0) tc::tmem_alloc_pair(&tmem_base, 512);
    tc::fence_before_sync();
    tc::cluster_sync();
    tc::fence_after_sync();
    let_next_start();

    if (warp < 4) {
        tc::reg_dec<kFfCtrl>();
        if (warp == 0 && lane == 0) {   // ----------------------------------- TMA producer
            bool ok = true;
            int it = 0;
            FfUnit u;
            for (int i = 0; ok && units.get(i, u); ++i) {
                int tm, tn;
                ff_tile(u.tile, p.tiles_m, p.tiles_n, tm, tn);
                for (int kb = u.k0; kb < u.k1; ++kb, ++it) {
                    const int s = it % C::NST, r = it / C::NST;
                    // (the parts' places get free one after the other, the smallest's first)
                    if (r >= 1 && !tc::mbar_wait_cluster(&empty[s][C::PARTS - 1], (r - 1) & 1, tc::kWaitLimit)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) tc::mbar_expect_tx(&full[s], MODE == FfMode::DX ? C::PARTS * (2 * C::TB + width * 128) : 2 * C::STAGE);
                    const uint32_t bar = tc::map_rank(&full[s], 0), at = sbase + s * C::STAGE;
                    const int seg = MODE == FfMode::DX && kb >= p.kb_seg, k = (kb - (seg ? p.kb_seg : 0)) * 64;
                    const int m0 = tm * 256 + rank * 128;
                    int b, n0;   // which B, and the first of this CTA's columns
                    if (MODE == FfMode::FWD) {
                        b = rank;
                        n0 = tn * 128;
                    } else if (MODE == FfMode::DX) {
                        b = seg;
                        n0 = tn * width + rank * (width / 2);
                    } else {
                        b = 2 * tn >= p.tiles_n;
                        n0 = (tn - (b ? p.tiles_n / 2 : 0)) * 256 + rank * 128;
                    }
#pragma unroll
                    for (int q = C::PARTS - 1; q >= 0; --q) {
                        if (q < C::PARTS - 1 && r >= 1) ok = ok && tc::mbar_wait_cluster(&empty[s][q], (r - 1) & 1, tc::kWaitLimit);
                        const uint32_t pa = at + q * C::TB, pb = at + (C::PARTS + q) * C::TB;
                        const CUtensorMap *ma = &p.ta[MODE == FfMode::DX ? seg : 0][q], *mb = &p.tb[b][q];
                        if (C::A_MN) {
                            tc::tma_load_2d_pair(pa, ma, m0, k, bar);
                            tc::tma_load_2d_pair(pa + 8192, ma, m0 + 64, k, bar);
                        } else {
                            tc::tma_load_2d_pair(pa, ma, k, m0, bar);
                        }
                        if (C::B_MN) {
                            tc::tma_load_2d_pair(pb, mb, n0, k, bar);
                            tc::tma_load_2d_pair(pb + 8192, mb, n0 + 64, k, bar);
                        } else {
                            tc::tma_load_2d_pair(pb, mb, k, n0, bar);
                        }
                    }
                    if (!ok) {   // (all of the stage is on its way, so that it can be waited for)
                        ++it;
                        break;
                    }
                }
            }
            // (what the products' completion arrives at, here and in the other CTA, stays until it has)
            for (int i = it - 1; ok && i >= 0 && i >= it - C::NST; --i)
                for (int q = 0; q < C::PARTS; ++q) ok = ok && tc::mbar_wait_cluster(&empty[i % C::NST][q], (i / C::NST) & 1, tc::kWaitLimit);
            if (!ok) atomicOr(&g_ff_err, tc::kErrMmaTimeout);
            // loads of both CTAs that no product consumed (only after a timeout) land before the pair ends
            if (rank == 0)
                for (int i = it - 1; i >= 0 && i >= it - C::NST; --i) tc::mbar_wait_cluster(&full[i % C::NST], (i / C::NST) & 1, tc::kWaitLimit);
        } else if (warp == 1 && rank == 0) {   // ---------------------------- MMA issuer (the warp in step)
            const uint32_t idesc = tc::idesc_bf16(256, MODE == FfMode::DX ? width : 256) | (C::A_MN ? tc::kMajorMnA : 0u) | (C::B_MN ? tc::kMajorMnB : 0u);
            // parts of A and B by product, the smallest products first
            constexpr int NP = F32 ? 6 : 1, PA[6] = {2, 0, 1, 1, 0, 0}, PB[6] = {0, 2, 1, 0, 1, 0};
            bool ok = true;
            int it = 0, chunk = 0;
            FfUnit u;
            for (int i = 0; ok && units.get(i, u); ++i)
                for (int c0 = u.k0; ok && c0 < u.k1; c0 += p.depth, ++chunk) {
                    const int buf = chunk & 1, use = chunk >> 1, c1 = min(u.k1, c0 + p.depth);
                    if (use >= 1 && !tc::warp_wait_cluster(&tempty[buf], (use - 1) & 1, tc::kWaitLimit)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t d = tmem_base + buf * 256;
                    for (int kb = c0; kb < c1; ++kb, ++it) {
                        const int s = it % C::NST;
                        if (!tc::warp_wait_cluster(&full[s], (it / C::NST) & 1, tc::kWaitLimit)) {
                            ok = false;
                            break;
                        }
                        tc::fence_after_sync();
                        const uint32_t at = sbase + s * C::STAGE;
#pragma unroll
                        for (int q = 0; q < NP; ++q) {
                            const uint32_t a = at + (F32 ? PA[q] : 0) * C::TB, b = at + (C::PARTS + (F32 ? PB[q] : 0)) * C::TB;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc::mma_bf16_pair_w(d, C::A_MN ? tc::desc_sw128_mn(a + kk * 2048, 8192) : tc::desc_sw128(a + kk * 32),
                                                    C::B_MN ? tc::desc_sw128_mn(b + kk * 2048, 8192) : tc::desc_sw128(b + kk * 32), idesc,
                                                    kb > c0 || q > 0 || kk > 0);
                            // a part's place is free after the last product that takes it
                            if (F32 && q == 1) tc::mma_commit_pair_w(&empty[s][2]);
                            if (F32 && q == 4) tc::mma_commit_pair_w(&empty[s][1]);
                        }
                        tc::mma_commit_pair_w(&empty[s][0]);
                    }
                    tc::mma_commit_pair_w(&tfull[buf]);
                }
            if (!ok && lane == 0) atomicOr(&g_ff_err, tc::kErrMmaTimeout);
            // (every product issued is complete before TMEM is released: the epilogue of both CTAs waits for tfull;
            // after a timeout the last commit is waited for here)
            if (!ok)
                for (int b = 0; b < 2; ++b) tc::warp_wait_cluster(&tfull[b], ((chunk + (b ^ (chunk & 1))) >> 1) & 1, 1u << 16);
        }
        __syncwarp();
    } else {   // ---------------------------------------------------- sums and results
        tc::reg_inc<kFfEpi>();
        const int quarter = warp & 3, half = (warp - 4) >> 2;   // TMEM lanes 32 quarter ..; which half of the columns
        const uint32_t tl = (uint32_t)(quarter * 32) << 16, stage = sbase + C::OUT0 + (warp - 4) * 4096;
        bool ok = true, stored = false;
        int chunk = 0;
        FfUnit u;
        // column of a tile at which the thread's j-th block of 32 lies (forward: gate, gate, up, up)
        auto column = [&](int j) { return MODE == FfMode::FWD ? (j >> 1) * 128 + half * 64 + (j & 1) * 32 : half * 128 + j * 32; };
        for (int i = 0; ok && units.get(i, u); ++i) {
            float acc[128];
#pragma unroll
            for (int k = 0; k < 128; ++k) acc[k] = 0.f;
            for (int c0 = u.k0; c0 < u.k1; c0 += p.depth, ++chunk) {
                const int buf = chunk & 1;
                if (!tc::warp_wait_cluster(&tfull[buf], (chunk >> 1) & 1, tc::kWaitLimit)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (MODE == FfMode::DX && column(j >> 1) >= width) continue;
                    uint32_t v[16];
                    tc::tmem_ld16(tmem_base + buf * 256 + column(j >> 1) + (j & 1) * 16 + tl, v);
#pragma unroll
                    for (int k = 0; k < 16; ++k) acc[16 * j + k] += __uint_as_float(v[k]);
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::arrive_at(tc::map_rank(&tempty[buf], 0));
            }
            if (!ok) break;
            int tm, tn;
            ff_tile(u.tile, p.tiles_m, p.tiles_n, tm, tn);
            const int r = rank * 128 + quarter * 32;   // the warp's first row of the tile
            const int64_t row0 = (int64_t)tm * 256 + r;
            const int rows = (int)max((int64_t)0, min((int64_t)32, p.rows - row0));
            if (u.slot >= 0) {   // a share: its sums
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (rows > 0 && (MODE != FfMode::DX || column(j) < width)) {
                        if (stored) tc::bulk_wait_read();   // (a result's store may still read the staging)
                        ff_store_block(stage, acc + 32 * j, p.partial + (int64_t)u.slot * kTileFloats + r * 256 + column(j), 256, rows, 32, true);
                    }
                continue;
            }
            const int which = MODE == FfMode::DW && 2 * tn >= p.tiles_n;   // dWu
            const int64_t col0 = (int64_t)(tn - (which ? p.tiles_n / 2 : 0)) * width, end = min(p.cols, col0 + width);
            // 64 columns x[0 .. 63] of result o, from column col
            auto store = [&](int o, const float *x, int64_t col) {
                if constexpr (F32) {
#pragma unroll
                    for (int j = 0; j < 64; j += 32)
                        if (rows > 0 && col + j < end)
                            ff_store_block(stage, x + j, static_cast<float *>(p.out[o]) + row0 * p.cols + col + j, p.cols, rows,
                                           (int)min((int64_t)32, end - col - j), p.tma_out);
                } else {   // staged in the swizzle of its tensor map
                    if (stored) tc::bulk_wait_read();   // (the lane that stored; others have nothing to wait for)
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint4 v = pack<__nv_bfloat16>(x + 8 * c);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + ((c ^ (lane & 7)) << 4)), "r"(v.x),
                                     "r"(v.y), "r"(v.z), "r"(v.w)
                                     : "memory");
                    }
                    if (p.tma_out) {
                        tc::fence_proxy_async();
                        __syncwarp();
                        if (lane == 0 && col < end && rows > 0) {
                            tc::tma_store_2d(&p.to[o], (int)col, (int)row0, stage);
                            tc::bulk_commit();
                            stored = true;
                        }
                    } else {   // rows off 16 bytes: two elements a lane, a row at a time
                        __syncwarp();
                        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out[o]);
                        for (int q = 0; q < rows; ++q) {
                            uint32_t v;
                            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(stage + q * 128 + (((lane >> 2) ^ (q & 7)) << 4) + (lane & 3) * 4));
                            unsigned short *d = reinterpret_cast<unsigned short *>(dst + (row0 + q) * p.cols + col + 2 * lane);
                            if (col + 2 * lane < end) d[0] = (unsigned short)v;
                            if (col + 2 * lane + 1 < end) d[1] = (unsigned short)(v >> 16);
                        }
                    }
                }
            };
            if constexpr (MODE == FfMode::FWD) {
                const int64_t col = col0 + half * 64;
                if (p.out[1]) {
                    store(1, acc, col);
                    store(2, acc + 64, col);
                }
                // (one activation's code after the other: chosen per element, it did not
                // fit the instruction caches)
                ff_with_act(p.act, [&](auto f) {
#pragma unroll
                    for (int e = 0; e < 64; ++e) acc[e] = f(acc[e]) * acc[64 + e];
                });
                store(0, acc, col);
            } else {
#pragma unroll
                for (int x = 0; x < 2; ++x) store(which, acc + 64 * x, col0 + half * 128 + 64 * x);
            }
        }
        if (stored) tc::bulk_wait_read();   // (shared memory stays until then; the kernel's end waits for the rest)
        if (!ok && lane == 0) atomicOr(&g_ff_err, tc::kErrMmaTimeout);
        tc::fence_before_sync();
    }
    __syncwarp();
    tc::cluster_sync();   // nothing arrives at this CTA's barriers, or reads its operands, any more
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc_pair(tmem_base, 512);
}

// A product's tiles of the last round, whose shares are to be joined: which ones make
// up each, in the order of their k-blocks (slot[first[t]] .. slot[first[t + 1] - 1] of
// tile whole + t).
constexpr int kFfMaxPairs = 128;
struct FfShares {
    const float *partial;
    void *out[3];
    int64_t rows, cols;
    int tiles_m, tiles_n, width, whole, tiles;   // tiles: of the last round
    int act, wide;                        // wide: rows on 16 bytes
    uint16_t first[kFfMaxPairs + 1], slot[2 * kFfMaxPairs];
};

// The shares of a tile (blockIdx.y) added in order, and its results; a thread four
// columns of a row (forward: of the gate and of the up half).  The backward's two
// products are joined together (the first's tiles before the second's).
template <bool FWD, bool F32>
__global__ void __launch_bounds__(256) ff_join_kernel(const __grid_constant__ FfShares a, const __grid_constant__ FfShares b) {
    constexpr int Q = (FWD ? 128 : 256) / 4, HALVES = FWD ? 2 : 1;   // threads of a row
    wait_previous();
    const bool second = !FWD && (int)blockIdx.y >= a.tiles;   // dWg, dWu
    const FfShares &p = second ? b : a;
    const int t = (int)blockIdx.y - (second ? a.tiles : 0);
    const int id = blockIdx.x * 256 + threadIdx.x, c = id % Q * 4, r = id / Q;
    int tm, tn;
    ff_tile(p.whole + t, p.tiles_m, p.tiles_n, tm, tn);
    const int64_t row = (int64_t)tm * 256 + r;
    if (row >= p.rows || (!FWD && c >= p.width)) return;   // (whose sums were not stored)
    float y[2][4] = {};
    const int end = p.first[t + 1];
#pragma unroll 4
    for (int k = p.first[t]; k < end; ++k) {
        const float *src = p.partial + (int64_t)p.slot[k] * kTileFloats + r * 256 + c;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            const float4 v = *reinterpret_cast<const float4 *>(src + 128 * h);
            y[h][0] += v.x;
            y[h][1] += v.y;
            y[h][2] += v.z;
            y[h][3] += v.w;
        }
    }
    const int which = second && 2 * tn >= p.tiles_n;
    const int64_t col = (int64_t)(tn - (which ? p.tiles_n / 2 : 0)) * (FWD ? 4 * Q : p.width) + c;
    using T = std::conditional_t<F32, float, __nv_bfloat16>;
    auto store = [&](void *base, const float *x) {
        T *dst = static_cast<T *>(base) + row * p.cols + col;
        if (p.wide) {
            if (col >= p.cols) return;
            if constexpr (F32) *reinterpret_cast<float4 *>(dst) = make_float4(x[0], x[1], x[2], x[3]);
            else *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
            return;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (col + k < p.cols) dst[k] = from_f32<T>(x[k]);
    };
    if (FWD) {
        float o[4];
        ff_with_act(p.act, [&](auto f) {
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = f(y[0][k]) * y[1][k];
        });
        store(p.out[0], o);
        if (p.out[1]) {
            store(p.out[1], y[0]);
            store(p.out[2], y[1]);
        }
    } else {
        store(p.out[which], y[0]);
    }
}

struct FfPlan {
    int64_t tiles_m, tiles_n, kb, kb_seg, tiles;
    int width, pairs, whole;
    bool split;
};
template <FfMode MODE> FfPlan ff_plan(int64_t T, int64_t F, int64_t M, bool f32) {
    FfPlan q{};
    q.width = FfCfg<MODE, false>::BN;
    auto div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    if (MODE == FfMode::FWD) {
        q.tiles_m = div(T, 256);
        q.tiles_n = div(M, 128);
        q.kb = q.kb_seg = div(F, 64);
    } else if (MODE == FfMode::DX) {
        q.tiles_m = div(T, 256);
        q.tiles_n = div(F, 256);
        // Tiles no wider than the columns' even shares, in whole blocks of what the
        // epilogue stores at a time.  (B lies along the depth here; across it, its
        // columns come in 64s a CTA.)  Backward, 256 wide and so: 4099 x 301 x 803 fp32
        // (two of 160) 101 : 94 us, 20000 x 32 x 128 fp32 (32) 63 : 57, 20000 x 520 x
        // 1300 bf16 (three of 192) 213 : 207.
        const int64_t block = f32 ? 32 : 64;
        q.width = (int)(div(div(F, q.tiles_n), block) * block);
        q.kb_seg = div(M, 64);
        q.kb = 2 * q.kb_seg;
    } else {
        q.tiles_m = div(F, 256);
        q.tiles_n = 2 * div(M, 256);
        q.kb = q.kb_seg = div(T, 64);
    }
    q.tiles = q.tiles_m * q.tiles_n;
    const int most = std::max(1, std::min(device_sms() / 2, kFfMaxPairs));
    q.pairs = (int)std::min<int64_t>(most, q.tiles);
    q.whole = (int)std::min<int64_t>(q.tiles, INT32_MAX);
    const int64_t rest = q.tiles % most;
    // Sharing the last round takes its k-blocks from kb to about rest kb / pairs, at the
    // cost of writing and reading the sums and a launch more: some 40 k-blocks, 20 where
    // a tile has few rows (in fp32, six products of parts a k-block, 8).  Shared : whole,
    // us: 2708 x 256 x 680 bf16 dWg, dWu (6 tiles of 43) 27.7 : 24.7; 4099 x 301 x 803 fp32
    // backward, whose dX has 34 of 26, 94 : 110; 16 x 4096 x 4096 bf16 forward (32 of 64)
    // 22.2 : 25.5; 16384 x 1024 x 2816 bf16 backward (28 of 88 and 12 of 256) 295 : 354.
    const int64_t cost = f32 ? 8 : (MODE == FfMode::DW ? F : T) <= 128 ? 20 : 40;
    if (rest && q.kb - (rest * q.kb + most - 1) / most > cost) {
        q.split = true;
        q.pairs = most;
        q.whole = (int)(q.tiles - rest);
    }
    return q;
}

}  // namespace

// Launches the product; what is left to join is noted in `shares`.
template <FfMode MODE, bool F32> cudaError_t ff_product(const FfProduct &a, FfShares &shares, cudaStream_t s) {
    using C = FfCfg<MODE, F32>;
    static_assert(C::BYTES + 1024 + 256 <= 227 * 1024, "shared memory");
    const FfPlan q = ff_plan<MODE>(a.T, a.F, a.M, F32);
    FfParams p{};
    cudaError_t e = cudaSuccess;
    auto operand = [&](CUtensorMap (&maps)[3], const FfMatrix &m, bool mn, uint32_t box = 128) {
        for (int i = 0; i < C::PARTS && e == cudaSuccess; ++i)
            e = bf16_tensor_map(&maps[i], m.p + i * m.part_elems(), m.rows, m.cols, m.ld, 64, mn ? 64 : box);
    };
    if (MODE == FfMode::FWD) {
        operand(p.ta[0], a.x, false);
        operand(p.tb[0], a.wg, true);
        operand(p.tb[1], a.wu, true);
        p.rows = a.T;
        p.cols = a.M;
        p.out[0] = a.out;
        p.out[1] = a.g;
        p.out[2] = a.u;
    } else if (MODE == FfMode::DX) {
        operand(p.ta[0], a.dg, false);
        operand(p.ta[1], a.du, false);
        operand(p.tb[0], a.wg, false, q.width / 2);
        operand(p.tb[1], a.wu, false, q.width / 2);
        p.rows = a.T;
        p.cols = a.F;
        p.out[0] = a.out;
    } else {
        operand(p.ta[0], a.x, true);
        operand(p.tb[0], a.dg, true);
        operand(p.tb[1], a.du, true);
        p.rows = a.F;
        p.cols = a.M;
        p.out[0] = a.g;
        p.out[1] = a.u;
    }
    p.tma_out = p.cols * (F32 ? 4 : 2) % 16 == 0;
    if (!F32 && p.tma_out)
        for (int i = 0; i < 3 && e == cudaSuccess; ++i)
            if (p.out[i]) e = bf16_tensor_map(&p.to[i], static_cast<const __nv_bfloat16 *>(p.out[i]), p.rows, p.cols, p.cols, 64, 32);
    if (e == cudaSuccess) e = allow_smem<ff_gemm_kernel<MODE, F32>>(C::BYTES + 1024);
    if (e != cudaSuccess) return e;
    p.partial = a.partial;
    p.tiles_m = (int)q.tiles_m;
    p.tiles_n = (int)q.tiles_n;
    p.width = q.width;
    p.kb = (int)q.kb;
    p.kb_seg = (int)q.kb_seg;
    // bf16: the 1024 additions of 16384 products' sum drop at most 2^-13 of it, half of
    // that where its terms are alike; a bf16 result is rounded by up to 2^-8 then.
    p.depth = F32 ? 1 : 256;
    p.pairs = q.pairs;
    p.whole = q.whole;
    p.act = a.act;
    const sga_kernel_id id = MODE == FfMode::FWD ? SGA_KERN_FF_FWD : MODE == FfMode::DX ? SGA_KERN_FF_DX : SGA_KERN_FF_DW;
    note_launch(id, s, false);
    e = launch_early(ff_gemm_kernel<MODE, F32>, dim3(2 * (unsigned)q.pairs), dim3(kFfThreads), C::BYTES + 1024, s, p);
    note_launch(id, s, true);
    if (e != cudaSuccess || !q.split) return e;
    shares.partial = p.partial;
    for (int i = 0; i < 3; ++i) shares.out[i] = p.out[i];
    shares.rows = p.rows;
    shares.cols = p.cols;
    shares.tiles_m = p.tiles_m;
    shares.tiles_n = p.tiles_n;
    shares.width = p.width;
    shares.whole = p.whole;
    shares.tiles = (int)(q.tiles - q.whole);   // (less than the pairs)
    shares.act = p.act;
    shares.wide = p.tma_out;
    int n = 0, begun = 0;   // shares, tiles that have one
    for (int pair = 0; pair < q.pairs; ++pair) {   // (end to end: the tiles and their k-blocks in order)
        const FfUnits units((int)q.tiles, q.whole, (int)q.kb, q.pairs, pair);
        FfUnit u;
        for (int i = units.full; units.get(i, u); ++i) {
            if (u.tile - q.whole == begun) shares.first[begun++] = (uint16_t)n;
            shares.slot[n++] = (uint16_t)u.slot;
        }
    }
    shares.first[shares.tiles] = (uint16_t)n;
    return e;
}

// Joins what one product (forward), or two, left.
template <bool FWD, bool F32> cudaError_t ff_join(const FfShares &a, const FfShares &b, cudaStream_t s) {
    if (a.tiles + b.tiles == 0) return cudaSuccess;
    note_launch(SGA_KERN_FF_JOIN, s, false);
    const cudaError_t e = launch_early(ff_join_kernel<FWD, F32>, dim3(FWD ? 32 : 64, (unsigned)(a.tiles + b.tiles)), dim3(256), 0, s, a, b);
    note_launch(SGA_KERN_FF_JOIN, s, true);
    return e;
}

}  // namespace sga
