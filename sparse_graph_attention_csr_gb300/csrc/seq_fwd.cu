// Packed-sequence attention forward on the tcgen05 tensor cores (bf16).
//
// A CTA takes one unit: NS row tiles of 128 queries (NS = 2: two query heads
// that share a key head, or two neighbouring tiles of one head) and the key
// tiles they see.
//   warp 0, one lane: TMA loads -- the query tiles, then K and V tiles of 128
//     keys in turn into a ring;
//   warp 1: the products, in the order P V (previous key tile), S =
//     Q K^T of one query tile, then of the other: while the softmax warps of
//     one tile work, the tensor core has the other tile's products;
//   (warps 2, 3 idle: registers are split by groups of four warps)
//   warps 4 .. : four softmax warps a query tile (thread = query row = TMEM
//     lane): online softmax with a lazily moved maximum (O is rescaled in TMEM
//     only when the maximum grows by more than 2^8, so weights stay below
//     2^8), the weights rounded to bf16 and written over the scores in TMEM,
//     from where they are the A operand of P V; and the epilogue.
// S of the next key tile is issued behind P V of the last one, so its arrival
// also tells the softmax warps that O may be rescaled.  The row sum is taken of
// the unrounded fp32 weights; rounding P (half a bf16 step relative, 2^-8) is
// of the size of the rounding of the output itself.
//
// A zero weight times an infinity or NaN is NaN, so a tile that is masked in
// part could carry one from a value row that the query does not see.  What is not
// finite in a row for such a value row is computed again by its warp over its own
// interval alone (seq_rows.cuh; nothing is spent on this otherwise).
//
// Measured: 16384 rows, 8/2 heads of 128, causal 357 us (1.54 PFLOP/s; the
// library's product of 8192^3 reaches 1.90 in a burst and 1.70 under the power
// limit, which holds the clock down here too: 16384 rows, 8 heads, full 1.42).
// A pair of key-tile steps takes about 2900 cycles of which the products are
// 2048; what is left is a tile's own chain (scores read, maximum, 128
// exponentials, weights written, two handoffs of about 120 cycles, P V and S).
// Tried and slower at D = 128: P handed over in two halves (377 us), all eight
// warps on each tile in turn with the two halves of a row exchanging maxima
// (373 us).  D = 64: 8192 rows, 8 heads, causal 80 us (0.86 PFLOP/s), the chain
// again, beside half the products.
//
// Every wait is bounded; a timeout sets the plan's error word and ends the role.
#include <algorithm>

#include "seq_rows.cuh"
#include "seq_tc.cuh"
#include "tc_dx.cuh"

namespace sga {
namespace {

template <int D, int NS> struct FwdCfg {
    static constexpr int DP = D < 64 ? 64 : D;             // head width in shared memory and TMEM
    static constexpr int DA = DP / 64;
    static constexpr uint32_t TB = DA * 128 * 128;         // a tile of 128 rows
    static constexpr int NST = NS == 2 ? (DP == 64 ? 8 : 5) : (DP == 64 ? 5 : 2);   // K and V tiles in flight
    static constexpr uint32_t Q0 = 0, ST0 = NS * TB;
    static constexpr uint32_t BYTES = ST0 + NST * TB;
    static constexpr int THREADS = 128 + 128 * NS;
    // Registers a thread at launch, and after the split: the softmax warps hold
    // a row of 128 scores.  The shares add up to the launch's total.
    static constexpr int R_LAUNCH = NS == 2 ? 168 : 128, R_CTRL = NS == 2 ? 56 : 40, R_SOFT = NS == 2 ? 224 : 216;
    static_assert(R_CTRL + NS * R_SOFT == (NS + 1) * R_LAUNCH, "register split");
    static constexpr uint32_t TCOLS = NS == 2 ? 512 : 256;
    static constexpr uint32_t TS = 0, TO = NS * 128;       // scores of stage s at 128 s, O behind them
};

struct FwdParams {
    CUtensorMap tq, tk, tv;
    SeqArgs a;
    int pair_heads;   // NS = 2: the two tiles are two heads of one row tile
};

template <int D, int NS>
__global__ void __launch_bounds__(FwdCfg<D, NS>::THREADS, NS == 2 ? 1 : 2)
    seq_fwd_kernel(const __grid_constant__ FwdParams prm) {
    using C = FwdCfg<D, NS>;
    const SeqArgs &a = prm.a;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t q_full, kv_full[C::NST], kv_empty[C::NST], s_full[NS], p_full[NS], o_full[NS], mma_done;
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
    const uint32_t sbase = tc::smem_u32(smem);

    // the unit: per stage a row tile (with its key tiles) and a head
    SeqTile st[NS];
    int head[NS];
    if (NS == 2 && !prm.pair_heads) {
        const SeqTile *p = a.qpairs + 2 * (blockIdx.x / a.H);
        st[0] = p[0];
        st[NS - 1] = p[1];
        head[0] = head[NS - 1] = blockIdx.x % a.H;
    } else {
        const int per = a.H / NS;
        st[0] = st[NS - 1] = a.qtiles[blockIdx.x / per];
        head[0] = (blockIdx.x % per) * NS;
        head[NS - 1] = head[0] + NS - 1;
    }
    const int hk = head[0] / (a.H / a.Hkv);
    const int t0 = min(st[0].t0, st[NS - 1].t0), t1 = max(st[0].t1, st[NS - 1].t1), n = t1 - t0;

    if (tid == 32) {
        tc::mbar_init(&q_full, 1);
        for (int i = 0; i < C::NST; ++i) {
            tc::mbar_init(&kv_full[i], 1);
            tc::mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < NS; ++i) {
            tc::mbar_init(&s_full[i], 1);
            tc::mbar_init(&p_full[i], 4);
            tc::mbar_init(&o_full[i], 1);
        }
        tc::mbar_init(&mma_done, 1);
    }
    wait_previous();
    if (warp == 0) tc::tmem_alloc(&tmem_base, C::TCOLS);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    let_next_start();
    const uint32_t tS = tmem_base + C::TS, tO = tmem_base + C::TO;

    if (warp < 4) {
        tc::reg_dec<C::R_CTRL>();
        if (warp == 0 && lane == 0) {   // ----------------------------------- TMA producer
            bool ok = true;
            tc::mbar_expect_tx(&q_full, NS * C::TB);
#pragma unroll
            for (int s = 0; s < NS; ++s)
                seq::load_tile<C::DA>(sbase + C::Q0 + s * C::TB, &prm.tq, head[s], st[s].tile * 128, &q_full);
            int e = 0;
            for (; e < 2 * n; ++e) {
                const int b = e % C::NST, r = e / C::NST;
                if (r >= 1 && !tc::mbar_wait(&kv_empty[b], (r - 1) & 1, tc::kWaitLimit)) {
                    ok = false;
                    break;
                }
                tc::mbar_expect_tx(&kv_full[b], C::TB);
                seq::load_tile<C::DA>(sbase + C::ST0 + b * C::TB, (e & 1) ? &prm.tv : &prm.tk, hk, (t0 + (e >> 1)) * 128,
                                      &kv_full[b]);
            }
            if (!ok) atomicOr(a.d_err, tc::kErrMmaTimeout);
            // loads that no product consumed (only after a timeout) land before the CTA ends
            tc::mbar_wait(&q_full, 0, tc::kWaitLimit);
            for (int i = e - 1; i >= 0 && i >= e - C::NST; --i)
                tc::mbar_wait(&kv_full[i % C::NST], (i / C::NST) & 1, tc::kWaitLimit);
        } else if (warp == 1) {   // ----------------------------------------- MMA issuer (the warp in step)
            constexpr uint32_t idesc_s = tc::idesc_bf16(128, 128), idesc_o = tc::idesc_bf16(128, C::DP) | tc::kMajorMnB;
            int pend[NS], np[NS];   // key tile whose P V is due, and P V's issued, per stage
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                pend[s] = -1;
                np[s] = 0;
            }
            auto issue_pv = [&](int s) -> bool {   // O(s) += P(s) V(pend[s])
                const int e = 2 * pend[s] + 1, b = e % C::NST;
                // (V first: it has landed, and the poll is done while P is formed)
                if (!tc::warp_wait(&kv_full[b], (e / C::NST) & 1, tc::kWaitLimit) ||
                    !tc::warp_wait(&p_full[s], np[s] & 1, tc::kWaitLimit))
                    return false;
                tc::fence_after_sync();
                const uint32_t va = sbase + C::ST0 + b * C::TB;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    tc::mma_bf16_ts_w(tO + s * C::DP, tS + s * 128 + kk * 8, tc::desc_sw128_mn(va + kk * 2048, 16384),
                                    idesc_o, (np[s] > 0 || kk > 0) ? 1u : 0u);
                ++np[s];
                if (t0 + pend[s] == st[s].t1 - 1) tc::mma_commit_w(&o_full[s]);
                pend[s] = -1;
                return true;
            };
            bool ok = tc::warp_wait(&q_full, 0, tc::kWaitLimit);
            for (int i = 0; i < n && ok; ++i) {
                const int e = 2 * i, b = e % C::NST;
                if (!tc::warp_wait(&kv_full[b], (e / C::NST) & 1, tc::kWaitLimit)) {
                    ok = false;
                    break;
                }
                const uint32_t ka = sbase + C::ST0 + b * C::TB;
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    if (!ok) break;
                    if (pend[s] >= 0 && !issue_pv(s)) {
                        ok = false;
                        break;
                    }
                    if (t0 + i < st[s].t0 || t0 + i >= st[s].t1) continue;
                    tc::fence_after_sync();
                    const uint32_t qa = sbase + C::Q0 + s * C::TB;
#pragma unroll
                    for (int kk = 0; kk < C::DP / 16; ++kk) {
                        const uint32_t o = (uint32_t)((kk >> 2) * 16384 + (kk & 3) * 32);
                        tc::mma_bf16_ss_w(tS + s * 128, tc::desc_sw128(qa + o), tc::desc_sw128(ka + o), idesc_s, kk > 0);
                    }
                    tc::mma_commit_w(&s_full[s]);
                    pend[s] = i;
                }
                if (!ok) break;
                tc::mma_commit_w(&kv_empty[b]);
                if (i >= 1) tc::mma_commit_w(&kv_empty[(e - 1) % C::NST]);
            }
#pragma unroll
            for (int s = 0; s < NS; ++s)
                if (ok && pend[s] >= 0 && !issue_pv(s)) ok = false;
            if (!ok && lane == 0) atomicOr(a.d_err, tc::kErrMmaTimeout);
            // every product issued is complete before TMEM is released
            tc::mma_commit_w(&mma_done);
            tc::warp_wait(&mma_done, 0, tc::kWaitLimit);
        }
        __syncwarp();
    } else {   // ---------------------------------------------------- softmax + epilogue
        tc::reg_inc<C::R_SOFT>();
        const int s = NS == 2 ? (warp - 4) >> 2 : 0, quarter = warp & 3;   // TMEM lanes 32 * (warp % 4) ..
        const uint32_t tl = (uint32_t)(quarter * 32) << 16;
        const SeqTile t = s ? st[NS - 1] : st[0];
        const int h = s ? head[NS - 1] : head[0];
        const int64_t row = (int64_t)t.tile * 128 + quarter * 32 + lane;
        const bool in = row < a.rows;
        int64_t lo = 0, hi = 0;   // the keys that the row sees
        if (in) {
            const int2 se = __ldg(a.range + row);
            lo = se.x;
            hi = a.causal ? row + 1 : se.y;
        }
        const float scale2 = a.scale * kLog2e;
        const uint32_t ts = tS + s * 128 + tl, to = tO + s * C::DP + tl;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int kt = t.t0; kt < t.t1; ++kt) {
            if (!tc::warp_wait(&s_full[s], (kt - t.t0) & 1, tc::kWaitLimit)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            uint32_t v[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tc::tmem_ld32_async(ts + 32 * c, v + 32 * c);
#pragma unroll
            for (int c = 0; c < 4; ++c) tc::tmem_wait_ld(v + 32 * c);
            if (kt < t.f0 || kt >= t.f1) {
                const int cl = seq::rel(lo, (int64_t)kt * 128), ch = seq::rel(hi, (int64_t)kt * 128);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t bits = seq::column_bits(cl, ch, w);
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!((bits >> c) & 1u)) v[32 * w + c] = 0xff800000u;   // -inf
                }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 128; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(v[c]));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale2;
            const bool grow = top > m + kLazyLog2;   // (also from m = -inf)
            const bool move = grow && l > 0.f;
            const float mn = grow ? top : m;
            if (__any_sync(SGA_FULL_MASK, move)) {
                const float f = move ? exp2_diff(m, mn) : 1.f;
                l *= f;
                for (int cb = 0; cb < D; cb += 32) {
                    uint32_t o[32];
                    tc::tmem_ld32(to + cb, o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    tc::tmem_st32_async(to + cb, o);
                }
            }
            m = mn;
            const float sub = m == -INFINITY ? 0.f : m;   // nothing seen yet: every weight is zero
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 k2 = make_float2(scale2, scale2), s2 = make_float2(-sub, -sub);
#pragma unroll
            for (int c = 0; c < 128; c += 2) {
                float2 x = ffma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), k2, s2);
                x.x = fast_exp2(x.x);
                x.y = fast_exp2(x.y);
                sum[(c >> 1) & 1] = fadd2(sum[(c >> 1) & 1], x);
                v[c >> 1] = pack_bf16x2(x.x, x.y);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            tc::tmem_st32_async(ts, v);
            tc::tmem_st32_async(ts + 32, v + 32);
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&p_full[s]);
        }
        const bool any = t.t0 < t.t1;   // (the second tile of a pair may be missing)
        if (ok && any && !tc::warp_wait(&o_full[s], 0, tc::kWaitLimit)) ok = false;
        if (ok && any) {
            tc::fence_after_sync();
            const float inv = 1.f / l;
            bool bad = false;
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out_w) + ((in ? row : 0) * a.H + h) * D;
#pragma unroll
            for (int cb = 0; cb < D; cb += 32) {
                uint32_t o[32];
                tc::tmem_ld32(to + cb, o);
                float x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    x[i] = __uint_as_float(o[i]) * inv;
                    bad |= !(fabsf(x[i]) < INFINITY);
                }
                if (in)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint4 *>(out + cb + 8 * q) = pack<__nv_bfloat16>(x + 8 * q);
            }
            if (in) a.lse_w[row * a.H + h] = (m + log2f(l)) * kLn2;
            uint32_t again = __ballot_sync(SGA_FULL_MASK, bad && in && l == l);
            __syncwarp();   // (the rows are read back)
            while (again) {
                const int src = __ffs(again) - 1;
                again &= again - 1;
                const seq::Span sp{__shfl_sync(SGA_FULL_MASK, lo, src), __shfl_sync(SGA_FULL_MASK, hi, src), (int64_t)t.t0 * 128,
                                   min(a.rows, (int64_t)t.t1 * 128)};
                seq::out_row_alone<__nv_bfloat16, D>(a, __shfl_sync(SGA_FULL_MASK, row, src), h, hk, sp);
            }
            tc::fence_before_sync();
        } else if (!ok && lane == 0) {
            atomicOr(a.d_err, tc::kErrMmaTimeout);
        }
    }
    // the MMA lane waited for all its products, the producer for its loads
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc::tmem_dealloc(tmem_base, C::TCOLS);
    }
}

template <int D, int NS> cudaError_t launch(const SeqArgs &a, cudaStream_t s) {
    using C = FwdCfg<D, NS>;
    static_assert(C::BYTES + 1024 <= (NS == 2 ? 226 : 113) * 1024, "shared memory");
    FwdParams prm{};
    prm.a = a;
    prm.pair_heads = NS == 2 && a.H / a.Hkv % 2 == 0;
    cudaError_t e = seq_tensor_map(&prm.tq, a.Q, a.rows, a.H, D);
    if (e == cudaSuccess) e = seq_tensor_map(&prm.tk, a.K, a.rows, a.Hkv, D);
    if (e == cudaSuccess) e = seq_tensor_map(&prm.tv, a.V, a.rows, a.Hkv, D);
    if (e == cudaSuccess) e = allow_smem<seq_fwd_kernel<D, NS>>(C::BYTES + 1024);
    if (e != cudaSuccess) return e;
    const int64_t units = NS == 1 ? (int64_t)a.n_tiles * a.H
                          : prm.pair_heads ? (int64_t)a.n_tiles * (a.H / 2)
                                           : (int64_t)((a.n_tiles + 1) / 2) * a.H;
    note_launch(SGA_KERN_SEQ_FWD, s, false);
    e = launch_early(seq_fwd_kernel<D, NS>, dim3((unsigned)units), dim3(C::THREADS), C::BYTES + 1024, s, prm);
    note_launch(SGA_KERN_SEQ_FWD, s, true);
    return e;
}

}  // namespace

cudaError_t seq_tensor_map(CUtensorMap *m, const void *base, int64_t rows, int heads, int D) {
    PFN_cuTensorMapEncodeTiled_v12000 encode;
    if (cudaError_t e = tmap_encoder(encode); e != cudaSuccess) return e;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)heads * D * 2};
    const cuuint32_t box[3] = {64, 1, 128}, estr[3] = {1, 1, 1};
    const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t seq_fwd_bf16(const SeqArgs &a, int D, cudaStream_t s) {
    // One row tile a CTA (two CTAs an SM) or two.  Two tiles share the key
    // tiles' loads and give the tensor core work while one of them waits; one
    // tile a CTA spreads few units over more SMs and ends more evenly.
    // Measured, one : two tiles a CTA, D = 128, causal: 2048 rows, 8/2 heads
    // (128 tiles) 31 : 35 us; 4096 (256) 54.5 : 55.7; 8192 (512) 117 : 103.
    // D = 64: causal 4096 rows, 8 heads 43 : 48, 8192 80 : 84; full 4096 rows,
    // 16 heads 92 : 88.
    const bool one = (int64_t)a.n_tiles * a.H <= 2 * (int64_t)a.num_sms || (D <= 64 && a.causal);
    if (D == 32) return one ? launch<32, 1>(a, s) : launch<32, 2>(a, s);
    if (D == 64) return one ? launch<64, 1>(a, s) : launch<64, 2>(a, s);
    return one ? launch<128, 1>(a, s) : launch<128, 2>(a, s);
}

}  // namespace sga
