// Packed-sequence attention backward on the tcgen05 tensor cores (bf16).
//
//   P = exp(S - lse), dP = dOut V^T, dS = P (dP - Delta),
//   dV = P^T dOut, dK = scale dS^T Q, dQ = scale dS K
//
// Two passes (in one launch), so that every output row is owned by one CTA: no atomics, no
// fp32 copy of dQ in memory, bitwise reproducible; S and dP are computed twice
// (seven products a tile pair instead of five).
//   dK/dV pass (unit: 128 keys x key head, over the query tiles that see them
//     and the heads of the group): S^T = K Q^T and dP^T = V dOut^T with keys in
//     the TMEM lanes, P^T and dS^T written back to TMEM in bf16 over the scores
//     they come from, where they are the A operands of dV += P^T dOut and
//     dK += dS^T Q.  The products are issued dV(i), S(i + 1), dK(i), dP(i + 1):
//     while the weights of i + 1 are formed the tensor core has dK(i) and
//     dP(i + 1), while its dS is formed it has dV(i + 1) and S(i + 2).
//   dQ pass (unit: 128 queries x head, over the key tiles they see): S and dP
//     with queries in the lanes, Q and dOut as A operands in TMEM (as shared
//     memory operands they would take half of its bandwidth, and with the loads
//     more than there is), dS in bf16 over dP, dQ += dS K; issued S(i + 1),
//     dQ(i), dP(i + 1): the weights of i + 1 are formed while dQ(i) and
//     dP(i + 1) are computed.
// Roles as in the forward: one lane loads by TMA, one issues the products,
// eight warps (two per TMEM lane quarter, each with half of a tile's columns)
// turn scores into weights.  P and dS are rounded to bf16 once (half a step,
// 2^-8 relative), which is of the size of the rounding of the gradients; in dQ,
// whose terms cancel where the keys share an offset, the sum of the roundings is
// taken out again (at the dQ pass).
//
// As in the forward, what is not finite in a row for a row that is masked for it
// is computed again over its own interval alone.
// Measured: 8192 rows, 8/4 heads of 128, causal 310 us, full 580 us: 1.18
// PFLOP/s of the five products that a backward pass needs, 1.66 of the seven
// computed (the library's product under the power limit: 1.70).
// What is left to gain is the two repeated products, against an fp32 dQ in
// memory that several CTAs add to.
//
// Every wait is bounded; a timeout sets the plan's error word and ends the role.
#include <algorithm>

#include "seq_rows.cuh"
#include "seq_tc.cuh"

namespace sga {
namespace {

// Control warps (load, MMA, two idle) and two weight warps a TMEM lane quarter,
// each with 64 of a tile's columns (four with 32 each measured the same at D =
// 128 and 2% slower at D = 64).  Registers a thread at launch and after the split.
constexpr int kParts = 2, kCols = 128 / kParts;
constexpr int kSoft = 4 * kParts;   // arrivals per handoff
constexpr int kThreads = 128 + 128 * kParts;
constexpr int kRLaunch = 168, kRCtrl = 56, kRSoft = 224;
static_assert(kRCtrl + kParts * kRSoft <= (kParts + 1) * kRLaunch, "register split");

template <int D> struct BwdCfg {
    static constexpr int DP = D < 64 ? 64 : D, DA = DP / 64;
    static constexpr uint32_t TB = DA * 128 * 128;    // a tile of 128 rows
    static constexpr uint32_t R0 = 0;                 // two resident tiles
    static constexpr uint32_t ST0 = 2 * TB;           // ring of streamed tiles
};
// The streamed tiles have a ring each: of the two that a step takes, one is
// held longer than the other (Q until dK, K until dQ), and a common ring would
// make the next loads wait for it.
template <int D> struct KvCfg : BwdCfg<D> {
    using B = BwdCfg<D>;
    static constexpr int NQ = B::DP == 64 ? 4 : 3, NG = B::DP == 64 ? 4 : 2;   // Q, dOut tiles in flight
    static constexpr uint32_t G0 = B::ST0 + NQ * B::TB;
    static constexpr uint32_t ROW0 = G0 + NG * B::TB;                         // -lse, -Delta of a step's queries: two slots
    static constexpr uint32_t BAR0 = ROW0 + 2 * 1024, BYTES = BAR0 + 256;     // barriers
    static constexpr uint32_t TS = 0, TP = 128, TK = 256, TV = 256 + B::DP;   // S^T, dP^T, dK, dV
};
template <int D> struct QCfg : BwdCfg<D> {
    using B = BwdCfg<D>;
    static constexpr int NK = 4, NV = 3;                          // K, V tiles in flight
    static constexpr uint32_t ST0 = 0, V0 = ST0 + NK * B::TB;
    static constexpr uint32_t RES0 = V0 + NV * B::TB;             // sums of a row's rounding errors, by part
    static constexpr uint32_t BAR0 = RES0 + kParts * 512, BYTES = BAR0 + 256;   // barriers
    static constexpr uint32_t TS = 0, TP = 128, TQ = 256, TA = 384, TG = 448;   // S, dP, dQ; Q and dOut as A operands
};
constexpr uint32_t kMaxSmem = 227 * 1024;
static_assert(KvCfg<128>::BYTES <= kMaxSmem && QCfg<128>::BYTES <= kMaxSmem, "shared memory");

// A ring of N tiles in shared memory from `base`.
template <int N, uint32_t TB> struct Ring {
    uint64_t *full, *empty;
    uint32_t base;
    __device__ __forceinline__ uint32_t at(int i) const { return base + (i % N) * TB; }
    __device__ __forceinline__ uint64_t *filled(int i) const { return &full[i % N]; }
    __device__ __forceinline__ uint64_t *freed(int i) const { return &empty[i % N]; }
    __device__ __forceinline__ bool wait_filled(int i) const { return tc::warp_wait(&full[i % N], (i / N) & 1, tc::kWaitLimit); }
    // (one lane) room for tile i
    __device__ __forceinline__ bool wait_room(int i) const {
        return i < N || tc::mbar_wait(&empty[i % N], (i / N - 1) & 1, tc::kWaitLimit);
    }
    // (one lane) the last loads, of `n` issued, have landed
    __device__ __forceinline__ void drain(int n) const {
        for (int i = n - 1; i >= 0 && i >= n - N; --i) tc::mbar_wait(&full[i % N], (i / N) & 1, tc::kWaitLimit);
    }
    __device__ __forceinline__ void init() const {
        for (int i = 0; i < N; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
    }
};

struct BwdParams {
    CUtensorMap tq, tk, tv, tg;
    SeqArgs a;
};

// A 128-deep product with the A operand in TMEM, written over scores by the
// weight warps (their parts kCols columns apart, half as many columns of bf16
// pairs each), and 128 rows of B as an MN-major operand.
__device__ __forceinline__ void mma_rows128(uint32_t d, uint32_t ta, uint32_t b, uint32_t idesc, bool first) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
        tc::mma_bf16_ts_w(d, ta + kk * kParts / 8 * kCols + kk % (8 / kParts) * 8, tc::desc_sw128_mn(b + kk * 2048, 16384), idesc,
                        (!first || kk > 0) ? 1u : 0u);
}
// 128 x 128 over the head width, both operands K-major tiles of 128 rows.
template <int DP> __device__ __forceinline__ void mma_over_d(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
        const uint32_t o = (uint32_t)((kk >> 2) * 16384 + (kk & 3) * 32);
        tc::mma_bf16_ss_w(d, tc::desc_sw128(a + o), tc::desc_sw128(b + o), idesc, kk > 0);
    }
}

// The same with the A operand a head's row in TMEM (bf16 pairs in order).
template <int DP> __device__ __forceinline__ void mma_over_d_ts(uint32_t d, uint32_t ta, uint32_t b, uint32_t idesc) {
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk)
        tc::mma_bf16_ts_w(d, ta + kk * 8, tc::desc_sw128(b + (uint32_t)((kk >> 2) * 16384 + (kk & 3) * 32)), idesc, kk > 0);
}

// This part's columns of scores of this thread's TMEM lane.
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t *v) {
    constexpr int N = kCols;
#pragma unroll
    for (int c = 0; c < N; c += 32) tc::tmem_ld32_async(taddr + c, v + c);
#pragma unroll
    for (int c = 0; c < N; c += 32) tc::tmem_wait_ld(v + c);
}
// The weights as bf16 pairs, over the first half of their scores' columns.
__device__ __forceinline__ void round_weights(const float *p, uint32_t *pk) {
#pragma unroll
    for (int c = 0; c < kCols; c += 2) pk[c >> 1] = pack_bf16x2(p[c], p[c + 1]);
}
__device__ __forceinline__ void store_weights(uint32_t taddr, const uint32_t *pk) {
    static_assert(kCols == 64, "one store of 32 columns");
    tc::tmem_st32_async(taddr, pk);
    tc::tmem_wait_st();
}
__device__ __forceinline__ void store_weights(uint32_t taddr, const float *p) {
    uint32_t pk[kCols / 2];
    round_weights(p, pk);
    store_weights(taddr, pk);
}

// 32 columns of a row from TMEM, less `sub` (if any), scaled, to bf16 at dst (if
// `in`); the lanes whose row was not finite.
__device__ __forceinline__ uint32_t store_from_tmem(uint32_t taddr, __nv_bfloat16 *dst, float f, bool in,
                                                    const float *sub = nullptr) {
    bool bad = false;
    uint32_t o[32];
    tc::tmem_ld32(taddr, o);   // warp-collective: every lane takes part
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        x[i] = (sub ? __uint_as_float(o[i]) - sub[i] : __uint_as_float(o[i])) * f;
        bad |= !(fabsf(x[i]) < INFINITY);
    }
    if (in)
#pragma unroll
        for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4 *>(dst + 8 * q) = pack<__nv_bfloat16>(x + 8 * q);
    return __ballot_sync(SGA_FULL_MASK, bad && in);
}

// ---- dK, dV -----------------------------------------------------------------------

template <int D> __device__ __forceinline__ void dkdv_pass(const BwdParams &prm, unsigned char *smem, uint32_t unit) {
    using C = KvCfg<D>;
    const SeqArgs &a = prm.a;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::BAR0);
    uint64_t &kv_full = bar[0], &s_full = bar[1], &dp_full = bar[2], &p_full = bar[3], &ds_full = bar[4], &acc_full = bar[5];
    uint32_t &tmem_base = *reinterpret_cast<uint32_t *>(bar + 6);
    uint64_t *ring_full = bar + 7, *ring_empty = ring_full + C::NQ + C::NG + 2;
    static_assert((7 + 2 * (C::NQ + C::NG + 2)) * 8 <= 256, "barriers");
    const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
    const uint32_t sbase = tc::smem_u32(smem);
    const Ring<C::NQ, C::TB> rq{ring_full, ring_empty, sbase + C::ST0};
    const Ring<C::NG, C::TB> rg{ring_full + C::NQ, ring_empty + C::NQ, sbase + C::G0};
    const Ring<2, 1024> rr{ring_full + C::NQ + C::NG, ring_empty + C::NQ + C::NG, sbase + C::ROW0};
    const SeqTile t = a.ktiles[unit / a.Hkv];
    const int hk = unit % a.Hkv, grp = a.H / a.Hkv;
    const int nt = t.t1 - t.t0, n = nt * grp;   // steps: (head of the group, query tile)

    if (tid == 32) {
        tc::mbar_init(&kv_full, 1);
        rq.init();
        rg.init();
        rr.init();
        tc::mbar_init(&s_full, 1);
        tc::mbar_init(&dp_full, 1);
        tc::mbar_init(&p_full, kSoft);
        tc::mbar_init(&ds_full, kSoft);
        tc::mbar_init(&acc_full, 1);
    }
    wait_previous();
    if (warp == 0) tc::tmem_alloc(&tmem_base, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tS = tmem_base + C::TS, tP = tmem_base + C::TP, tK = tmem_base + C::TK, tV = tmem_base + C::TV;

    if (warp < 4) {
        tc::reg_dec<kRCtrl>();
        if (warp == 0 && lane == 0) {   // ----------------------------------- TMA producer
            bool ok = true;
            tc::mbar_expect_tx(&kv_full, 2 * C::TB);
            seq::load_tile<C::DA>(sbase + C::R0, &prm.tk, hk, t.tile * 128, &kv_full);
            seq::load_tile<C::DA>(sbase + C::R0 + C::TB, &prm.tv, hk, t.tile * 128, &kv_full);
            int nq = 0, ng = 0, nr = 0;   // loads issued
            for (int i = 0; i < n; ++i) {
                const int hd = hk * grp + i / nt, row = (t.t0 + i % nt) * 128;
                if (!(ok = rq.wait_room(i))) break;
                tc::mbar_expect_tx(rq.filled(i), C::TB);
                seq::load_tile<C::DA>(rq.at(i), &prm.tq, hd, row, rq.filled(i));
                ++nq;
                if (!(ok = rg.wait_room(i))) break;
                tc::mbar_expect_tx(rg.filled(i), C::TB);
                seq::load_tile<C::DA>(rg.at(i), &prm.tg, hd, row, rg.filled(i));
                ++ng;
                if (!(ok = rr.wait_room(i))) break;
                tc::mbar_expect_tx(rr.filled(i), 1024);
                tc::bulk_load(rr.at(i), a.ws_nlse + (int64_t)hd * a.rows_pad + row, 512, rr.filled(i));
                tc::bulk_load(rr.at(i) + 512, a.ws_ndelta + (int64_t)hd * a.rows_pad + row, 512, rr.filled(i));
                ++nr;
            }
            if (!ok) atomicOr(a.d_err, tc::kErrMmaTimeout);
            // loads that no product consumed (only after a timeout) land before the CTA ends
            tc::mbar_wait(&kv_full, 0, tc::kWaitLimit);
            rq.drain(nq);
            rg.drain(ng);
            rr.drain(nr);
        } else if (warp == 1) {   // ----------------------------------------- MMA issuer (the warp in step)
            constexpr uint32_t idesc_s = tc::idesc_bf16(128, 128), idesc_g = tc::idesc_bf16(128, C::DP) | tc::kMajorMnB;
            const uint32_t ka = sbase + C::R0, va = ka + C::TB;
            auto scores = [&](int i) {   // S^T = K Q^T
                mma_over_d<C::DP>(tS, ka, rq.at(i), idesc_s);
                tc::mma_commit_w(&s_full);
            };
            auto dprod = [&](int i) {    // dP^T = V dOut^T
                mma_over_d<C::DP>(tP, va, rg.at(i), idesc_s);
                tc::mma_commit_w(&dp_full);
            };
            bool ok = tc::warp_wait(&kv_full, 0, tc::kWaitLimit) && rq.wait_filled(0) && rg.wait_filled(0);
            if (ok) {
                tc::fence_after_sync();
                scores(0);
                dprod(0);
            }
            for (int i = 0; i < n && ok; ++i) {
                // the next tiles have landed; their barriers are polled while the weights are formed
                if ((i + 1 < n && !(rq.wait_filled(i + 1) && rg.wait_filled(i + 1))) ||
                    !tc::warp_wait(&p_full, i & 1, tc::kWaitLimit)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                mma_rows128(tV, tS, rg.at(i), idesc_g, i == 0);   // dV += P^T dOut
                tc::mma_commit_w(rg.freed(i));
                if (i + 1 < n) scores(i + 1);
                if (!tc::warp_wait(&ds_full, i & 1, tc::kWaitLimit)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                mma_rows128(tK, tP, rq.at(i), idesc_g, i == 0);   // dK += dS^T Q
                tc::mma_commit_w(rq.freed(i));
                tc::mma_commit_w(rr.freed(i));   // (read before dS arrived)
                if (i + 1 < n) dprod(i + 1);
            }
            if (!ok && lane == 0) atomicOr(a.d_err, tc::kErrMmaTimeout);
            // every product issued is complete before TMEM is released
            tc::mma_commit_w(&acc_full);
            tc::warp_wait(&acc_full, 0, tc::kWaitLimit);
        }
        __syncwarp();
    } else {   // ---------------------------------------------------- weights and epilogue
        tc::reg_inc<kRSoft>();
        const int quarter = warp & 3, part = (warp - 4) >> 2;   // part: queries N part .. of a tile
        const uint32_t tl = (uint32_t)(quarter * 32) << 16;
        const int64_t row = (int64_t)t.tile * 128 + quarter * 32 + lane;
        const bool in = row < a.rows;
        int64_t lo = 0, hi = 0;   // the queries that see the key
        if (in) {
            const int2 se = __ldg(a.range + row);
            lo = a.causal ? row : se.x;
            hi = se.y;
        }
        const float scale2 = a.scale * kLog2e;
        const float2 k2 = make_float2(scale2, scale2);
        constexpr int N = kCols;
        const uint32_t ts = tS + part * N + tl, tp = tP + part * N + tl;
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int qt = t.t0 + i % nt;
            if (!rr.wait_filled(i)) {
                ok = false;
                break;
            }
            // the columns' -lse, read while the scores are computed
            float p[N], r[N];
#pragma unroll
            for (int c = 0; c < N; c += 4) tc::lds128(rr.at(i) + 4 * (part * N + c), r + c);
            if (!tc::warp_wait(&s_full, i & 1, tc::kWaitLimit)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            uint32_t v[N];
            load_scores(ts, v);
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                const float2 x = ffma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), k2,
                                       make_float2(r[c], r[c + 1]));
                p[c] = fast_exp2(x.x);
                p[c + 1] = fast_exp2(x.y);
            }
            const bool masked = qt < t.f0 || qt >= t.f1;
            uint32_t bits[N / 32];
            if (masked) {
                const int cl = seq::rel(lo, (int64_t)qt * 128), ch = seq::rel(hi, (int64_t)qt * 128);
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    if (c % 32 == 0) bits[c / 32] = seq::column_bits(cl, ch, (part * N + c) / 32);
                    if (!((bits[c / 32] >> (c & 31)) & 1u)) p[c] = 0.f;
                }
            }
            store_weights(ts, p);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&p_full);

#pragma unroll
            for (int c = 0; c < N; c += 4) tc::lds128(rr.at(i) + 512 + 4 * (part * N + c), r + c);   // the columns' -Delta
            if (!tc::warp_wait(&dp_full, i & 1, tc::kWaitLimit)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            load_scores(tp, v);
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                const float2 x = fmul2(make_float2(p[c], p[c + 1]),
                                       fadd2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                                             make_float2(r[c], r[c + 1])));
                p[c] = x.x;
                p[c + 1] = x.y;
            }
            if (masked)   // (zero weights times an infinity)
#pragma unroll
                for (int c = 0; c < N; ++c)
                    if (!((bits[c / 32] >> (c & 31)) & 1u)) p[c] = 0.f;
            store_weights(tp, p);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ds_full);
        }
        if (ok && !tc::warp_wait(&acc_full, 0, tc::kWaitLimit)) ok = false;
        if (ok) {
            tc::fence_after_sync();
            uint32_t again[2] = {0, 0};   // rows of dV, dK
            for (int c = part; c < D / 16; c += kParts) {   // 32 columns each: dV's, then dK's
                const bool dk = c >= D / 32;
                const int c0 = (dk ? c - D / 32 : c) * 32;
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(dk ? a.dK : a.dV) + ((in ? row : 0) * a.Hkv + hk) * D + c0;
                const uint32_t bad = store_from_tmem((dk ? tK : tV) + c0 + tl, dst, dk ? a.scale : 1.f, in);
                if (dk) again[1] |= bad;
                else again[0] |= bad;
            }
            __syncwarp();   // (the rows are read back)
#pragma unroll
            for (int dk = 0; dk < 2; ++dk)
                while (again[dk]) {
                    const int src = __ffs(again[dk]) - 1;
                    again[dk] &= again[dk] - 1;
                    const seq::Span sp{__shfl_sync(SGA_FULL_MASK, lo, src), __shfl_sync(SGA_FULL_MASK, hi, src), (int64_t)t.t0 * 128,
                                       min(a.rows, (int64_t)t.t1 * 128)};
                    seq::key_row_alone<__nv_bfloat16, D>(a, dk != 0, __shfl_sync(SGA_FULL_MASK, row, src), hk, sp,
                                                         seq::slice_columns<D>(dk * (D / 32), part, kParts));
                }
        } else if (lane == 0) {
            atomicOr(a.d_err, tc::kErrMmaTimeout);
        }
    }
    // the MMA lane waited for all its products, the producer for its loads
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc::tmem_dealloc(tmem_base, 512);
    }
}

// ---- dQ ----------------------------------------------------------------------------
//
// A row's dS sum to zero, so an offset that all keys share leaves no trace in dQ =
// sum_j dS_j k_j; but of dS rounded to bf16, dS_j + e_j, it leaves offset x sum_j
// e_j, which grows with the offset while dQ does not.  The weight warps know every
// e_j, so in a column with an offset dQ is formed as sum_j (dS_j + e_j) k_j - (sum_j
// e_j) c, c being the mean of four of the row's own keys: an error of sum_j e_j (k_j
// - c), in which the offset is gone.  Nothing is assumed of dS itself.  (A second
// product, of the e_j, would be the eighth of the two passes; what is left of dQ's
// error is then the forward's, whose rounded out enters Delta.)  512 keys of 64 +-
// 1, bf16, D = 64, queries of 1 / 64: dQ's error against the formula with that out
// is 0.0025 of its norm, and was 0.104 with single roundings.  It costs 2% at 8192
// rows, 8/4 heads of 128 (causal 303 -> 310 us), 5% at 8 heads of 64 (235 -> 251)
// and 1.7 us on 128 graphs of 9 to 38 rows, 4 heads of 64 (16.6 -> 18.3).  In dK =
// sum_i dS_i q_i the terms of a key's queries do not cancel: its roundings are of
// the size of dK's own.

// c at the columns [c0, c0 + 32) as bf16 pairs, zero in a column where the four
// are farther apart than |c| / 2 (no offset to speak of).  c lies between them:
// they are representable, and each rounding on the way to it is monotone.  Of
// eight keys and more rows of similar lengths take the same four, so that their
// loads are one.
__device__ __forceinline__ void mean_key(const SeqArgs &a, int D, int64_t lo, int64_t hi, int hk, int c0, uint32_t (&c)[16]) {
    const int64_t n = max(hi - lo, (int64_t)1), m = n < 8 ? n : (int64_t)1 << (31 - __clz((int)n));   // (n < 2^31)
    uint4 raw[4][4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.K) + ((lo + (m * (2 * s + 1) >> 3)) * a.Hkv + hk) * D + c0;
#pragma unroll
        for (int q = 0; q < 4; ++q) raw[s][q] = ldg16(k + 8 * q);
    }
    const __nv_bfloat162 fourth = __float2bfloat162_rn(0.25f), half = __float2bfloat162_rn(0.5f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        __nv_bfloat162 x[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) x[s] = reinterpret_cast<const __nv_bfloat162 *>(raw[s])[i];
        const __nv_bfloat162 mean = __hadd2(__hfma2(x[1], fourth, __hmul2(x[0], fourth)), __hfma2(x[3], fourth, __hmul2(x[2], fourth))),
                             apart = __hsub2(__hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3])),
                                             __hmin2(__hmin2(x[0], x[1]), __hmin2(x[2], x[3])));
        c[i] = reinterpret_cast<const uint32_t &>(mean) & __hle2_mask(apart, __hmul2(__habs2(mean), half));
    }
}

template <int D> __device__ __forceinline__ void dq_pass(const BwdParams &prm, unsigned char *smem, uint32_t unit) {
    using C = QCfg<D>;
    const SeqArgs &a = prm.a;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::BAR0);
    uint64_t &q_full = bar[0], &s_full = bar[1], &s_free = bar[2], &dp_full = bar[3], &ds_full = bar[4], &acc_full = bar[5];
    uint32_t &tmem_base = *reinterpret_cast<uint32_t *>(bar + 6);
    uint64_t *ring_full = bar + 7, *ring_empty = ring_full + C::NK + C::NV;
    static_assert((7 + 2 * (C::NK + C::NV)) * 8 <= 256, "barriers");
    const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
    const uint32_t sbase = tc::smem_u32(smem);
    const Ring<C::NK, C::TB> rk{ring_full, ring_empty, sbase + C::ST0};
    const Ring<C::NV, C::TB> rv{ring_full + C::NK, ring_empty + C::NK, sbase + C::V0};
    const SeqTile t = a.qtiles[unit / a.H];
    const int h = unit % a.H, hk = h / (a.H / a.Hkv);
    const int n = t.t1 - t.t0;

    if (tid == 32) {
        tc::mbar_init(&q_full, kSoft);
        tc::mbar_init(&s_free, kSoft);
        rk.init();
        rv.init();
        tc::mbar_init(&s_full, 1);
        tc::mbar_init(&dp_full, 1);
        tc::mbar_init(&ds_full, kSoft);
        tc::mbar_init(&acc_full, 1);
    }
    wait_previous();
    if (warp == 0) tc::tmem_alloc(&tmem_base, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tS = tmem_base + C::TS, tP = tmem_base + C::TP, tQ = tmem_base + C::TQ, tA = tmem_base + C::TA,
                   tG = tmem_base + C::TG;

    if (warp < 4) {
        tc::reg_dec<kRCtrl>();
        if (warp == 0 && lane == 0) {   // ----------------------------------- TMA producer
            bool ok = true;
            int i = 0, v = 0;   // tiles of K and V issued
            for (; i < n; ++i) {
                if (!rk.wait_room(i)) {
                    ok = false;
                    break;
                }
                tc::mbar_expect_tx(rk.filled(i), C::TB);
                seq::load_tile<C::DA>(rk.at(i), &prm.tk, hk, (t.t0 + i) * 128, rk.filled(i));
                if (!rv.wait_room(i)) {
                    ok = false;
                    ++i;
                    break;
                }
                tc::mbar_expect_tx(rv.filled(i), C::TB);
                seq::load_tile<C::DA>(rv.at(i), &prm.tv, hk, (t.t0 + i) * 128, rv.filled(i));
                ++v;
            }
            if (!ok) atomicOr(a.d_err, tc::kErrMmaTimeout);
            // loads that no product consumed (only after a timeout) land before the CTA ends
            rk.drain(i);
            rv.drain(v);
        } else if (warp == 1) {   // ----------------------------------------- MMA issuer (the warp in step)
            constexpr uint32_t idesc_s = tc::idesc_bf16(128, 128), idesc_g = tc::idesc_bf16(128, C::DP) | tc::kMajorMnB;
            auto scores = [&](int i) {
                mma_over_d_ts<C::DP>(tS, tA, rk.at(i), idesc_s);
                tc::mma_commit_w(&s_full);
            };
            auto dprod = [&](int i) {
                mma_over_d_ts<C::DP>(tP, tG, rv.at(i), idesc_s);
                tc::mma_commit_w(&dp_full);
                tc::mma_commit_w(rv.freed(i));
            };
            bool ok = tc::warp_wait(&q_full, 0, tc::kWaitLimit) && rk.wait_filled(0) && rv.wait_filled(0);
            if (ok) {
                tc::fence_after_sync();
                scores(0);
                dprod(0);
            }
            for (int i = 0; i < n && ok; ++i) {
                if (i + 1 < n) {   // (the next V has landed; its barrier is polled while dS is formed)
                    if (!rk.wait_filled(i + 1) || !tc::warp_wait(&s_free, i & 1, tc::kWaitLimit)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    scores(i + 1);
                    ok = rv.wait_filled(i + 1);
                }
                if (!ok || !tc::warp_wait(&ds_full, i & 1, tc::kWaitLimit)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                mma_rows128(tQ, tP, rk.at(i), idesc_g, i == 0);   // dQ += dS K
                tc::mma_commit_w(rk.freed(i));
                if (i + 1 < n) dprod(i + 1);
            }
            if (!ok && lane == 0) atomicOr(a.d_err, tc::kErrMmaTimeout);
            // every product issued is complete before TMEM is released
            tc::mma_commit_w(&acc_full);
            tc::warp_wait(&acc_full, 0, tc::kWaitLimit);
        }
        __syncwarp();
    } else {   // ---------------------------------------------------- weights and epilogue
        tc::reg_inc<kRSoft>();
        const int quarter = warp & 3, part = (warp - 4) >> 2;   // part: keys N part .. of a tile
        const uint32_t tl = (uint32_t)(quarter * 32) << 16;
        const int64_t row = (int64_t)t.tile * 128 + quarter * 32 + lane;
        const bool in = row < a.rows;
        int64_t lo = 0, hi = 0;   // the keys that the row sees
        if (in) {
            const int2 se = __ldg(a.range + row);
            lo = se.x;
            hi = a.causal ? row + 1 : se.y;
        }
        const float scale2 = a.scale * kLog2e;
        const float nlse = a.ws_nlse[(int64_t)h * a.rows_pad + row], nd = a.ws_ndelta[(int64_t)h * a.rows_pad + row];
        const float2 k2 = make_float2(scale2, scale2), l2 = make_float2(nlse, nlse), d2 = make_float2(nd, nd);
        constexpr int N = kCols;
        // the row's share of Q and dOut into TMEM (rows past the last, and the
        // columns past a head of 32, as zeros)
        {
            constexpr int CW = C::DP / 2 / kParts;   // columns (bf16 pairs) of a part
            for (int x = 0; x < 2; ++x) {
                const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(x ? a.dOut : a.Q) + ((in ? row : 0) * a.H + h) * D;
#pragma unroll
                for (int c = 0; c < CW; c += 8) {
                    const int e = 2 * (part * CW + c);    // first element
                    uint32_t u[8];
#pragma unroll
                    for (int k = 0; k < 8; k += 4) {
                        const uint4 q = in && e + 2 * k < D ? ldg16(src + e + 2 * k) : make_uint4(0, 0, 0, 0);
                        u[k] = q.x;
                        u[k + 1] = q.y;
                        u[k + 2] = q.z;
                        u[k + 3] = q.w;
                    }
                    tc::tmem_st8_async((x ? tG : tA) + part * CW + c + tl, u);
                }
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&q_full);
        }
        const uint32_t ts = tS + part * N + tl, tp = tP + part * N + tl;
        constexpr int SL = D <= 32 * kParts ? 1 : D / (32 * kParts);   // slices of 32 columns that a part stores
        uint32_t mean[SL][16];
#pragma unroll
        for (int k = 0; k < SL; ++k)   // (while the first tiles arrive)
            if ((k * kParts + part) * 32 < D) mean_key(a, D, lo, hi, hk, (k * kParts + part) * 32, mean[k]);
        float2 res = make_float2(0.f, 0.f);   // the part's sum of e_j
        float p[N];                           // a tile's dS, and rounded
        uint32_t pk[N / 2];
#pragma unroll
        for (int c = 0; c < N; ++c) p[c] = __uint_as_float(pk[c >> 1] = 0u);
        auto add_errors = [&](int c) {   // of the columns c, c + 1
            const float2 r = make_float2(__uint_as_float(pk[c >> 1] << 16), __uint_as_float(pk[c >> 1] & 0xffff0000u));
            res = fadd2(res, ffma2(make_float2(p[c], p[c + 1]), make_float2(-1.f, -1.f), r));
        };
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int kt = t.t0 + i;
            if (!tc::warp_wait(&s_full, i & 1, tc::kWaitLimit)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            uint32_t v[N];
            load_scores(ts, v);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&s_free);
            // the errors of the tile before are added between the exponentials, which
            // leave issue slots (after the dS have been handed over: 8% slower)
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                add_errors(c);
                const float2 x = ffma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), k2, l2);
                p[c] = fast_exp2(x.x);
                p[c + 1] = fast_exp2(x.y);
            }
            if (!tc::warp_wait(&dp_full, i & 1, tc::kWaitLimit)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            load_scores(tp, v);
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                const float2 x = fmul2(make_float2(p[c], p[c + 1]),
                                       fadd2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), d2));
                p[c] = x.x;
                p[c + 1] = x.y;
            }
            if (kt < t.f0 || kt >= t.f1) {
                const int cl = seq::rel(lo, (int64_t)kt * 128), ch = seq::rel(hi, (int64_t)kt * 128);
                uint32_t bits = 0;
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    if (c % 32 == 0) bits = seq::column_bits(cl, ch, (part * N + c) / 32);
                    if (!((bits >> (c & 31)) & 1u)) p[c] = 0.f;
                }
            }
            round_weights(p, pk);
            store_weights(tp, pk);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ds_full);
        }
#pragma unroll
        for (int c = 0; c < N; c += 2) add_errors(c);
        // the parts' sums, added in order (every weight warp comes here, after a timeout too)
        float *sums = reinterpret_cast<float *>(smem + C::RES0);
        sums[part * 128 + quarter * 32 + lane] = res.x + res.y;
        asm volatile("bar.sync 1, %0;" ::"n"(128 * kParts) : "memory");
        float err = sums[quarter * 32 + lane];
#pragma unroll
        for (int k = 1; k < kParts; ++k) err += sums[k * 128 + quarter * 32 + lane];
        if (ok && !tc::warp_wait(&acc_full, 0, tc::kWaitLimit)) ok = false;
        if (ok) {
            tc::fence_after_sync();
            uint32_t again = 0;
#pragma unroll
            for (int k = 0; k < SL; ++k) {
                const int c0 = (k * kParts + part) * 32;
                if (c0 >= D) break;
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.dQ) + ((in ? row : 0) * a.H + h) * D + c0;
                float sub[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sub[2 * i] = err * __uint_as_float(mean[k][i] << 16);
                    sub[2 * i + 1] = err * __uint_as_float(mean[k][i] & 0xffff0000u);
                }
                again |= store_from_tmem(tQ + c0 + tl, dst, a.scale, in, sub);
            }
            __syncwarp();   // (the rows are read back)
            while (again) {
                const int src = __ffs(again) - 1;
                again &= again - 1;
                const seq::Span sp{__shfl_sync(SGA_FULL_MASK, lo, src), __shfl_sync(SGA_FULL_MASK, hi, src), (int64_t)t.t0 * 128,
                                   min(a.rows, (int64_t)t.t1 * 128)};
                seq::query_row_alone<__nv_bfloat16, D>(a, __shfl_sync(SGA_FULL_MASK, row, src), h, sp, seq::slice_columns<D>(0, part, kParts));
            }
        } else if (lane == 0) {
            atomicOr(a.d_err, tc::kErrMmaTimeout);
        }
    }
    // the MMA lane waited for all its products, the producer for its loads
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc::tmem_dealloc(tmem_base, 512);
    }
}

// Both passes in one launch, the dK/dV units first: they are the longer ones,
// and the dQ units fill the SMs that run out of them.  The tiles take all but a
// few hundred bytes of an SM's shared memory, so the barriers lie behind them
// and the block's memory has to begin on the tiles' alignment, as it does for a
// kernel without static shared memory.
template <int D> __global__ void __launch_bounds__(kThreads, 1) seq_bwd_kernel(const __grid_constant__ BwdParams prm) {
    extern __shared__ __align__(1024) unsigned char smem[];
    if (tc::smem_u32(smem) & 1023) {
        wait_previous();
        if (threadIdx.x == 0) atomicOr(prm.a.d_err, tc::kErrMmaTimeout);
        return;
    }
    const uint32_t kv = (uint32_t)prm.a.n_tiles * prm.a.Hkv;
    if (blockIdx.x < kv) dkdv_pass<D>(prm, smem, blockIdx.x);
    else dq_pass<D>(prm, smem, blockIdx.x - kv);
}

template <int D> cudaError_t launch(const SeqArgs &a, cudaStream_t s) {
    BwdParams prm{};
    prm.a = a;
    cudaError_t e = seq_tensor_map(&prm.tq, a.Q, a.rows, a.H, D);
    if (e == cudaSuccess) e = seq_tensor_map(&prm.tg, a.dOut, a.rows, a.H, D);
    if (e == cudaSuccess) e = seq_tensor_map(&prm.tk, a.K, a.rows, a.Hkv, D);
    if (e == cudaSuccess) e = seq_tensor_map(&prm.tv, a.V, a.rows, a.Hkv, D);
    constexpr size_t smem = KvCfg<D>::BYTES > QCfg<D>::BYTES ? KvCfg<D>::BYTES : QCfg<D>::BYTES;
    if (e == cudaSuccess) e = allow_smem<seq_bwd_kernel<D>>(smem);
    if (e == cudaSuccess) e = seq_row_terms<__nv_bfloat16>(a, D, s);
    if (e != cudaSuccess) return e;
    note_launch(SGA_KERN_SEQ_BWD, s, false);
    e = launch_early(seq_bwd_kernel<D>, dim3((unsigned)((int64_t)a.n_tiles * (a.Hkv + a.H))), dim3(kThreads), smem, s, prm);
    note_launch(SGA_KERN_SEQ_BWD, s, true);
    return e;
}

}  // namespace

cudaError_t seq_bwd_bf16(const SeqArgs &a, int D, cudaStream_t s) {
    return D == 32 ? launch<32>(a, s) : D == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace sga
