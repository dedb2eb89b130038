// Packed-sequence attention backward on the tcgen05 tensor cores (bf16).
//
//   P = exp(S - lse), dP = dOut V^T, dS = P (dP - Delta),
//   dV = P^T dOut, dK = scale dS^T Q, dQ = scale dS K
//
// Two passes, so that every output row is owned by one CTA: no atomics, no
// fp32 copy of dQ in memory, bitwise reproducible; S and dP are computed twice
// (seven products a tile pair instead of five).
//   dK/dV pass (unit: 128 keys x key head, over the query tiles that see them
//     and the heads of the group): S^T = K Q^T and dP^T = V dOut^T with keys in
//     the TMEM lanes, P^T and dS^T written back to TMEM in bf16 over the scores
//     they come from, where they are the A operands of dV += P^T dOut and
//     dK += dS^T Q.  The products are issued dV(i), S(i + 1), dK(i), dP(i + 1):
//     while the weights of i + 1 are formed the tensor core has dK(i) and
//     dP(i + 1), while its dS is formed it has dV(i + 1) and S(i + 2).
//   dQ pass (unit: 128 queries x head, over the key tiles they see): S, two
//     buffers, dP with queries in the lanes, dS in bf16 over dP, dQ += dS K,
//     issued S(i + 1), dQ(i), dP(i + 1).
// Roles as in the forward: one lane loads by TMA, one issues the products,
// eight warps (two per TMEM lane quarter, each with half of a tile's columns)
// turn scores into weights.  P and dS are rounded to bf16 once (half a step,
// 2^-8 relative), which is of the size of the rounding of the gradients.
//
// As in the forward, a row whose result is not finite is computed again over
// its own interval alone, so that nothing of a pair that is masked reaches it.
// Every wait is bounded; a timeout sets the plan's error word and ends the role.
#include <algorithm>

#include "seq_tc.cuh"

namespace sga {
namespace {

constexpr int kThreads = 384;   // control warps (load, MMA, two idle), eight weight warps
constexpr int kSoft = 8;        // arrivals per handoff
constexpr int kRCtrl = 56, kRSoft = 224;   // registers a thread after the split; 168 at launch
static_assert(kRCtrl + 2 * kRSoft == 3 * 168, "register split");

template <int D> struct BwdCfg {
    static constexpr int DP = D < 64 ? 64 : D, DA = DP / 64;
    static constexpr uint32_t TB = DA * 128 * 128;    // a tile of 128 rows
    static constexpr uint32_t R0 = 0;                 // two resident tiles
    static constexpr uint32_t ST0 = 2 * TB;           // ring of streamed tiles
};
template <int D> struct KvCfg : BwdCfg<D> {
    using B = BwdCfg<D>;
    static constexpr int NST = B::DP == 64 ? 8 : 4;
    static constexpr uint32_t ROW0 = B::ST0 + NST * B::TB;        // lse, Delta of the queries of ring entry 2j
    static constexpr uint32_t BYTES = ROW0 + NST / 2 * 1024;
    static constexpr uint32_t TS = 0, TP = 128, TK = 256, TV = 256 + B::DP;   // S^T, dP^T, dK, dV
};
template <int D> struct QCfg : BwdCfg<D> {
    using B = BwdCfg<D>;
    static constexpr int NST = B::DP == 64 ? 8 : 5;
    static constexpr uint32_t BYTES = B::ST0 + NST * B::TB;
    static constexpr uint32_t TS = 0, TP = 256, TQ = 384;         // two S buffers, dP, dQ
};
static_assert(KvCfg<128>::BYTES + 1024 <= 226 * 1024 && QCfg<128>::BYTES + 1024 <= 226 * 1024, "shared memory");

struct BwdParams {
    CUtensorMap tq, tk, tv, tg;
    SeqArgs a;
};

// A 128-deep product with the A operand in TMEM (its halves 64 columns apart,
// 32 columns of bf16 pairs each) and 128 rows of B as an MN-major operand.
__device__ __forceinline__ void mma_rows128(uint32_t d, uint32_t ta, uint32_t b, uint32_t idesc, bool first) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
        tc::mma_bf16_ts_w(d, ta + (kk >> 2) * 64 + (kk & 3) * 8, tc::desc_sw128_mn(b + kk * 2048, 16384), idesc,
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

template <int D> struct RowFrag {
    static constexpr int W = D / 32;
    float x[W];
    __device__ __forceinline__ void load(const void *base, int64_t off) {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(base) + off + (threadIdx.x & 31) * W;
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = __bfloat162float(p[i]);
    }
    __device__ __forceinline__ float dot(const RowFrag &o) const {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) s = fmaf(x[i], o.x[i], s);
        return group_sum<32>(s);
    }
    // store the columns [c0, c1)
    __device__ __forceinline__ void store(void *base, int64_t off, float f, int c0, int c1) const {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int c = (threadIdx.x & 31) * W + i;
            if (c >= c0 && c < c1) static_cast<__nv_bfloat16 *>(base)[off + c] = __float2bfloat16_rn(x[i] * f);
        }
    }
};

// dK (DK) or dV of one key row by its warp, over the queries [lo, hi) alone.
template <int D, bool DK>
__device__ __forceinline__ void key_row_alone(const SeqArgs &a, int64_t row, int hk, int64_t lo, int64_t hi) {
    RowFrag<D> k, v, acc;
    const int64_t at = (row * a.Hkv + hk) * D;
    k.load(a.K, at);
    v.load(a.V, at);
#pragma unroll
    for (int i = 0; i < RowFrag<D>::W; ++i) acc.x[i] = 0.f;
    const int grp = a.H / a.Hkv;
    for (int h = hk * grp; h < (hk + 1) * grp; ++h)
        for (int64_t r = lo; r < hi; ++r) {
            RowFrag<D> q, g;
            q.load(a.Q, (r * a.H + h) * D);
            g.load(a.dOut, (r * a.H + h) * D);
            const int64_t t = (int64_t)h * a.rows_pad + r;
            const float p = fast_exp2(fmaf(q.dot(k), a.scale * kLog2e, -a.ws_lse[t]));
            const float w = DK ? p * (g.dot(v) - a.ws_delta[t]) : p;
#pragma unroll
            for (int i = 0; i < RowFrag<D>::W; ++i) acc.x[i] = fmaf(w, DK ? q.x[i] : g.x[i], acc.x[i]);
        }
    acc.store(DK ? a.dK : a.dV, at, DK ? a.scale : 1.f, 0, D);
}

// Columns [c0, c1) of dQ of one query row by its warp, over the keys [lo, hi) alone.
template <int D>
__device__ __forceinline__ void query_row_alone(const SeqArgs &a, int64_t row, int h, int64_t lo, int64_t hi, int c0,
                                                int c1) {
    RowFrag<D> q, g, acc;
    const int64_t at = (row * a.H + h) * D, t = (int64_t)h * a.rows_pad + row;
    const int hk = h / (a.H / a.Hkv);
    q.load(a.Q, at);
    g.load(a.dOut, at);
#pragma unroll
    for (int i = 0; i < RowFrag<D>::W; ++i) acc.x[i] = 0.f;
    for (int64_t j = lo; j < hi; ++j) {
        RowFrag<D> k, v;
        k.load(a.K, (j * a.Hkv + hk) * D);
        v.load(a.V, (j * a.Hkv + hk) * D);
        const float p = fast_exp2(fmaf(q.dot(k), a.scale * kLog2e, -a.ws_lse[t]));
        const float w = p * (g.dot(v) - a.ws_delta[t]);
#pragma unroll
        for (int i = 0; i < RowFrag<D>::W; ++i) acc.x[i] = fmaf(w, k.x[i], acc.x[i]);
    }
    acc.store(a.dQ, at, a.scale, c0, c1);
}

// N columns of a row from TMEM, scaled, to bf16 at dst (if `in`); whether any was not finite.
template <int N>
__device__ __forceinline__ bool store_from_tmem(uint32_t taddr, __nv_bfloat16 *dst, float f, bool in) {
    bool bad = false;
#pragma unroll
    for (int cb = 0; cb < N; cb += 32) {
        uint32_t o[32];
        tc::tmem_ld32(taddr + cb, o);   // warp-collective: every lane takes part
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            x[i] = __uint_as_float(o[i]) * f;
            bad |= !(fabsf(x[i]) < INFINITY);
        }
        if (in)
#pragma unroll
            for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4 *>(dst + cb + 8 * q) = pack<__nv_bfloat16>(x + 8 * q);
    }
    return bad && in;
}

// ---- dK, dV -----------------------------------------------------------------------

template <int D> __global__ void __launch_bounds__(kThreads, 1) seq_bwd_dkdv_kernel(const __grid_constant__ BwdParams prm) {
    using C = KvCfg<D>;
    const SeqArgs &a = prm.a;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t kv_full, full[C::NST], empty[C::NST], s_full, dp_full, p_full, ds_full, acc_full;
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
    const uint32_t sbase = tc::smem_u32(smem);
    const SeqTile t = a.ktiles[blockIdx.x / a.Hkv];
    const int hk = blockIdx.x % a.Hkv, grp = a.H / a.Hkv;
    const int nt = t.t1 - t.t0, n = nt * grp;   // steps: (head of the group, query tile)

    if (warp == 0) tc::tmem_alloc(&tmem_base, 512);
    if (tid == 32) {
        tc::mbar_init(&kv_full, 1);
        for (int i = 0; i < C::NST; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        tc::mbar_init(&s_full, 1);
        tc::mbar_init(&dp_full, 1);
        tc::mbar_init(&p_full, kSoft);
        tc::mbar_init(&ds_full, kSoft);
        tc::mbar_init(&acc_full, 1);
    }
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
            int e = 0;   // entry 2 i: Q, lse and Delta of step i; 2 i + 1: dOut
            for (; e < 2 * n; ++e) {
                const int b = e % C::NST, r = e / C::NST;
                if (r >= 1 && !tc::mbar_wait(&empty[b], (r - 1) & 1, tc::kWaitLimit)) {
                    ok = false;
                    break;
                }
                const int h = hk * grp + (e >> 1) / nt, qt = t.t0 + (e >> 1) % nt;
                const uint32_t dst = sbase + C::ST0 + b * C::TB;
                if (e & 1) {
                    tc::mbar_expect_tx(&full[b], C::TB);
                    seq::load_tile<C::DA>(dst, &prm.tg, h, qt * 128, &full[b]);
                } else {
                    tc::mbar_expect_tx(&full[b], C::TB + 1024);
                    seq::load_tile<C::DA>(dst, &prm.tq, h, qt * 128, &full[b]);
                    const int64_t r0 = (int64_t)h * a.rows_pad + (int64_t)qt * 128;
                    const uint32_t rows = sbase + C::ROW0 + (b >> 1) * 1024;
                    tc::bulk_load(rows, a.ws_lse + r0, 512, &full[b]);
                    tc::bulk_load(rows + 512, a.ws_delta + r0, 512, &full[b]);
                }
            }
            if (!ok) atomicOr(a.d_err, tc::kErrMmaTimeout);
            // loads that no product consumed (only after a timeout) land before the CTA ends
            tc::mbar_wait(&kv_full, 0, tc::kWaitLimit);
            for (int i = e - 1; i >= 0 && i >= e - C::NST; --i)
                tc::mbar_wait(&full[i % C::NST], (i / C::NST) & 1, tc::kWaitLimit);
        } else if (warp == 1) {   // ----------------------------------------- MMA issuer (the warp in step)
            constexpr uint32_t idesc_s = tc::idesc_bf16(128, 128), idesc_g = tc::idesc_bf16(128, C::DP) | tc::kMajorMnB;
            const uint32_t ka = sbase + C::R0, va = ka + C::TB;
            auto entry = [&](int e) { return sbase + C::ST0 + (e % C::NST) * C::TB; };
            auto landed = [&](int e) { return tc::warp_wait(&full[e % C::NST], (e / C::NST) & 1, tc::kWaitLimit); };
            bool ok = tc::warp_wait(&kv_full, 0, tc::kWaitLimit) && landed(0);
            if (ok) {
                tc::fence_after_sync();
                mma_over_d<C::DP>(tS, ka, entry(0), idesc_s);
                tc::mma_commit_w(&s_full);
                ok = landed(1);
            }
            if (ok) {
                tc::fence_after_sync();
                mma_over_d<C::DP>(tP, va, entry(1), idesc_s);
                tc::mma_commit_w(&dp_full);
            }
            for (int i = 0; i < n && ok; ++i) {
                const int e = 2 * i;
                if (!tc::warp_wait(&p_full, i & 1, tc::kWaitLimit)) ok = false;
                if (!ok) break;
                tc::fence_after_sync();
                mma_rows128(tV, tS, entry(e + 1), idesc_g, i == 0);   // dV += P^T dOut
                tc::mma_commit_w(&empty[(e + 1) % C::NST]);
                if (i + 1 < n) {
                    if (!landed(e + 2)) ok = false;
                    if (!ok) break;
                    tc::fence_after_sync();
                    mma_over_d<C::DP>(tS, ka, entry(e + 2), idesc_s);
                    tc::mma_commit_w(&s_full);
                }
                if (!tc::warp_wait(&ds_full, i & 1, tc::kWaitLimit)) ok = false;
                if (!ok) break;
                tc::fence_after_sync();
                mma_rows128(tK, tP, entry(e), idesc_g, i == 0);       // dK += dS^T Q
                tc::mma_commit_w(&empty[e % C::NST]);
                if (i + 1 < n) {
                    if (!landed(e + 3)) ok = false;
                    if (!ok) break;
                    tc::fence_after_sync();
                    mma_over_d<C::DP>(tP, va, entry(e + 3), idesc_s);
                    tc::mma_commit_w(&dp_full);
                }
            }
            if (!ok && lane == 0) atomicOr(a.d_err, tc::kErrMmaTimeout);
            // every product issued is complete before TMEM is released
            tc::mma_commit_w(&acc_full);
            tc::warp_wait(&acc_full, 0, tc::kWaitLimit);
        }
        __syncwarp();
    } else {   // ---------------------------------------------------- weights and epilogue
        tc::reg_inc<kRSoft>();
        const int quarter = warp & 3, hf = (warp - 4) >> 2;   // half hf: queries 64 hf .. of a tile
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
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int qt = t.t0 + i % nt, b = (2 * i) % C::NST;
            if (!tc::warp_wait(&full[b], ((2 * i) / C::NST) & 1, tc::kWaitLimit) ||
                !tc::warp_wait(&s_full, i & 1, tc::kWaitLimit)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            const float4 *ls = reinterpret_cast<const float4 *>(smem + C::ROW0 + (b >> 1) * 1024) + hf * 16;
            const float4 *dl = ls + 32;
            uint32_t v[64], pk[32];
            tc::tmem_ld32_async(tS + hf * 64 + tl, v);
            tc::tmem_ld32_async(tS + hf * 64 + 32 + tl, v + 32);
            tc::tmem_wait_ld(v);
            tc::tmem_wait_ld(v + 32);
            float p[64];
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 l4 = ls[c >> 2];
                const float2 x = ffma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), k2,
                                       make_float2(-l4.x, -l4.y));
                const float2 y = ffma2(make_float2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])), k2,
                                       make_float2(-l4.z, -l4.w));
                p[c] = fast_exp2(x.x);
                p[c + 1] = fast_exp2(x.y);
                p[c + 2] = fast_exp2(y.x);
                p[c + 3] = fast_exp2(y.y);
            }
            uint32_t bits[2] = {0xffffffffu, 0xffffffffu};
            const bool part = qt < t.f0 || qt >= t.f1;
            if (part) {
                const int cl = seq::rel(lo, (int64_t)qt * 128), ch = seq::rel(hi, (int64_t)qt * 128);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    bits[w] = seq::column_bits(cl, ch, 2 * hf + w);
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!((bits[w] >> c) & 1u)) p[32 * w + c] = 0.f;
                }
            }
#pragma unroll
            for (int c = 0; c < 64; c += 2) pk[c >> 1] = pack_bf16x2(p[c], p[c + 1]);
            tc::tmem_st32_async(tS + hf * 64 + tl, pk);
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&p_full);

            if (!tc::warp_wait(&dp_full, i & 1, tc::kWaitLimit)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            tc::tmem_ld32_async(tP + hf * 64 + tl, v);
            tc::tmem_ld32_async(tP + hf * 64 + 32 + tl, v + 32);
            tc::tmem_wait_ld(v);
            tc::tmem_wait_ld(v + 32);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 d4 = dl[c >> 2];
                const float2 x = fmul2(make_float2(p[c], p[c + 1]),
                                       fadd2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                                             make_float2(-d4.x, -d4.y)));
                const float2 y = fmul2(make_float2(p[c + 2], p[c + 3]),
                                       fadd2(make_float2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])),
                                             make_float2(-d4.z, -d4.w)));
                p[c] = x.x;
                p[c + 1] = x.y;
                p[c + 2] = y.x;
                p[c + 3] = y.y;
            }
            if (part)   // (zero weights times an infinity)
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!((bits[w] >> c) & 1u)) p[32 * w + c] = 0.f;
#pragma unroll
            for (int c = 0; c < 64; c += 2) pk[c >> 1] = pack_bf16x2(p[c], p[c + 1]);
            tc::tmem_st32_async(tP + hf * 64 + tl, pk);
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ds_full);
        }
        if (ok && !tc::warp_wait(&acc_full, 0, tc::kWaitLimit)) ok = false;
        if (ok) {
            tc::fence_after_sync();
            // half 0 stores dV, half 1 dK
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(hf ? a.dK : a.dV) + ((in ? row : 0) * a.Hkv + hk) * D;
            const bool bad = store_from_tmem<D>((hf ? tK : tV) + tl, dst, hf ? a.scale : 1.f, in);
            uint32_t again = __ballot_sync(SGA_FULL_MASK, bad);
            while (again) {
                const int src = __ffs(again) - 1;
                again &= again - 1;
                const int64_t r = __shfl_sync(SGA_FULL_MASK, row, src), l = __shfl_sync(SGA_FULL_MASK, lo, src),
                              u = __shfl_sync(SGA_FULL_MASK, hi, src);
                if (hf) key_row_alone<D, true>(a, r, hk, l, u);
                else key_row_alone<D, false>(a, r, hk, l, u);
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

template <int D> __global__ void __launch_bounds__(kThreads, 1) seq_bwd_dq_kernel(const __grid_constant__ BwdParams prm) {
    using C = QCfg<D>;
    const SeqArgs &a = prm.a;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t q_full, full[C::NST], empty[C::NST], s_full[2], dp_full, ds_full, acc_full;
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
    const uint32_t sbase = tc::smem_u32(smem);
    const SeqTile t = a.qtiles[blockIdx.x / a.H];
    const int h = blockIdx.x % a.H, hk = h / (a.H / a.Hkv);
    const int n = t.t1 - t.t0;

    if (warp == 0) tc::tmem_alloc(&tmem_base, 512);
    if (tid == 32) {
        tc::mbar_init(&q_full, 1);
        for (int i = 0; i < C::NST; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        tc::mbar_init(&s_full[0], 1);
        tc::mbar_init(&s_full[1], 1);
        tc::mbar_init(&dp_full, 1);
        tc::mbar_init(&ds_full, kSoft);
        tc::mbar_init(&acc_full, 1);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tS = tmem_base + C::TS, tP = tmem_base + C::TP, tQ = tmem_base + C::TQ;

    if (warp < 4) {
        tc::reg_dec<kRCtrl>();
        if (warp == 0 && lane == 0) {   // ----------------------------------- TMA producer
            bool ok = true;
            tc::mbar_expect_tx(&q_full, 2 * C::TB);
            seq::load_tile<C::DA>(sbase + C::R0, &prm.tq, h, t.tile * 128, &q_full);
            seq::load_tile<C::DA>(sbase + C::R0 + C::TB, &prm.tg, h, t.tile * 128, &q_full);
            int e = 0;   // entry 2 i: K, 2 i + 1: V of key tile i
            for (; e < 2 * n; ++e) {
                const int b = e % C::NST, r = e / C::NST;
                if (r >= 1 && !tc::mbar_wait(&empty[b], (r - 1) & 1, tc::kWaitLimit)) {
                    ok = false;
                    break;
                }
                tc::mbar_expect_tx(&full[b], C::TB);
                seq::load_tile<C::DA>(sbase + C::ST0 + b * C::TB, (e & 1) ? &prm.tv : &prm.tk, hk, (t.t0 + (e >> 1)) * 128,
                                      &full[b]);
            }
            if (!ok) atomicOr(a.d_err, tc::kErrMmaTimeout);
            // loads that no product consumed (only after a timeout) land before the CTA ends
            tc::mbar_wait(&q_full, 0, tc::kWaitLimit);
            for (int i = e - 1; i >= 0 && i >= e - C::NST; --i)
                tc::mbar_wait(&full[i % C::NST], (i / C::NST) & 1, tc::kWaitLimit);
        } else if (warp == 1) {   // ----------------------------------------- MMA issuer (the warp in step)
            constexpr uint32_t idesc_s = tc::idesc_bf16(128, 128), idesc_g = tc::idesc_bf16(128, C::DP) | tc::kMajorMnB;
            const uint32_t qa = sbase + C::R0, ga = qa + C::TB;
            auto entry = [&](int e) { return sbase + C::ST0 + (e % C::NST) * C::TB; };
            auto landed = [&](int e) { return tc::warp_wait(&full[e % C::NST], (e / C::NST) & 1, tc::kWaitLimit); };
            auto scores = [&](int i) -> bool {
                if (!landed(2 * i)) return false;
                tc::fence_after_sync();
                mma_over_d<C::DP>(tS + (i & 1) * 128, qa, entry(2 * i), idesc_s);
                tc::mma_commit_w(&s_full[i & 1]);
                return true;
            };
            auto dprod = [&](int i) -> bool {
                if (!landed(2 * i + 1)) return false;
                tc::fence_after_sync();
                mma_over_d<C::DP>(tP, ga, entry(2 * i + 1), idesc_s);
                tc::mma_commit_w(&dp_full);
                tc::mma_commit_w(&empty[(2 * i + 1) % C::NST]);
                return true;
            };
            bool ok = tc::warp_wait(&q_full, 0, tc::kWaitLimit) && scores(0) && dprod(0);
            for (int i = 0; i < n && ok; ++i) {
                // S(i + 1) overwrites S(i - 1), read before dS(i - 1) arrived
                if (i + 1 < n && !scores(i + 1)) ok = false;
                if (!ok || !tc::warp_wait(&ds_full, i & 1, tc::kWaitLimit)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                mma_rows128(tQ, tP, entry(2 * i), idesc_g, i == 0);   // dQ += dS K
                tc::mma_commit_w(&empty[(2 * i) % C::NST]);
                if (i + 1 < n && !dprod(i + 1)) ok = false;
            }
            if (!ok && lane == 0) atomicOr(a.d_err, tc::kErrMmaTimeout);
            // every product issued is complete before TMEM is released
            tc::mma_commit_w(&acc_full);
            tc::warp_wait(&acc_full, 0, tc::kWaitLimit);
        }
        __syncwarp();
    } else {   // ---------------------------------------------------- weights and epilogue
        tc::reg_inc<kRSoft>();
        const int quarter = warp & 3, hf = (warp - 4) >> 2;   // half hf: keys 64 hf .. of a tile
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
        const float lse = a.ws_lse[(int64_t)h * a.rows_pad + row], delta = a.ws_delta[(int64_t)h * a.rows_pad + row];
        const float2 k2 = make_float2(scale2, scale2), l2 = make_float2(-lse, -lse), d2 = make_float2(-delta, -delta);
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int kt = t.t0 + i;
            if (!tc::warp_wait(&s_full[i & 1], (i >> 1) & 1, tc::kWaitLimit)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            uint32_t v[64], pk[32];
            tc::tmem_ld32_async(tS + (i & 1) * 128 + hf * 64 + tl, v);
            tc::tmem_ld32_async(tS + (i & 1) * 128 + hf * 64 + 32 + tl, v + 32);
            tc::tmem_wait_ld(v);
            tc::tmem_wait_ld(v + 32);
            float p[64];
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
                const float2 x = ffma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), k2, l2);
                p[c] = fast_exp2(x.x);
                p[c + 1] = fast_exp2(x.y);
            }
            if (!tc::warp_wait(&dp_full, i & 1, tc::kWaitLimit)) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            tc::tmem_ld32_async(tP + hf * 64 + tl, v);
            tc::tmem_ld32_async(tP + hf * 64 + 32 + tl, v + 32);
            tc::tmem_wait_ld(v);
            tc::tmem_wait_ld(v + 32);
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
                const float2 x = fmul2(make_float2(p[c], p[c + 1]),
                                       fadd2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), d2));
                p[c] = x.x;
                p[c + 1] = x.y;
            }
            if (kt < t.f0 || kt >= t.f1) {
                const int cl = seq::rel(lo, (int64_t)kt * 128), ch = seq::rel(hi, (int64_t)kt * 128);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t bits = seq::column_bits(cl, ch, 2 * hf + w);
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!((bits >> c) & 1u)) p[32 * w + c] = 0.f;
                }
            }
#pragma unroll
            for (int c = 0; c < 64; c += 2) pk[c >> 1] = pack_bf16x2(p[c], p[c + 1]);
            tc::tmem_st32_async(tP + hf * 64 + tl, pk);
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ds_full);
        }
        if (ok && !tc::warp_wait(&acc_full, 0, tc::kWaitLimit)) ok = false;
        if (ok) {
            tc::fence_after_sync();
            constexpr int HC = D < 64 ? 32 : D / 2;   // columns a half stores
            if (hf * HC < D) {
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.dQ) + ((in ? row : 0) * a.H + h) * D + hf * HC;
                const bool bad = store_from_tmem<HC>(tQ + hf * HC + tl, dst, a.scale, in);
                uint32_t again = __ballot_sync(SGA_FULL_MASK, bad);
                while (again) {
                    const int src = __ffs(again) - 1;
                    again &= again - 1;
                    query_row_alone<D>(a, __shfl_sync(SGA_FULL_MASK, row, src), h, __shfl_sync(SGA_FULL_MASK, lo, src),
                                       __shfl_sync(SGA_FULL_MASK, hi, src), hf * HC, hf * HC + HC);
                }
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

template <int D> cudaError_t launch(const SeqArgs &a, cudaStream_t s) {
    BwdParams prm{};
    prm.a = a;
    cudaError_t e = seq_tensor_map(&prm.tq, a.Q, a.rows, a.H, D);
    if (e == cudaSuccess) e = seq_tensor_map(&prm.tg, a.dOut, a.rows, a.H, D);
    if (e == cudaSuccess) e = seq_tensor_map(&prm.tk, a.K, a.rows, a.Hkv, D);
    if (e == cudaSuccess) e = seq_tensor_map(&prm.tv, a.V, a.rows, a.Hkv, D);
    if (e == cudaSuccess) e = allow_smem<seq_bwd_dkdv_kernel<D>>(KvCfg<D>::BYTES + 1024);
    if (e == cudaSuccess) e = allow_smem<seq_bwd_dq_kernel<D>>(QCfg<D>::BYTES + 1024);
    if (e == cudaSuccess) e = seq_row_terms<__nv_bfloat16>(a, D, s);
    if (e != cudaSuccess) return e;
    note_launch(SGA_KERN_SEQ_BWD_DKDV, s, false);
    seq_bwd_dkdv_kernel<D><<<(unsigned)((int64_t)a.n_tiles * a.Hkv), kThreads, KvCfg<D>::BYTES + 1024, s>>>(prm);
    note_launch(SGA_KERN_SEQ_BWD_DKDV, s, true);
    note_launch(SGA_KERN_SEQ_BWD_DQ, s, false);
    seq_bwd_dq_kernel<D><<<(unsigned)((int64_t)a.n_tiles * a.H), kThreads, QCfg<D>::BYTES + 1024, s>>>(prm);
    note_launch(SGA_KERN_SEQ_BWD_DQ, s, true);
    return cudaGetLastError();
}

}  // namespace

cudaError_t seq_bwd_bf16(const SeqArgs &a, int D, cudaStream_t s) {
    return D == 32 ? launch<32>(a, s) : D == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace sga
