"""Attention over packed sequences whose keys share a large offset.  dQ does not
depend on the offset (a row's dS sum to zero), so rounding must not bring it in."""
import math

import pytest
import torch

from dense_ref import ROUND, U

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(lens, H, Hk, D, dt, offset, device, seed=0):
    """Scores of order one beside keys of order `offset`: queries of order 1 / offset."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    n = lambda h: torch.randn(T, h, D, generator=g)
    return [t.to(device, DT[dt]) for t in (n(H) / offset, n(Hk) + offset * (0.75 + 0.5 * torch.rand(Hk, D, generator=g)), n(Hk), n(H))]


def dq_reference(lens, Q, K, V, out, dO, scale, causal, offset):
    """dQ in 64 bits of the operator's formula (Delta from the given out) and the
    bound of an evaluation in fp32 that rounds dS to the inputs' type, but whose
    rounding errors meet keys measured from a point among the row's own.

    R |dS_j| is the most that rounding adds to a weight; it meets k_j - c, where c
    is a mean of some of the row's keys, and so not farther from one of them than
    they are apart (`width`).  Where they are farther apart than |c| / 2, nothing
    is subtracted and it meets k_j, |k_j| <= |c| + width <= 3 width: not at an
    offset of 64, of which a column has 48 or more and spreads by a few.
    Errors of fp32 meet the whole key: of a score (a dot product of D terms and
    the exponential's argument) and of lse (the worst of the row's scores, and a
    sum of n terms) relative to P, of dP and Delta (dot products of D terms), and
    of the products' sum."""
    assert offset == 64 or offset == 1
    far = 1 if offset == 64 else 3
    R, last = (0.0 if Q.dtype == torch.float32 else ROUND[Q.dtype]), ROUND[Q.dtype]
    H, D = Q.shape[1:]
    grp = H // K.shape[1]
    q, k, v, o, do = (t.double() for t in (Q, K, V, out, dO))
    val, bound, at = torch.zeros_like(q), torch.zeros_like(q), 0
    for n in lens:
        s_ = slice(at, at + n)
        at += n
        vis = torch.ones(n, n, dtype=torch.bool, device=Q.device)
        if causal:
            vis = vis.tril()
        for h in range(H):
            ki, vi, qi, di = k[s_, h // grp], v[s_, h // grp], q[s_, h], do[s_, h]
            s = torch.where(vis, scale * (qi @ ki.T), -torch.inf)
            lse = torch.logsumexp(s, 1, keepdim=True)
            p = torch.exp(s - lse)
            delta = (di * o[s_, h]).sum(1, keepdim=True)
            ds = p * (di @ vi.T - delta)
            es = torch.where(vis, (D + 4) * U * scale * (qi.abs() @ ki.abs().T) + 8 * U * (1 + lse.abs()), 0.0)
            ep = es + es.amax(1, keepdim=True) + (n + 16) * U * (1 + lse.abs())
            e32 = ds.abs() * (ep + 4 * U) + p * (D + 4) * U * (di.abs() @ vi.abs().T + (di * o[s_, h]).abs().sum(1, keepdim=True))
            lo = torch.where(vis[:, :, None], ki[None], torch.inf).amin(1)
            hi = torch.where(vis[:, :, None], ki[None], -torch.inf).amax(1)
            val[s_, h] = scale * (ds @ ki)
            bound[s_, h] = scale * (R * ds.abs().sum(1, keepdim=True) * (far * (hi - lo)) + (e32 + (n + 8) * U * ds.abs()) @ ki.abs())
    return val, bound + last * (val.abs() + bound) + 1e-30


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,H,Hk", [([8] * 50 + [1, 2, 3, 5, 13], 2, 2), ([200, 1, 90], 4, 2), ([700, 129], 2, 1)],
                         ids=["short", "middle", "long"])
def test_an_offset_of_the_keys_does_not_reach_dq(dt, D, causal, lens, H, Hk):
    import sparse_graph_attention_csr_gb300 as sga
    ptr = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    plan = sga.SeqPlan(ptr, H, D, DT[dt], kv_heads=Hk, causal=causal)
    for offset in (1.0, 64.0):
        Q, K, V, dO = inputs(lens, H, Hk, D, dt, offset, "cuda", D)
        out, lse = sga.seq_attn_fwd(plan, Q, K, V)
        dQ = sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO)[0]
        val, bound = dq_reference(lens, Q, K, V, out, dO, 1 / math.sqrt(D), causal, offset)
        err = (dQ.double() - val).abs()
        assert (err <= bound).all(), (offset, float((err / bound).max()))


def test_the_bound_tells_one_rounding_from_the_other():
    """On the CPU: dS rounded once to bf16 is outside the bound, and less its
    errors' sum times a mean key inside."""
    lens, D = [8] * 50, 64
    Q, K, V, dO = inputs(lens, 1, 1, D, "bf16", 64.0, "cpu", D)
    scale = 1 / math.sqrt(D)
    out, dq, dq_sub = torch.zeros_like(Q), torch.zeros(400, 1, D), torch.zeros(400, 1, D)
    for i in range(0, 400, 8):
        q, k, v, d = (t[i:i + 8, 0].double() for t in (Q, K, V, dO))
        p = torch.softmax(scale * q @ k.T, 1)
        out[i:i + 8, 0] = (p @ v).bfloat16()
        ds = p * (d @ v.T - (d * out[i:i + 8, 0].double()).sum(1, keepdim=True))
        r = ds.bfloat16().double()
        dq[i:i + 8, 0] = scale * (r @ k)
        dq_sub[i:i + 8, 0] = scale * (r @ k - (r - ds).sum(1, keepdim=True) * k[[1, 3, 5, 7]].mean(0))
    val, bound = dq_reference(lens, Q, K, V, out, dO, scale, False, 64)
    inside = lambda x: ((x.bfloat16().double() - val).abs() <= bound)
    assert inside(dq_sub).all() and not inside(dq).all()
