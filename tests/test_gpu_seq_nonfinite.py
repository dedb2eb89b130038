"""Infinities and NaN in single rows of packed sequences: what they reach, and what they cost."""
import math

import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# a redone column holds unrounded weights, the others bf16 ones: 2^-8 of sums of weights of one each
TOL = {"f32": dict(rtol=1e-4, atol=1e-4), "bf16": dict(rtol=2e-2, atol=2e-2)}


def setup(lens, H, Hk, D, dt, causal, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda h: torch.randn(sum(lens), h, D, generator=g, device="cuda").to(DT[dt])
    ptr = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    return sga.SeqPlan(ptr, H, D, DT[dt], kv_heads=Hk, causal=causal), [n(H), n(Hk), n(Hk), n(H)]


def both(plan, Q, K, V, dO):
    out, lse = sga.seq_attn_fwd(plan, Q, K, V)
    return (out, lse, *sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("causal", [True, False])
def test_one_value_reaches_its_column_of_the_rows_that_see_it(dt, D, bad, causal):
    """lens 300, 700, 20; the value is in the middle sequence, one column of V, K or dOut."""
    lens, p, c = [300, 700, 20], 300 + 333, D - 5
    plan, x = setup(lens, 4, 2, D, dt, causal)
    good = both(plan, *x)
    rows = torch.arange(sum(lens), device="cuda")
    inside = (rows >= 300) & (rows < 1000)
    later, earlier = (inside & (rows >= p), inside & (rows <= p)) if causal else (inside, inside)

    def check(got, ref, name, cells):
        """not finite in `cells`, elsewhere as before"""
        assert not torch.isfinite(got[cells]).any(), name
        assert torch.isfinite(got[~cells]).all(), name
        torch.testing.assert_close(got[~cells], ref[~cells], **TOL[dt])

    def cells(t, at, head=None, col=None):
        m = torch.zeros_like(t, dtype=torch.bool)
        m[at] = True
        if head is not None:
            keep = torch.zeros_like(m)
            keep[:, head] = True
            m &= keep
        if col is not None:
            keep = torch.zeros_like(m)
            keep[..., col] = True
            m &= keep
        return m

    # V of key head 1: out of query heads 2, 3
    y = [t.clone() for t in x]
    y[2][p, 1, c] = bad
    out, lse = sga.seq_attn_fwd(plan, *y[:3])
    check(out, good[0], "out", cells(out, later, slice(2, 4), c))
    assert torch.equal(lse, good[1])
    other = torch.ones(D, dtype=torch.bool, device="cuda")
    other[c] = False
    assert torch.equal(out[..., other], good[0][..., other])
    # dOut of head 3, the forward's results as they were: dV of key head 1 in its column; dQ of its own row
    # and dK of the keys it sees throughout (dP is not finite)
    y = [t.clone() for t in x]
    y[3][p, 3, c] = bad
    dQ, dK, dV = sga.seq_attn_bwd(plan, *y[:3], good[0], good[1], y[3])
    check(dV, good[4], "dV", cells(dV, earlier, 1, c))
    check(dQ, good[2], "dQ", cells(dQ, rows == p, 3))
    check(dK, good[3], "dK", cells(dK, earlier, 1))
    # Q of head 2, whose scores are then not finite
    y = [t.clone() for t in x]
    y[0][p, 2, c] = math.nan
    got = both(plan, *y)
    check(got[0], good[0], "out", cells(got[0], rows == p, 2))
    check(got[2], good[2], "dQ", cells(got[2], rows == p, 2))
    check(got[3], good[3], "dK", cells(got[3], earlier, 1))
    check(got[4], good[4], "dV", cells(got[4], earlier, 1))
    # K of key head 0
    y = [t.clone() for t in x]
    y[1][p, 0, c] = math.nan
    got = both(plan, *y)
    check(got[0], good[0], "out", cells(got[0], later, slice(0, 2)))
    check(got[2], good[2], "dQ", cells(got[2], later, slice(0, 2)))


def milliseconds(f):
    f()
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    t0.record()
    f()
    t1.record()
    torch.cuda.synchronize()
    return t0.elapsed_time(t1)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["token", "V", "dOut", "all V"])
def test_what_one_value_costs(dt, which):
    """8192 causal rows: one token that is NaN, one infinity in V, one NaN in dOut,
    V all NaN.  The rows that see it are some thousand a head; walked one by one
    over their intervals they would take hundreds of milliseconds.  What is
    allowed is the walks of one tile (at most 127 rows of a head, 32 a warp one
    after the other, of 8192 steps of some 100 cycles: 14 ms a direction, twice
    that for dK beside dV) and ten times the call itself."""
    plan, x = setup([8192], 4, 2, 64, dt, True)
    p = 2000
    if which == "token":
        for t in x:
            t[p] = math.nan
    elif which == "V":
        x[2][p, 0, 7] = math.inf
    elif which == "dOut":
        x[3][p, 0, 7] = math.nan
    else:
        x[2].fill_(math.nan)
    clean = setup([8192], 4, 2, 64, dt, True)[1]
    base = milliseconds(lambda: both(plan, *clean))
    took = milliseconds(lambda: both(plan, *x))
    print(f"{dt} {which}: {base:.3f} ms clean, {took:.3f} ms")
    assert took <= 45 + 10 * base
