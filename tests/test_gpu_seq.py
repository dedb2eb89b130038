"""Attention over packed sequences against its definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from dense_ref import seq_reference, within

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def ptr_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def make(lens, H, Hk, D, dt, seed=0, tail=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = int(sum(lens)) + tail
    n = lambda h: torch.randn(T, h, D, generator=g, device="cuda").to(DT[dt])
    return ptr_of(lens), n(H), n(Hk), n(Hk), n(H)


def check(lens, H, Hk, D, dt, causal, scale=None, seed=0, tail=0):
    sp, Q, K, V, dO = make(lens, H, Hk, D, dt, seed, tail)
    plan = sga.SeqPlan(sp, H, D, DT[dt], kv_heads=Hk, causal=causal)
    R = plan.rows
    if tail:   # rows behind the last sequence may hold anything
        for t in (Q, K, V, dO):
            t[R:] = float("nan")
    out, lse = sga.seq_attn_fwd(plan, Q, K, V, scale)
    dQ, dK, dV = sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO, scale)
    torch.cuda.synchronize()
    assert plan.device_error() == 0
    ref = seq_reference(sp.cpu(), Q[:R], K[:R], V[:R], 1 / math.sqrt(D) if scale is None else scale, causal, dO[:R], out[:R])
    for name, t in (("out", out), ("lse", lse), ("dQ", dQ), ("dK", dK), ("dV", dV)):
        within(t[:R], ref[name], f"{name} {lens[:6]} H{H}/{Hk} D{D} {dt} causal={causal}")
        if tail:
            assert (t[R:] == (-math.inf if name == "lse" else 0)).all()
    return out, lse, dQ, dK, dV


LENS = [[1], [2], [63], [64], [65], [127], [128], [129], [257], [1, 1, 1], [5, 0, 0, 123, 1, 300], [0, 0, 7], [40] * 20,
        [255, 1, 128, 129]]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x[:6])))
def test_lengths(lens, dt, causal):
    check(lens, 2, 2, 64, dt, causal, seed=len(lens))


@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 1), (3, 1), (6, 2), (8, 8), (5, 5), (16, 4)])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_heads(H, Hk, D, dt):
    check([150, 1, 77, 260], H, Hk, D, dt, True, seed=H)
    check([150, 1, 77, 260], H, Hk, D, dt, False, seed=H)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
def test_long(dt, causal):
    check([1900, 3, 700], 2, 1, 128, dt, causal)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-3, 1.0, 3.0])
def test_scale(dt, scale):
    """Scores from nearly equal to so far apart that a row has one weight."""
    check([200, 90], 2, 2, 32, dt, True, scale)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_behind_the_last_sequence(dt):
    check([100, 60], 2, 1, 64, dt, True, tail=70)
    # given results keep what they held there
    sp, Q, K, V, dO = make([100, 60], 2, 1, 64, dt, tail=70)
    plan = sga.SeqPlan(sp, 2, 64, DT[dt], kv_heads=1)
    full = lambda t, x: torch.full_like(t, x)
    out, lse = full(Q, 7.0), torch.full((230, 2), 7.0, device="cuda")
    sga.seq_attn_fwd(plan, Q, K, V, out=out, lse=lse)
    g = [full(t, 7.0) for t in (Q, K, V)]
    sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO, dQ=g[0], dK=g[1], dV=g[2])
    for t in (out, lse, *g):
        assert (t[160:] == 7).all() and not (t[:160] == 7).all()


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_a_row_does_not_see_does_not_reach_it(dt, D, bad):
    """One sequence is spoilt in every tensor; the others give the same bits as
    before.  Under causal, a spoilt last row leaves the rows before it."""
    lens = [50, 70, 30, 200]
    for causal in (True, False):
        sp, Q, K, V, dO = make(lens, 4, 2, D, dt)
        plan = sga.SeqPlan(sp, 4, D, DT[dt], kv_heads=2, causal=causal)
        out, lse = sga.seq_attn_fwd(plan, Q, K, V)
        good = (out, lse, *sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO))
        x = [t.clone() for t in (Q, K, V, dO)]
        for t in x:
            t[50:120] = bad
        out, lse = sga.seq_attn_fwd(plan, *x[:3])
        got = (out, lse, *sga.seq_attn_bwd(plan, *x[:3], out, lse, x[3]))
        for name, a, b in zip(("out", "lse", "dQ", "dK", "dV"), got, good):
            assert torch.isfinite(a[:50]).all() and torch.isfinite(a[120:]).all(), name
            for s in (slice(0, 50), slice(120, None)):
                torch.testing.assert_close(a[s], b[s], rtol=2e-2 if dt == "bf16" else 1e-4, atol=2e-2 if dt == "bf16" else 1e-4)
    sp, Q, K, V, _ = make(lens, 4, 2, D, dt)
    plan = sga.SeqPlan(sp, 4, D, DT[dt], kv_heads=2)
    good, _ = sga.seq_attn_fwd(plan, Q, K, V)
    for t in (K, V):
        t[349] = bad
    got, _ = sga.seq_attn_fwd(plan, Q, K, V)
    assert torch.isfinite(got[:349]).all()
    torch.testing.assert_close(got[:349], good[:349], rtol=2e-2 if dt == "bf16" else 1e-4, atol=2e-2 if dt == "bf16" else 1e-4)
    assert not torch.isfinite(got[349]).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_bitwise_reproducible(dt):
    a = check([700, 300], 4, 2, 64, dt, True, seed=3)
    b = check([700, 300], 4, 2, 64, dt, True, seed=3)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_autograd_and_empty():
    sp, Q, K, V, dO = make([90, 200], 4, 2, 64, "bf16")
    plan = sga.SeqPlan(sp, 4, 64, kv_heads=2)
    out, lse = sga.seq_attn_fwd(plan, Q, K, V)
    ref = sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO)
    x = [t.clone().requires_grad_() for t in (Q, K, V)]
    o = sga.SeqAttention.apply(*x, plan)
    o.backward(dO)
    assert torch.equal(o, out)
    for t, r in zip(x, ref):
        assert torch.equal(t.grad, r)
    # a gradient that is one value for every element, of zero strides
    y = [t.clone().requires_grad_() for t in (Q, K, V)]
    sga.SeqAttention.apply(*y, plan).sum().backward()
    ones = sga.seq_attn_bwd(plan, Q, K, V, out, lse, torch.ones_like(Q))
    for t, r in zip(y, ones):
        assert torch.equal(t.grad, r)
    for lens in ([], [0], [0, 0, 0]):
        p = sga.SeqPlan(ptr_of(lens), 2, 32, torch.float32)
        e = torch.empty(0, 2, 32, device="cuda")
        out, lse = sga.seq_attn_fwd(p, e, e, e)
        assert out.shape == e.shape and lse.shape == (0, 2)
        assert all(t.shape == e.shape for t in sga.seq_attn_bwd(p, e, e, e, out, lse, e))


def test_gradients_against_differences():
    """d(sum(out * G)) along a random direction, by central differences in fp32."""
    sp, Q, K, V, G = make([40, 25], 2, 1, 32, "f32")
    plan = sga.SeqPlan(sp, 2, 32, torch.float32, kv_heads=1)
    x = [t.clone().requires_grad_() for t in (Q, K, V)]
    sga.SeqAttention.apply(*x, plan).backward(G)
    h = 1e-2
    for i, t in enumerate((Q, K, V)):
        d = torch.randn_like(t)
        args = lambda s: [u + s * h * d if j == i else u for j, u in enumerate((Q, K, V))]
        f = lambda s: (sga.seq_attn_fwd(plan, *args(s))[0].double() * G.double()).sum()
        num, ana = float((f(1) - f(-1)) / (2 * h)), float((x[i].grad.double() * d.double()).sum())
        # truncation h^2 / 6 f''' (f''' of order the gradient's size) and fp32 noise / h
        assert abs(num - ana) <= 1e-3 * float(x[i].grad.norm() * d.norm()), (i, num, ana)


def test_streams_graphs_and_overlap():
    sp, Q, K, V, dO = make([333, 50, 700], 4, 4, 64, "bf16")
    plan = sga.SeqPlan(sp, 4, 64)
    out, lse = sga.seq_attn_fwd(plan, Q, K, V)
    ref = (out, lse, *sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO))
    torch.cuda.synchronize()
    # two streams at once on one plan
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    res = []
    for _ in range(4):
        for s in streams:
            o, l = sga.seq_attn_fwd(plan, Q, K, V, stream=s)
            res.append((o, l, *sga.seq_attn_bwd(plan, Q, K, V, o, l, dO, stream=s)))
    torch.cuda.synchronize()
    for r in res:
        for a, b in zip(r, ref):
            assert torch.equal(a, b)
    # two captured graphs of both directions, replayed together on new inputs
    graphs = []
    for s in streams:
        x = [t.clone() for t in (Q, K, V, dO)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            o, l = sga.seq_attn_fwd(plan, *x[:3])
            r = (o, l, *sga.seq_attn_bwd(plan, *x[:3], o, l, x[3]))
        graphs.append((g, x, r))
    for _, x, _ in graphs:
        for t in x:
            t.neg_()
    torch.cuda.synchronize()
    for s, (g, _, _) in zip(streams, graphs):
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    o, l = sga.seq_attn_fwd(plan, -Q, -K, -V)
    want = (o, l, *sga.seq_attn_bwd(plan, -Q, -K, -V, o, l, -dO))
    for _, _, r in graphs:
        for a, b in zip(r, want):
            assert torch.equal(a, b)
    assert plan.device_error() == 0


def test_inputs_freed_while_another_stream_uses_them():
    """The inputs of a call on a given stream are dropped, and their memory is
    asked for again, before that stream has begun: the allocator has to hold it."""
    sp, Q, K, V, dO = make([1500, 700], 4, 4, 64, "bf16")
    plan = sga.SeqPlan(sp, 4, 64)
    out, lse = sga.seq_attn_fwd(plan, Q, K, V)
    ref = sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    gate = torch.randn(6000, 6000, device="cuda")
    x = [t.clone() for t in (Q, K, V, dO)]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(8):
            gate = gate @ gate * 1e-4   # keeps the stream busy for some milliseconds
    o, l = sga.seq_attn_fwd(plan, *x[:3], stream=s)
    g = sga.seq_attn_bwd(plan, *x[:3], o, l, x[3], stream=s)
    shapes = [t.shape for t in x]
    del x
    junk = [torch.full(sh, float("nan"), device="cuda", dtype=torch.bfloat16) for sh in shapes for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(o, out) and all(torch.equal(a, b) for a, b in zip(g, ref))
    del junk


def test_a_batch_that_is_nan_throughout():
    """Results are NaN, and no row is computed again for it (4096 rows would
    take seconds)."""
    for dt in ("bf16", "f32"):
        sp, Q, K, V, dO = make([4096], 2, 2, 64, dt)
        for t in (Q, K, V, dO):
            t.fill_(float("nan"))
        plan = sga.SeqPlan(sp, 2, 64, DT[dt])
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        out, lse = sga.seq_attn_fwd(plan, Q, K, V)
        g = sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO)
        t1.record()
        torch.cuda.synchronize()
        assert all(torch.isnan(t).all() for t in (out, *g))
        assert t0.elapsed_time(t1) < 200


def test_refusals():
    sp = ptr_of([10, 20])
    for bad in ([1, 5], [0, 5, 4], [0, -1]):
        with pytest.raises(sga.SgaError):
            sga.SeqPlan(torch.tensor(bad, dtype=torch.int32, device="cuda"), 2, 64)
    for H, D, hk in ((2, 48, 2), (3, 64, 2), (0, 64, 1), (256, 128, 1)):
        with pytest.raises(sga.SgaError):
            sga.SeqPlan(sp, H, D, kv_heads=hk)
    plan = sga.SeqPlan(sp, 2, 64, kv_heads=1)
    Q, K = torch.randn(30, 2, 64, device="cuda").bfloat16(), torch.randn(30, 1, 64, device="cuda").bfloat16()
    with pytest.raises(ValueError):
        sga.seq_attn_fwd(plan, Q[:29].contiguous(), K[:29].contiguous(), K[:29].contiguous())
    with pytest.raises(ValueError):
        sga.seq_attn_fwd(plan, Q, Q, Q)
    with pytest.raises(TypeError):
        sga.seq_attn_fwd(plan, Q.float(), K, K)
    with pytest.raises(ValueError):
        sga.seq_attn_fwd(plan, Q, K, Q[:, :1])
    for scale in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(ValueError):
            sga.seq_attn_fwd(plan, Q, K, K, scale)
    out, lse = sga.seq_attn_fwd(plan, Q, K, K)
    with pytest.raises(ValueError, match="shares memory"):
        sga.seq_attn_fwd(plan, Q, K, K, out=Q)
    with pytest.raises(ValueError, match="shares memory"):
        sga.seq_attn_bwd(plan, Q, K, K, out, lse, Q, dK=K)
    # off a 16-byte boundary: refused by the library before any launch
    off = torch.empty(30 * 2 * 64 + 1, device="cuda").bfloat16()[1:].view(30, 2, 64)
    with pytest.raises(sga.SgaError):
        sga.seq_attn_fwd(plan, off, K, K)


@pytest.mark.parametrize("scale", [1e39, 1e-60])
def test_scale_past_float32(scale):
    plan = sga.SeqPlan(ptr_of([10, 20]), 2, 64)
    Q = torch.randn(30, 2, 64, device="cuda").bfloat16()
    with pytest.raises(ValueError, match="scale"):
        sga.seq_attn_fwd(plan, Q, Q, Q, scale)
