"""Packed-sequence attention with a sliding window and first rows that stay visible, against the 64-bit definition."""
import numpy as np
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from layer_ref import visible, window_reference, within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def setup(lens, H, Hk, D, dt, causal, window, sinks, pad=0, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ptr = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    T = sum(lens) + pad
    n = lambda h: torch.randn(T, h, D, generator=g, device="cuda").to(dt)
    plan = sga.SeqPlan(ptr, H, D, dt, kv_heads=Hk, causal=causal, window=window, sinks=sinks)
    return plan, ptr, n(H), n(Hk), n(Hk), n(H)


def check(lens, H, Hk, D, dt, causal, window, sinks, pad=0):
    plan, ptr, Q, K, V, dO = setup(lens, H, Hk, D, dt, causal, window, sinks, pad)
    out, lse = sga.seq_attn_fwd(plan, Q, K, V)
    grads = sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO)
    again = sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO)
    assert plan.device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    n = sum(lens)
    if pad:
        assert (out[n:] == 0).all() and (lse[n:] == -torch.inf).all() and all((x[n:] == 0).all() for x in grads)
    cut = lambda x: x[:n]
    ref = window_reference(ptr, cut(Q), cut(K), cut(V), D ** -0.5, causal, window, sinks, cut(dO), cut(out))
    for name, x in {"out": out, "lse": lse, "dQ": grads[0], "dK": grads[1], "dV": grads[2]}.items():
        within(cut(x), ref[name], name)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (17, 4), (64, 0), (65, 1), (127, 5), (128, 128), (129, 2), (200, 130),
                                          (299, 1), (300, 0), (1000, 2), (3, 1000)])
def test_windows_and_sinks(window, sinks, dt, causal):
    check([300, 1, 0, 77, 128, 5], 2, 1, 64, dt, causal, window, sinks)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("H,Hk,D", [(1, 1, 32), (3, 3, 64), (4, 2, 128), (6, 2, 32), (5, 1, 128), (8, 1, 64)])
def test_heads(H, Hk, D, dt, causal):
    check([513, 2, 700, 131], H, Hk, D, dt, causal, 100, 3, pad=9)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("sinks", [1, 140, 700])
def test_cut_walks(sinks, dt, causal):
    """Sequences long enough for their sinks' walks over the queries to be cut into parts (over 32 tiles)."""
    check([130, 4500 if dt == F32 else 6200, 60, 4700 if dt == F32 else 1], 2, 1, 32, dt, causal, 70, sinks, pad=3)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dt", [BF, F32])
def test_many_sequences_and_units(dt, causal):
    """Many short sequences share tiles; enough of them for every choice by the number of units."""
    r = np.random.default_rng(4)
    check(list(r.integers(0, 40, 300)), 4, 4, 32, dt, causal, 6, 2)
    check(list(r.integers(0, 700, 40)), 4, 2, 64, dt, causal, 90, 3)
    if dt == BF:
        check(list(r.integers(0, 900, 40)), 6, 2, 128, dt, causal, 140, 3)   # neighbouring tiles by twos (odd group)


def test_pairs_of_tiles_whose_sinks_differ():
    """Neighbouring tiles of one unit in which another sequence begins, so that their sinks lie in different tiles."""
    for first in (700, 768, 769, 895, 896):
        check([first, 640, 1280] * 6, 3, 1, 128, BF, True, 60, 5)


@pytest.mark.parametrize("dt", [BF, F32])
def test_a_window_over_everything_is_no_window(dt):
    lens = [200, 33, 512]
    for causal in (True, False):
        for window, sinks in ((512, 0), (10 ** 12, 7), (1, 512)):
            plan, ptr, Q, K, V, dO = setup(lens, 4, 2, 64, dt, causal, window, sinks)
            plain = sga.SeqPlan(ptr, 4, 64, dt, kv_heads=2, causal=causal)
            a, b = sga.seq_attn_fwd(plan, Q, K, V), sga.seq_attn_fwd(plain, Q, K, V)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            c, d = sga.seq_attn_bwd(plan, Q, K, V, *a, dO), sga.seq_attn_bwd(plain, Q, K, V, *b, dO)
            assert all(torch.equal(x, y) for x, y in zip(c, d))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("what", ["K", "V", "Q", "dO"])
def test_what_is_not_seen_does_not_reach(what, dt, causal):
    """An infinity or NaN in one row leaves every result that does not see the row as it was, bit for bit."""
    lens, window, sinks = [300, 90, 420], 50, 2
    plan, ptr, Q, K, V, dO = setup(lens, 2, 1, 64, dt, causal, window, sinks)
    vis = torch.block_diag(*[visible(n, causal, window, sinks).float() for n in lens]).bool()   # row i sees key j

    def run():
        out, lse = sga.seq_attn_fwd(plan, Q, K, V)
        return (out, lse, *sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO))

    clean = run()
    T = sum(lens)
    ref = None
    for row, value in ((1, torch.nan), (150, torch.inf), (301, -torch.inf), (500, torch.nan), (809, torch.inf)):
        t = {"K": K, "V": V, "Q": Q, "dO": dO}[what]
        was = t[row].clone()
        t[row, 0, 3] = value
        got = run()
        t[row] = was
        assert plan.device_error() == 0
        # query rows whose own results may change: those that see the key row (K, V), or the row itself
        rows = vis[:, row] if what in "KV" else torch.arange(T, device="cuda") == row
        # keys: seen by such a query row; or the row itself
        keys = vis[rows].any(0)
        if what in "KV":
            keys[row] = True
        if ref is None:
            ref = window_reference(ptr, Q, K, V, 64 ** -0.5, causal, window, sinks, dO, clean[0])
        for name, a, b, may in zip(("out", "lse", "dQ", "dK", "dV"), clean, got, (rows, rows, rows, keys, keys)):
            if what == "dO" and name in ("out", "lse"):
                may = torch.zeros_like(rows)
            assert torch.isfinite(b[~may]).all(), (name, row)
            # (what was computed again, alone, is summed in another order)
            value_, bound = ref[name]
            err = (b.double() - value_).abs()
            assert (err[~may] <= bound[~may]).all(), (name, row)


def test_gradients_against_differences():
    plan, ptr, Q, K, V, dO = setup([90, 40], 2, 1, 32, F32, True, 20, 2)
    f = lambda q, k, v: float((sga.seq_attn_fwd(plan, q, k, v)[0].double() * dO.double()).sum())
    out, lse = sga.seq_attn_fwd(plan, Q, K, V)
    grads = sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO)
    g = torch.Generator(device="cuda").manual_seed(1)
    xs = (Q, K, V)
    for i, d in enumerate(grads):
        v = torch.randn(xs[i].shape, generator=g, device="cuda")
        v /= v.norm()
        up, down = (f(*(x + s * 2.0 ** -6 * v if j == i else x for j, x in enumerate(xs))) for s in (1, -1))
        assert abs((up - down) * 2.0 ** 5 - float((d.double() * v.double()).sum())) < 2e-3 * float(d.double().norm())


@pytest.mark.parametrize("dt", [BF, F32])
def test_captured_overlapping_and_on_streams(dt):
    plan, ptr, Q, K, V, dO = setup([700, 1, 5000], 4, 2, 64, dt, True, 90, 3)

    def call():
        out, lse = sga.seq_attn_fwd(plan, Q, K, V)
        return (out, lse, *sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO))

    want = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    s = torch.cuda.Stream()
    for _ in range(3):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = call()
        graph.replay()
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip(other, want))
    assert plan.device_error() == 0


def test_refusals():
    ptr = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    for window, sinks in ((0, 0), (-1, 0), (None, 1), (4, -1)):
        with pytest.raises(ValueError, match="window|sinks"):
            sga.SeqPlan(ptr, 1, 32, window=window, sinks=sinks)
