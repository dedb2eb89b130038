"""Packed-sequence attention with more work than SMs: two row tiles a CTA in the
bf16 forward (two heads of a group, or neighbouring tiles), four blocks an SM in
the fp32 forward, larger tiles in the fp32 backward.  Sizes follow the device."""
import math

import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from dense_ref import seq_reference, within

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def lengths(tiles, rows_a_tile, even=None):
    """Sequences of many lengths that fill more than `tiles` row tiles; their number even or odd."""
    out, total = [], 0
    for n in (700, 1, 129, 0, 333, 64, 500, 2, 38, 255) * 1000:
        if total > tiles * rows_a_tile and (even is None or (total + rows_a_tile - 1) // rows_a_tile % 2 == (not even)):
            return out
        out.append(n)
        total += n
    raise AssertionError


def check(lens, H, Hk, D, dt, causal):
    g = torch.Generator(device="cuda").manual_seed(H * D)
    n = lambda h: torch.randn(sum(lens), h, D, generator=g, device="cuda").to(DT[dt])
    ptr = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    plan = sga.SeqPlan(ptr, H, D, DT[dt], kv_heads=Hk, causal=causal)
    Q, K, V, dO = n(H), n(Hk), n(Hk), n(H)
    out, lse = sga.seq_attn_fwd(plan, Q, K, V)
    grads = sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO)
    assert plan.device_error() == 0
    ref = seq_reference(ptr.cpu(), Q, K, V, 1 / math.sqrt(D), causal, dO, out)
    for name, t in zip(("out", "lse", "dQ", "dK", "dV"), (out, lse, *grads)):
        within(t, ref[name], name)
    return plan, (Q, K, V, dO), (out, lse, *grads)


# 16/4: two heads of a group a CTA; 15/5 and 9/9: neighbouring tiles, their number odd or even
@pytest.mark.parametrize("H,Hk,even", [(16, 4, True), (16, 4, False), (15, 5, True), (15, 5, False), (9, 9, True), (9, 9, False)])
@pytest.mark.parametrize("D,causal", [(32, False), (64, False), (128, False), (128, True)])
def test_two_tiles_a_cta(H, Hk, even, D, causal):
    lens = lengths(2 * sms() // H, 128, even)
    assert (sum(lens) + 127) // 128 * H > 2 * sms()
    check(lens, H, Hk, D, "bf16", causal)


@pytest.mark.parametrize("H,Hk", [(8, 8), (8, 2)])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_fp32_with_many_blocks(H, Hk, D, causal):
    lens = lengths(3 * sms() // (2 * H), 64)
    assert 2 * ((sum(lens) + 63) // 64) * H > 3 * sms()
    check(lens, H, Hk, D, "f32", causal)


@pytest.mark.parametrize("H,Hk", [(16, 4), (9, 9)])
@pytest.mark.parametrize("D", [64, 128])
def test_spoilt_sequence_and_capture(H, Hk, D):
    """A sequence that is NaN throughout leaves the bits of the first one, which
    shares no tile with it, and the others as they were but for the rounding of
    weights; captured and replayed."""
    lens = lengths(2 * sms() // H, 128)
    plan, x, good = check(lens, H, Hk, D, "bf16", False)
    b = 6
    lo, hi = sum(lens[:b]), sum(lens[:b + 1])
    y = [t.clone() for t in x]
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out, lse = sga.seq_attn_fwd(plan, *y[:3])
        got = (out, lse, *sga.seq_attn_bwd(plan, *y[:3], out, lse, y[3]))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, r) for a, r in zip(got, good))
    for t in y:
        t[lo:hi] = math.nan
    g.replay()
    torch.cuda.synchronize()
    for a, r in zip(got, good):
        assert torch.isnan(a[lo:hi]).all()
        assert torch.equal(a[:lens[0]], r[:lens[0]])
        rest = torch.ones(a.shape[0], dtype=torch.bool, device="cuda")
        rest[lo:hi] = False
        assert torch.isfinite(a[rest]).all()
        torch.testing.assert_close(a[rest], r[rest], rtol=2e-2, atol=2e-2)
    assert plan.device_error() == 0
