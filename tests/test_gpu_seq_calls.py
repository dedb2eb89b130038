"""Calls of packed-sequence attention at the edges of what its documentation allows."""
import threading

import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def ptr_of(lens):
    return torch.tensor([0] + list(lens), device="cuda").cumsum(0).int()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_largest_scale(dt):
    """Scores are held in units of log2: a scale whose product with log2(e)
    leaves float32 is refused, the largest below it gives the mean of V for
    scores of zero (2^-8 and 2^-24 of a mean of 20 values around one)."""
    plan = sga.SeqPlan(ptr_of([20]), 2, 64, DT[dt], causal=False)
    Q, K = torch.zeros(20, 2, 64, device="cuda", dtype=DT[dt]), torch.randn(20, 2, 64, device="cuda").to(DT[dt])
    for scale in (2.4e38, 3e38):
        with pytest.raises(ValueError, match="scale"):
            sga.seq_attn_fwd(plan, Q, K, K, scale)
        with pytest.raises(ValueError, match="scale"):
            sga.seq_attn_bwd(plan, Q, K, K, Q, torch.zeros(20, 2, device="cuda"), K, scale)
    out, lse = sga.seq_attn_fwd(plan, Q, K, K, 2.3e38)
    mean = K.double().mean(0, keepdim=True)
    bound = (2 ** -8 if dt == "bf16" else 0) * K.double().abs().mean(0) + 32 * 2 ** -24 * K.double().abs().mean(0)
    last = (2 ** -8 if dt == "bf16" else 2 ** -24) * (mean.abs() + bound)
    assert ((out.double() - mean).abs() <= bound + last).all()


@pytest.mark.parametrize("where", ["here", "another thread"])
def test_plans_dropped_during_a_capture(where):
    """Plans that the capture does not use, freed while it runs: it goes on."""
    ptr = ptr_of([20, 300])
    plans = [sga.SeqPlan(ptr, 3, 64), sga.SeqPlan(ptr, 2, 32, torch.float32), sga.Plan(ptr_of([1] * 320), ptr_of([1] * 319), 2, 32)]
    kept, Q = sga.SeqPlan(ptr, 2, 64), torch.randn(320, 2, 64, device="cuda").bfloat16()
    want = sga.seq_attn_fwd(kept, Q, Q, Q)[0]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        if where == "here":
            plans.clear()
        else:
            t = threading.Thread(target=plans.clear)
            t.start()
            t.join()
        out = sga.seq_attn_fwd(kept, Q, Q, Q)[0]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and kept.device_error() == 0
