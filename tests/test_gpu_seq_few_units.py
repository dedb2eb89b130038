"""A sequence's rows are the same, bit for bit, alone and among enough others that their results are stored another way."""
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("window", [None, 40])
@pytest.mark.parametrize("rows", [1, 76, 300])
def test_alone_and_among_others(rows, window, D):
    H, Hk, B = 4, 2, torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda h: torch.randn(rows, h, D, generator=g, device="cuda").bfloat16()
    Q, K, V = n(H), n(Hk), n(Hk)

    def call(copies, fill):
        ptr = torch.arange(copies + 1, device="cuda", dtype=torch.int32) * 384   # (each begins on a tile)
        pad = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, 384 - rows)).repeat(copies, 1, 1)
        plan = sga.SeqPlan(ptr, H, D, kv_heads=Hk, causal=True, window=window)
        out = torch.full((384 * copies, H, D), fill, device="cuda", dtype=torch.bfloat16)
        lse = torch.empty(384 * copies, H, device="cuda")
        sga.seq_attn_fwd(plan, pad(Q), pad(K), pad(V), out=out, lse=lse)
        assert plan.device_error() == 0
        return out.view(copies, 384, H, D), lse.view(copies, 384, H)

    (a, la), (b, lb) = call(1, 3.0), call(B, torch.nan)
    assert torch.isfinite(b).all() and torch.equal(b, a.expand_as(b)) and torch.equal(lb, la.expand_as(lb))


def test_rows_behind_the_last_sequence_stay():
    for copies in (1, 400):
        T = 76 * copies
        n = lambda: torch.randn(T + 9, 4, 64, device="cuda").bfloat16()
        plan = sga.SeqPlan(torch.arange(copies + 1, device="cuda", dtype=torch.int32) * 76, 4, 64)
        out = torch.full((T + 9, 4, 64), 3.0, device="cuda", dtype=torch.bfloat16)
        lse = torch.full((T + 9, 4), 3.0, device="cuda")
        sga.seq_attn_fwd(plan, n(), n(), n(), out=out, lse=lse)
        assert (out[T:] == 3).all() and (lse[T:] == 3).all() and (out[:T] != 3).float().mean() > 0.9
