"""Calls of the embedding gradient at the edges of its range."""
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from dense_ref import embed_bwd_reference, within

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def microseconds(f, n=10):
    for _ in range(3):
        f()
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    t0.record()
    for _ in range(n):
        f()
    t1.record()
    torch.cuda.synchronize()
    return t0.elapsed_time(t1) / n * 1e3


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 100, 300])
def test_few_tokens_into_a_large_table(N, dt):
    """Most of the work is a table of zeros: no more than three fills of it and
    the steps of the sort (some ten barriers of the whole grid, 60 us)."""
    V, C = 50257, 512
    ids = torch.randint(0, V, (N,), device="cuda")
    ids[N // 2:] = int(ids[0])
    dO = torch.randn(N, C, device="cuda").to(DT[dt])
    dT = sga.embed_bwd(ids, dO, V, 0.5)
    within(dT, embed_bwd_reference(ids, dO, V, 0.5))
    fill = microseconds(lambda: dT.fill_(0))
    took = microseconds(lambda: sga.embed_bwd(ids, dO, V, 0.5, dTable=dT))
    print(f"{N} {dt}: {took:.1f} us, a fill {fill:.1f} us")
    assert took <= 3 * fill + 60


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,C", [(1, 1, 1 << 20), (8, 5, 65536), (8, 5, 65537), (1000, 1, 4096), (1000, 1, 16384), (1000, 5, 4096), (1000, 5, 16387),
                                   (130, 16, 20000), (100, 300, 65536), (1000, 300, 16384), (1000, 300, 16385), (700, 17, 5000)])
def test_wide_rows(N, V, C, dt):
    """Wide rows and few tokens, into few rows and (300) sorted, with a frequent
    row: right, reproducible, and no longer than the sum in plain torch."""
    g = torch.Generator(device="cuda").manual_seed(C + V)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda")
    ids[torch.rand(N, generator=g, device="cuda") < 0.5] = V // 2
    dO = torch.randn(N, C, generator=g, device="cuda").to(DT[dt])
    table = torch.randn(V, C, generator=g, device="cuda").to(DT[dt])
    dT = sga.embed_bwd(ids, dO, V, 0.5)
    within(dT, embed_bwd_reference(ids, dO, V, 0.5))
    assert torch.equal(dT, sga.embed_bwd(ids, dO, V, 0.5))
    assert torch.equal(sga.embed_fwd(ids, table, 0.5), (table[ids].float() * 0.5).to(DT[dt]))
    bwd = microseconds(lambda: sga.embed_bwd(ids, dO, V, 0.5, dTable=dT))
    fwd = microseconds(lambda: sga.embed_fwd(ids, table, 0.5))
    plain_bwd = microseconds(lambda: (torch.zeros(V, C, dtype=torch.float64, device="cuda").index_add_(0, ids, dO.double()) * 0.5).to(DT[dt]))
    plain_fwd = microseconds(lambda: (table[ids].float() * 0.5).to(DT[dt]))
    print(f"{N} into {V} x {C} {dt}: backward {bwd:.1f} us (torch {plain_bwd:.1f}), forward {fwd:.1f} (torch {plain_fwd:.1f})")
    assert bwd <= plain_bwd and fwd <= plain_fwd
