"""Embedding lookup and its gradient by sorted tokens, against 64 bits."""
import math

import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from dense_ref import ROUND, embed_bwd_reference, within

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def zipf(N, V, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(V + 1)) - 1).floor().clamp(0, V - 1).to(dtype)


def check(N, V, C, dt, ids_dt=torch.int64, ids=None, scale=1.7, padding_idx=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = zipf(N, V, ids_dt, seed) if ids is None else ids
    table = torch.randn(V, C, generator=g, device="cuda").to(DT[dt])
    dO = torch.randn(N, C, generator=g, device="cuda").to(DT[dt])
    out = sga.embed_fwd(ids, table, scale)
    dT = sga.embed_bwd(ids, dO, V, scale, padding_idx)
    torch.cuda.synchronize()
    val = table.double()[ids.long()] * scale
    # the scale itself is rounded to fp32
    within(out, (val, (ROUND[DT[dt]] + 2 ** -23) * val.abs() + 1e-30), "out")
    v, b = embed_bwd_reference(ids, dO, V, scale, padding_idx)
    within(dT, (v, b + 2 ** -24 * v.abs()), "dTable")
    assert sga.embed_device_error() == 0
    return out, dT


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 3, 4, 8, 31, 100, 128, 256, 260, 301, 512, 1024, 1500, 4096])
def test_widths(C, dt):
    check(500, 37, C, dt, seed=C)


@pytest.mark.parametrize("ids_dt", [torch.int32, torch.int64])
@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 33, 1000, 1024, 1025, 4097, 100003])
@pytest.mark.parametrize("V", [1, 2, 119, 256, 257, 70000])
def test_tokens(N, V, ids_dt):
    check(N, V, 64, "bf16", ids_dt, seed=N)


def test_one_row_takes_all_and_runs_cross_chunks():
    N = 200000
    check(N, 5, 40, "f32", ids=torch.full((N,), 3, device="cuda"))
    ids = torch.arange(N, device="cuda") // 1000      # every row a thousand tokens, in order
    check(N, 300, 40, "f32", ids=ids)
    check(N, 200000, 8, "bf16", ids=torch.arange(N, device="cuda").flip(0))   # every row one


def test_sum_of_ones_is_the_count():
    """Whole numbers, exact in fp32: every token is summed once."""
    N, V = 300001, 1003
    ids = zipf(N, V, torch.int64, 5)
    dT = sga.embed_bwd(ids, torch.ones(N, 12, device="cuda"), V)
    assert torch.equal(dT, torch.bincount(ids, minlength=V).float()[:, None].expand(V, 12))


def test_padding_bad_ids_and_empty():
    ids = torch.tensor([0, 3, -1, 7, 3, 2 ** 40, 2], device="cuda")
    table = torch.randn(7, 16, device="cuda")
    out = sga.embed_fwd(ids, table)
    assert sga.embed_device_error() == 1 and sga.embed_device_error() == 0
    ok = torch.tensor([True, True, False, False, True, False, True], device="cuda")
    assert (out[~ok] == 0).all() and torch.equal(out[ok], table[ids[ok]])
    dO = torch.randn(7, 16, device="cuda")
    dT = sga.embed_bwd(ids, dO, 7, padding_idx=3)
    assert sga.embed_device_error() == 1
    v, b = embed_bwd_reference(ids, dO, 7, 1.0, 3)
    within(dT, (v, b))
    assert (dT[3] == 0).all()
    # a NaN in a row that nobody reads, and in the gradient of a padded token, stays there
    table[1] = math.nan
    dO[1] = dO[4] = math.nan
    assert torch.isfinite(sga.embed_fwd(ids[ok], table)).all()
    assert torch.isfinite(sga.embed_bwd(ids[ok], dO[ok], 7, padding_idx=3)).all()
    e = torch.empty(0, dtype=torch.int64, device="cuda")
    assert sga.embed_fwd(e, table).shape == (0, 16)
    assert (sga.embed_bwd(e, torch.empty(0, 16, device="cuda"), 7) == 0).all()
    assert sga.embed_bwd(e, torch.empty(0, 16, device="cuda"), 0).shape == (0, 16)
    assert sga.embed_device_error() == 0


def test_shapes_and_offsets():
    ids = zipf(60, 20, torch.int32).view(3, 20)
    table = torch.randn(20, 24, device="cuda").bfloat16()
    out = sga.embed_fwd(ids, table, 2.0)
    assert out.shape == (3, 20, 24) and torch.equal(out, table[ids.long()] * 2)
    off = torch.empty(20 * 24 + 1, device="cuda").bfloat16()[1:].view(20, 24)
    off.copy_(table)
    assert torch.equal(sga.embed_fwd(ids, off, 2.0), out)
    dO = torch.randn(3, 20, 24, device="cuda").bfloat16()
    dT = sga.embed_bwd(ids, dO, 20)
    odd = torch.empty(60 * 24 + 1, device="cuda").bfloat16()[1:].view(3, 20, 24)
    odd.copy_(dO)
    assert torch.equal(sga.embed_bwd(ids, odd, 20), dT)


def test_autograd_and_reproducible():
    ids = zipf(5000, 300, torch.int64).view(50, 100)
    table = torch.randn(300, 64, device="cuda").bfloat16().requires_grad_()
    dO = torch.randn(50, 100, 64, device="cuda").bfloat16()
    out = sga.Embedding.apply(ids, table, 0.5, 2)
    out.backward(dO)
    assert torch.equal(out, sga.embed_fwd(ids, table.detach(), 0.5))
    for _ in range(3):
        assert torch.equal(table.grad, sga.embed_bwd(ids, dO, 300, 0.5, 2))
    t2 = table.detach().clone().requires_grad_()
    sga.Embedding.apply(ids.t(), t2).sum().backward()
    count = torch.bincount(ids.flatten(), minlength=300).float()[:, None].expand(300, 64)
    assert torch.equal(t2.grad, count.bfloat16())


def test_gradient_against_differences():
    ids = zipf(100, 9, torch.int64)
    table, G, d = (torch.randn(*s, device="cuda") for s in ((9, 10), (100, 10), (9, 10)))
    f = lambda s: (sga.embed_fwd(ids, table + s * d, 3.0).double() * G.double()).sum()
    num, ana = float((f(1) - f(-1)) / 2), float((sga.embed_bwd(ids, G, 9, 3.0).double() * d.double()).sum())
    assert abs(num - ana) <= 1e-4 * max(1.0, abs(ana))   # linear in the table: rounding only


def test_streams_and_graphs():
    ids = zipf(50000, 1000, torch.int64)
    dO = torch.randn(50000, 64, device="cuda").bfloat16()
    ref = sga.embed_bwd(ids, dO, 1000)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    res = [sga.embed_bwd(ids, dO, 1000, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(r, ref) for r in res)
    graphs = []
    for s in streams:
        i = ids.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r = sga.embed_bwd(i, dO, 1000)
        graphs.append((s, g, i, r))
    for _, _, i, _ in graphs:
        i.copy_(999 - ids)
    torch.cuda.synchronize()
    for s, g, _, _ in graphs:
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    for _, _, _, r in graphs:
        assert torch.equal(r, ref.flip(0))


def test_refusals():
    ids, table = zipf(10, 5, torch.int64), torch.randn(5, 8, device="cuda")
    with pytest.raises(TypeError):
        sga.embed_fwd(ids.short(), table)
    with pytest.raises(TypeError):
        sga.embed_fwd(ids, table.half())
    with pytest.raises(ValueError):
        sga.embed_fwd(ids, table.t())
    with pytest.raises(ValueError):
        sga.embed_fwd(ids, table, math.nan)
    with pytest.raises(ValueError):
        sga.embed_fwd(ids, table, out=torch.empty(9, 8, device="cuda"))
    with pytest.raises(ValueError):
        sga.embed_bwd(ids, torch.randn(9, 8, device="cuda"), 5)
    for p in (-1, 5):
        with pytest.raises(ValueError):
            sga.embed_bwd(ids, torch.randn(10, 8, device="cuda"), 5, padding_idx=p)
        with pytest.raises(ValueError):
            sga.Embedding.apply(ids, table, 1.0, p)   # in the forward, not first in the backward
    with pytest.raises(ValueError):
        sga.embed_bwd(ids, torch.randn(10, 8, device="cuda"), -1)


@pytest.mark.parametrize("scale", [1e39, -1e39])
def test_scale_past_float32(scale):
    ids, table = zipf(10, 5, torch.int64), torch.randn(5, 8, device="cuda")
    with pytest.raises(ValueError, match="scale"):
        sga.embed_fwd(ids, table, scale)
    with pytest.raises(ValueError, match="scale"):
        sga.embed_bwd(ids, torch.randn(10, 8, device="cuda"), 5, scale)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C", [8, 31, 100, 400])
def test_few_rows_off_a_16_byte_boundary(C, dt):
    """Few rows and tokens: a gradient that begins off 16 bytes gives what an aligned one does."""
    N, V = 1003, 119
    ids = zipf(N, V, torch.int64, C)
    flat = torch.randn(N * C + 1, device="cuda").to(DT[dt])
    off = flat[1:].view(N, C)
    assert off.data_ptr() % 16
    dT = sga.embed_bwd(ids, off, V, 0.5)
    assert torch.equal(dT, sga.embed_bwd(ids, off.clone(), V, 0.5))
    v, b = embed_bwd_reference(ids, off, V, 0.5, None)
    within(dT, (v, b + 2 ** -24 * v.abs()), "dTable")
