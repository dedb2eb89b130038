"""The embedding gradient where tokens are sorted (more than 256 rows, or more
tokens than blocks can list): widths, offsets, frequent rows, padding, bad ids."""
import math

import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from dense_ref import embed_bwd_reference, within

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def gradient(N, C, dt, seed, off=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(N * C + 1, generator=g, device="cuda").to(DT[dt])
    return t[1:].view(N, C) if off else t[:-1].view(N, C)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 3, 4, 8, 31, 100, 128, 256, 260, 301, 512, 1024, 1500, 4096])
def test_widths(C, dt):
    N, V = 5000, 300
    ids = torch.randint(0, V, (N,), generator=torch.Generator(device="cuda").manual_seed(C), device="cuda")
    dO = gradient(N, C, dt, C)
    within(sga.embed_bwd(ids, dO, V, 0.5), embed_bwd_reference(ids, dO, V, 0.5), "dTable")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C", [31, 40, 301, 512, 1500, 4096])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "off"])
def test_rows_that_cross_many_chunks(C, dt, off):
    """Half of the tokens in one row, an eighth in each of two more, runs of any length in the rest."""
    N, V = 6000, 400
    g = torch.Generator(device="cuda").manual_seed(C)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand(N, generator=g, device="cuda")
    ids[u < 0.75] = 399
    ids[u < 0.625] = 17
    ids[u < 0.5] = 200
    dO = gradient(N, C, dt, C, off)
    assert off == (dO.data_ptr() % 16 != 0)
    dT = sga.embed_bwd(ids, dO, V, 2.0)
    within(dT, embed_bwd_reference(ids, dO, V, 2.0), "dTable")
    assert torch.equal(dT, sga.embed_bwd(ids, dO, V, 2.0))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C", [64, 33])
@pytest.mark.parametrize("padding", [0, 150, 299])
def test_padding_and_bad_ids(C, dt, padding):
    N, V = 3000, 300
    g = torch.Generator(device="cuda").manual_seed(padding)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda")
    ids[::7] = padding
    bad = torch.rand(N, generator=g, device="cuda") < 0.1
    ids[bad] = torch.tensor([-1, V, 2 ** 40, -2 ** 40], device="cuda")[torch.arange(int(bad.sum()), device="cuda") % 4]
    dO = gradient(N, C, dt, padding)
    dO[ids == padding] = math.nan   # (never read into a sum)
    dO[bad] = math.inf
    dT = sga.embed_bwd(ids, dO, V, 1.5, padding)
    assert sga.embed_device_error() == 1
    ref = embed_bwd_reference(ids, torch.where((ids == padding)[:, None] | bad[:, None], torch.zeros_like(dO), dO), V, 1.5, padding)
    within(dT, ref, "dTable")
    assert (dT[padding] == 0).all()


def test_few_rows_and_more_tokens_than_blocks_can_list():
    N, V, C = 200003, 119, 100
    ids = torch.randint(0, V, (N,), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    for dt in DT:
        dO = gradient(N, C, dt, 1)
        within(sga.embed_bwd(ids, dO, V), embed_bwd_reference(ids, dO, V, 1.0), "dTable")
