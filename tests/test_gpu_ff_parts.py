"""fp32 results of the gated feed-forward product that are single products, elementwise to the accuracy of the operands'
three bf16 parts (8 + 8 + 8 bits): the bounds of long sums would not show a part that is missing or in the wrong place."""
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga

pytestmark = pytest.mark.gpu

# One product: of the nine products of parts the three left out are at most 2^-27, 2^-27 and 2^-36 of it; the smaller parts
# are summed first, so that one addition alone drops up to 2^-23 of the result, and the five before it as much of sums that
# are below 2^-7 of it; its rounding from the registers is none.
SINGLE = 2.0 ** -22


def single(got, want):
    err = (got.double() - want).abs()
    assert (err <= SINGLE * want.abs()).all(), f"{float((err / want.abs()).nan_to_num(0).max()) * 2 ** 24:.3g} units of 2^-24"


def full(*s, g):
    """Random mantissas of 24 bits, both signs, over four octaves."""
    x = torch.rand(*s, generator=g, device="cuda") + 1
    return x * torch.where(torch.rand(*s, generator=g, device="cuda") < 0.5, -1.0, 1.0) * 2.0 ** torch.randint(-2, 2, s, generator=g, device="cuda")


@pytest.mark.parametrize("T,M", [(64, 128), (91, 45), (300, 301), (700, 256), (1100, 1100), (33, 2000)])
def test_forward(T, M):
    """X has one element a row."""
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.zeros(T, T, device="cuda")
    at = torch.randperm(T, generator=g, device="cuda")
    i = torch.arange(T, device="cuda")
    X[i, at] = full(T, g=g)
    Wg, Wu = full(T, M, g=g), full(T, M, g=g)
    _, G, U = sga.gated_ff_fwd(X, Wg, Wu, "relu")
    x = X[i, at].double()[:, None]
    single(G, x * Wg.double()[at])
    single(U, x * Wu.double()[at])
    assert sga.gated_ff_device_error() == 0


@pytest.mark.parametrize("n,F", [(64, 64), (91, 45), (300, 301), (700, 40), (1100, 513), (2000, 33)])
def test_backward(n, F):
    """dOut has one element a row and column; every other column of each weight is zero."""
    g = torch.Generator(device="cuda").manual_seed(2)
    X, Wg, Wu, G, U = full(n, F, g=g), full(F, n, g=g), full(F, n, g=g), full(n, n, g=g).abs(), full(n, n, g=g)
    i = torch.arange(n, device="cuda")
    at = torch.randperm(n, generator=g, device="cuda")
    dOut = torch.zeros(n, n, device="cuda")
    dOut[i, at] = full(n, g=g)
    Wg[:, ::2] = 0
    Wu[:, 1::2] = 0
    dX, dWg, dWu = sga.gated_ff_bwd(X, Wg, Wu, G, U, dOut, "relu")
    # (relu's slope is one: dG and dU are rounded once)
    dg, du = (dOut[i, at] * U[i, at]).double()[:, None], (dOut[i, at] * G[i, at]).double()[:, None]
    single(dX, dg * Wg.double().T[at] + du * Wu.double().T[at])
    single(dWg.T[at], dg * X.double())
    single(dWu.T[at], du * X.double())
    assert sga.gated_ff_device_error() == 0
