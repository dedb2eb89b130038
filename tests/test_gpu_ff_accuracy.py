"""fp32 products of the gated feed-forward block, normwise to fp32's accuracy, of random and of equal signs.

Units of U = 2^-24 of the result's norm.  A run of 64 products is summed by the tensor cores: its four additions of the
leading parts' products drop at most 2 U each of what is summed, one-sided; the smaller parts' twenty, of sums 2^-8 as
large, 0.2 together; the products of parts that are left out 0.25; operands of the backward are rounded once, 0.6.  The
runs are added in fp32, rounded to nearest: of R runs, sqrt(R / 3) at random."""
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga

pytestmark = pytest.mark.gpu


def near(got, want, depth, what):
    units = float((got.double() - want).norm() / want.norm()) * 2 ** 24
    assert units <= 10 + (depth / 64 / 3) ** 0.5, (what, units)


@pytest.mark.parametrize("signs", ["random", "equal"])
@pytest.mark.parametrize("T,F,M", [(300, 64, 200), (512, 256, 512), (700, 1024, 300), (512, 4096, 256), (5000, 100, 2048), (2100, 301, 803)])
def test_norm_of_the_error(T, F, M, signs):
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda") if signs == "random" else torch.rand(*s, generator=g, device="cuda") + 0.5
    X, Wg, Wu, dOut, G, U = n(T, F), n(F, M), n(F, M), n(T, M), n(T, M), n(T, M)
    _, g_, u_ = sga.gated_ff_fwd(X, Wg, Wu, "relu")
    x, wg, wu = X.double(), Wg.double(), Wu.double()
    near(g_, x @ wg, F, "G")
    near(u_, x @ wu, F, "U")
    dX, dWg, dWu = sga.gated_ff_bwd(X, Wg, Wu, G, U, dOut, "relu")
    d = dOut.double()
    dg, du = d * U.double() * (G > 0), d * G.double().clamp(min=0)
    near(dX, dg @ wg.T + du @ wu.T, 2 * M, "dX")
    near(dWg, x.T @ dg, T, "dWg")
    near(dWu, x.T @ du, T, "dWu")
    assert sga.gated_ff_device_error() == 0
