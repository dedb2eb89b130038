"""Calls of the layer norm at the edges of what its documentation allows."""
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [1e-50, 1e39])
def test_eps_that_float32_cannot_hold(eps):
    """1e-50 would be zero, and a constant row NaN instead of its bias."""
    with pytest.raises(ValueError, match="eps"):
        sga.layer_norm_fwd(torch.ones(3, 8, device="cuda"), eps=eps)


@pytest.mark.parametrize("eps", [1e-37, 1e-44])
def test_small_eps_of_a_constant_row(eps):
    out, mean, rstd = sga.layer_norm_fwd(torch.full((3, 8), 2.0, device="cuda"), eps=eps)
    assert (out == 0).all() and (mean == 2).all() and torch.isfinite(rstd).all()
    torch.testing.assert_close(rstd.double(), torch.full_like(rstd, float(torch.tensor(eps))).double() ** -0.5, rtol=2 ** -21, atol=0)
