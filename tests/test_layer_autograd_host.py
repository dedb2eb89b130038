"""What the autograd functions of the transformer-layer operators ask of the calls below them (CPU; the calls are replaced)."""
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga


@pytest.fixture
def saves(monkeypatch):
    """The `save` of each forward call of the gated product."""
    seen = []

    def fwd(X, Wg, Wu, act="silu", save=True):
        seen.append(save)
        G, U = X @ Wg, X @ Wu
        return torch.relu(G) * U, G if save else None, U if save else None

    def bwd(X, Wg, Wu, G, U, dOut, act="silu", input=True, weights=True):
        dG, dU = dOut * U * (G > 0), dOut * torch.relu(G)
        return dG @ Wg.T + dU @ Wu.T, X.T @ dG, X.T @ dU

    monkeypatch.setattr(sga, "gated_ff_fwd", fwd)
    monkeypatch.setattr(sga, "gated_ff_bwd", bwd)
    return seen


def test_gated_product_keeps_its_projections_for_a_gradient_alone(saves):
    X, Wg, Wu = torch.randn(5, 4), torch.randn(4, 3, requires_grad=True), torch.randn(4, 3, requires_grad=True)
    want = sga.GatedFF.apply(X, Wg, Wu, "relu")
    assert saves == [True] and want.requires_grad
    for off in (torch.no_grad(), torch.inference_mode()):   # a model's parameters ask for gradients there too
        with off:
            got = sga.GatedFF.apply(X, Wg, Wu, "relu")
        assert saves.pop() is False and torch.equal(got, want) and not got.requires_grad
    sga.GatedFF.apply(X, Wg.detach(), Wu.detach())
    assert saves.pop() is False
    with torch.no_grad(), torch.enable_grad():
        again = sga.GatedFF.apply(X.clone().requires_grad_(), Wg.detach(), Wu.detach(), "relu")
    assert saves == [True, True] and again.requires_grad
    want.sum().backward()
    assert torch.allclose(Wu.grad, X.T @ torch.relu(X @ Wg.detach()))
