"""Calls of the layer norm at the edges of what its documentation allows."""
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from dense_ref import norm_reference, within

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


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [1, 8])
def test_few_rows_of_the_largest_width(N, dt):
    """2^20 columns, at most 4 MB, are read three times in the forward, and x, dOut
    and the weight twice in the backward, and once more for the column sums.  One
    SM would take some 40 us for each; the plain forms, on all of them, take 112
    us and up forward, 206 and up backward.  Neither direction may take longer."""
    C = 1 << 20
    X, dO, w = torch.randn(N, C, device="cuda").to(dt), torch.randn(N, C, device="cuda").to(dt), torch.rand(C, device="cuda")
    out, mean, rstd = sga.layer_norm_fwd(X, w, w)
    for name, t in norm_reference(X, w, w, 1e-5).items():
        within({"out": out, "mean": mean, "rstd": rstd}[name], t, name)
    fwd = microseconds(lambda: sga.layer_norm_fwd(X, w, w, out=out, mean=mean, rstd=rstd))
    bwd = microseconds(lambda: sga.layer_norm_bwd(X, w, mean, rstd, dO))
    print(f"{N} {dt}: {fwd:.0f} us, {bwd:.0f} us")
    assert fwd <= 112 and bwd <= 206


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("C", [65537, 65544, 100000, 99999, 16385, 16392])
@pytest.mark.parametrize("N", [1, 3, 60])
def test_wide_rows(C, N, dt):
    """Widths past 16384 (1024 threads a row) and 65536 (eight blocks a row, more rows than clusters)."""
    g = torch.Generator(device="cuda").manual_seed(C)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    X, dO, w, b = (n(N, C) * 1.7 + 0.3).to(dt), n(N, C).to(dt), n(C) * 0.2 + 1, n(C) * 0.2
    ref = norm_reference(X, w, b, 1e-5, dO)
    out, mean, rstd = sga.layer_norm_fwd(X, w, b)
    dX, dw, db = sga.layer_norm_bwd(X, w, mean, rstd, dO)
    for name, t in {"out": out, "mean": mean, "rstd": rstd, "dX": dX, "dweight": dw, "dbias": db}.items():
        within(t, ref[name], name)
    again = sga.layer_norm_bwd(X, w, mean, rstd, dO)
    assert all(torch.equal(a, c) for a, c in zip(again, (dX, dw, db)))
    sga.layer_norm_fwd(X, w, b, out=X)
    assert torch.equal(X, out)
