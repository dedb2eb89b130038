"""Layer norm against its definition in 64 bits."""
import math

import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from dense_ref import norm_reference, within

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", None), ("bf16", None)]


def make(N, C, dt, wt, seed=0, mean=0.3, std=1.7):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    X, dO = (n(N, C) * std + mean).to(DT[dt]), n(N, C).to(DT[dt])
    w, b = (None, None) if wt is None else ((n(C) * 0.2 + 1).to(DT[wt]), (n(C) * 0.2).to(DT[wt]))
    return X, w, b, dO


def check(N, C, dt, wt, eps=1e-5, **kw):
    X, w, b, dO = make(N, C, dt, wt, **kw)
    ref = norm_reference(X, w, b, eps, dO)
    out, mean, rstd = sga.layer_norm_fwd(X, w, b, eps)
    dX, dw, db = sga.layer_norm_bwd(X, w, mean, rstd, dO)
    torch.cuda.synchronize()
    got = {"out": out, "mean": mean, "rstd": rstd, "dX": dX, "dweight": dw, "dbias": db}
    for name, t in got.items():
        if wt is None and name in ("dweight", "dbias"):
            assert t is None
        else:
            within(t, ref[name], f"{name} {N}x{C} {dt} {wt}")
    return got


@pytest.mark.parametrize("dt,wt", TYPES)
@pytest.mark.parametrize("C", [1, 2, 3, 8, 31, 32, 64, 65, 100, 128, 129, 256, 301, 512, 513, 520, 1000, 1024, 1032, 2048,
                               4096, 4097, 4100, 8192, 8200, 20000])
def test_widths(C, dt, wt):
    check(37, C, dt, wt, seed=C)


@pytest.mark.parametrize("dt,wt", TYPES[:3])
@pytest.mark.parametrize("N", [1, 2, 5, 152, 2000, 30011])
def test_rows(N, dt, wt):
    check(N, 256, dt, wt, seed=N)
    check(N, 37, dt, wt, seed=N)


def test_far_mean_and_constant_rows():
    """A mean 100 times the spread: the variance is taken about the mean.  A
    constant row gives the bias."""
    check(64, 256, "f32", "f32", mean=100.0, std=1.0)
    X = torch.full((5, 64), 3.0, device="cuda")
    b = torch.randn(64, device="cuda")
    out, mean, rstd = sga.layer_norm_fwd(X, torch.ones(64, device="cuda"), b)
    assert torch.equal(out, b.expand(5, 64)) and (mean == 3).all()
    torch.testing.assert_close(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6, atol=0)


def test_shapes_offsets_and_in_place():
    X, w, b, dO = make(60, 64, "bf16", "f32")
    out, mean, rstd = sga.layer_norm_fwd(X, w, b)
    o3, m3, r3 = sga.layer_norm_fwd(X.view(3, 20, 64), w, b)
    assert o3.shape == (3, 20, 64) and m3.shape == (3, 20) and torch.equal(o3.view(60, 64), out) and torch.equal(m3.view(60), mean)
    o1, m1, _ = sga.layer_norm_fwd(X[7], w, b)
    assert torch.equal(o1, out[7]) and m1.shape == ()
    # rows off a 16-byte boundary take the elementwise path
    off = torch.empty(60 * 64 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(60, 64)
    off.copy_(X)
    within(sga.layer_norm_fwd(off, w, b)[0], norm_reference(X, w, b, 1e-5)["out"])
    within(sga.layer_norm_bwd(off, w, mean, rstd, dO)[1], norm_reference(X, w, b, 1e-5, dO)["dweight"])
    Y = X.clone()
    sga.layer_norm_fwd(Y, w, b, out=Y)
    assert torch.equal(Y, out)
    dX, dw, db = sga.layer_norm_bwd(X, w, mean, rstd, dO)
    d2, w2, b2 = sga.layer_norm_bwd(X, w, mean, rstd, dO, bias=False)
    assert torch.equal(d2, dX) and torch.equal(w2, dw) and b2 is None


def test_no_rows():
    X, w = torch.empty(0, 16, device="cuda"), torch.ones(16, device="cuda")
    out, mean, rstd = sga.layer_norm_fwd(X, w, w)
    dX, dw, db = sga.layer_norm_bwd(X, w, mean, rstd, X)
    assert out.shape == X.shape and dX.shape == X.shape and (dw == 0).all() and (db == 0).all()


def test_nan_stays_in_its_row():
    X, w, b, dO = make(40, 256, "bf16", "f32")
    ref = sga.layer_norm_fwd(X, w, b)[0]
    X[3, 5], X[9, 0] = math.nan, math.inf
    out = sga.layer_norm_fwd(X, w, b)[0]
    keep = [i for i in range(40) if i not in (3, 9)]
    assert torch.equal(out[keep], ref[keep]) and torch.isnan(out[3]).all() and torch.isnan(out[9]).any()


@pytest.mark.parametrize("affine", [True, False])
def test_autograd(affine):
    X, w, b, dO = make(300, 96, "bf16", "f32" if affine else None)
    out, mean, rstd = sga.layer_norm_fwd(X, w, b, 1e-3)
    ref = sga.layer_norm_bwd(X, w, mean, rstd, dO)
    x = [None if t is None else t.clone().requires_grad_() for t in (X, w, b)]
    o = sga.LayerNorm.apply(*x, 1e-3)
    o.backward(dO)
    assert torch.equal(o, out)
    for t, r in zip(x, ref):
        assert (t is None and r is None) or torch.equal(t.grad, r)
    y = X.clone().requires_grad_()
    sga.LayerNorm.apply(y, w, None, 1e-3).sum().backward()
    assert torch.equal(y.grad, sga.layer_norm_bwd(X, w, mean, rstd, torch.ones_like(X))[0])


def test_gradients_against_differences():
    X, w, b, G = make(20, 33, "f32", "f32")
    x = [t.clone().requires_grad_() for t in (X, w, b)]
    sga.LayerNorm.apply(*x).backward(G)
    h = 1e-2
    for i, t in enumerate((X, w, b)):
        d = torch.randn_like(t)
        f = lambda s: (sga.layer_norm_fwd(*[u + s * h * d if j == i else u for j, u in enumerate((X, w, b))])[0].double()
                       * G.double()).sum()
        num, ana = float((f(1) - f(-1)) / (2 * h)), float((x[i].grad.double() * d.double()).sum())
        assert abs(num - ana) <= 1e-3 * float(x[i].grad.norm() * d.norm()), (i, num, ana)


def test_reproducible_streams_and_graphs():
    X, w, b, dO = make(5000, 512, "bf16", "f32")
    out, mean, rstd = sga.layer_norm_fwd(X, w, b)
    ref = (out, mean, rstd, *sga.layer_norm_bwd(X, w, mean, rstd, dO))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    for s in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            f = sga.layer_norm_fwd(X, w, b)
            r = (*f, *sga.layer_norm_bwd(X, w, f[1], f[2], dO))
        graphs.append((s, g, r))
    for s, g, _ in graphs:
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    for _, _, r in graphs:
        for a, c in zip(r, ref):
            assert torch.equal(a, c)
    s = streams[0]
    got = sga.layer_norm_bwd(X, w, mean, rstd, dO, stream=s)
    s.synchronize()
    for a, c in zip(got, ref[3:]):
        assert torch.equal(a, c)


def test_refusals():
    X, w, b, dO = make(10, 64, "bf16", "f32")
    with pytest.raises(ValueError):
        sga.layer_norm_fwd(X, w[:-1], b)
    with pytest.raises(ValueError):
        sga.layer_norm_fwd(X, None, b)
    with pytest.raises(TypeError):
        sga.layer_norm_fwd(X, w, b.bfloat16())
    with pytest.raises(TypeError):
        sga.layer_norm_fwd(X.float(), w.bfloat16(), b.bfloat16())
    with pytest.raises(TypeError):
        sga.layer_norm_fwd(X.half())
    with pytest.raises(ValueError):
        sga.layer_norm_fwd(X.t())
    for eps in (-1e-5, math.nan, math.inf):
        with pytest.raises(ValueError):
            sga.layer_norm_fwd(X, w, b, eps)
    out, mean, rstd = sga.layer_norm_fwd(X, w, b)
    with pytest.raises(ValueError):
        sga.layer_norm_bwd(X, w, mean[:-1], rstd, dO)
    with pytest.raises(ValueError, match="shares memory"):
        sga.layer_norm_bwd(X, w, mean, rstd, dO, dX=dO)
    with pytest.raises(ValueError):
        sga.layer_norm_bwd(X, None, mean, rstd, dO, dbias=b)
