"""The gated feed-forward product against its 64-bit definition, elementwise bounds."""
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from layer_ref import ff_bwd_reference, ff_reference, within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def inputs(T, F, M, dt, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return n(T, F).to(dt), (n(F, M) * F ** -0.5).to(dt), (n(F, M) * F ** -0.5).to(dt), n(T, M).to(dt)


def check(T, F, M, dt, act="silu", seed=1):
    X, Wg, Wu, dO = inputs(T, F, M, dt, seed)
    out, G, U = sga.gated_ff_fwd(X, Wg, Wu, act)
    assert sga.gated_ff_device_error() == 0
    for name, t in ff_reference(X, Wg, Wu, act).items():
        within({"out": out, "G": G, "U": U}[name], t, f"{name} {T} {F} {M}")
    bare = sga.gated_ff_fwd(X, Wg, Wu, act, save=False)
    assert torch.equal(bare[0], out) and bare[1] is None and bare[2] is None
    grads = sga.gated_ff_bwd(X, Wg, Wu, G, U, dO, act)
    assert sga.gated_ff_device_error() == 0
    for name, t in ff_bwd_reference(X, Wg, Wu, G, U, dO, act).items():
        within(grads[("dX", "dWg", "dWu").index(name)], t, f"{name} {T} {F} {M}")
    again = sga.gated_ff_bwd(X, Wg, Wu, G, U, dO, act)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    half = sga.gated_ff_bwd(X, Wg, Wu, G, U, dO, act, weights=False), sga.gated_ff_bwd(X, Wg, Wu, G, U, dO, act, input=False)
    assert torch.equal(half[0][0], grads[0]) and half[0][1] is None and half[1][0] is None
    assert torch.equal(half[1][1], grads[1]) and torch.equal(half[1][2], grads[2])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,F,M", [(256, 64, 128), (1, 8, 8), (1, 1, 1), (300, 72, 200), (128, 256, 136), (513, 520, 264), (37, 100, 301),
                                   (1000, 33, 65), (2, 511, 3), (255, 7, 129), (257, 128, 1024)])
def test_sizes(T, F, M, dt):
    check(T, F, M, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("F", [5, 32, 40, 65, 96, 129, 160, 192, 200, 257, 301, 320, 384, 392, 513, 577, 1025])
def test_widths_of_tiles(F, dt):
    """dX's tiles are as wide as its columns' even shares: from one block to 256 columns."""
    check(300, F, 72, dt, "relu")
    check(1100, F, 800, dt)


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("dt", [BF, F32])
def test_activations(dt, act):
    check(700, 128, 192, dt, act)
    check(70, 45, 91, dt, act)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,F,M", [(64, 4096, 640), (5000, 256, 256), (2900, 300, 900), (30000, 64, 72), (1, 2048, 5000), (9000, 1024, 40)])
def test_shared_depth_and_rounds(T, F, M, dt):
    """Few tiles of great depth (shared by many pairs), and several rounds of tiles."""
    check(T, F, M, dt, "gelu")


def test_long_sums_in_runs():
    """A depth of more than 16384, over which the tensor cores' sums are taken apart."""
    check(70001, 64, 64, BF)
    check(33000, 320, 24, BF)


@pytest.mark.parametrize("dt", [BF, F32])
def test_leading_dimensions_and_no_rows(dt):
    X, Wg, Wu, dO = inputs(60, 48, 40, dt)
    a = sga.gated_ff_fwd(X, Wg, Wu)
    b = sga.gated_ff_fwd(X.view(3, 4, 5, 48), Wg, Wu)
    assert b[0].shape == (3, 4, 5, 40) and all(torch.equal(x, y.view(60, 40)) for x, y in zip(a, b))
    c = sga.gated_ff_bwd(X.view(12, 5, 48), Wg, Wu, *(t.view(12, 5, 40) for t in a[1:]), dO.view(12, 5, 40))
    d = sga.gated_ff_bwd(X, Wg, Wu, *a[1:], dO)
    assert c[0].shape == (12, 5, 48) and torch.equal(c[0].view(60, 48), d[0]) and torch.equal(c[1], d[1])
    one = sga.gated_ff_fwd(X[7], Wg, Wu)
    assert one[0].shape == (40,)
    e = torch.empty(0, 48, device="cuda", dtype=dt)
    out, G, U = sga.gated_ff_fwd(e, Wg, Wu)
    assert out.shape == (0, 40)
    dX, dWg, dWu = sga.gated_ff_bwd(e, Wg, Wu, G, U, out)
    assert dX.shape == (0, 48) and (dWg == 0).all() and (dWu == 0).all()


def test_fp32_of_any_size_and_sign():
    """Values across fp32's range, where bf16 parts round away, overflow or fall below its smallest."""
    X = torch.zeros(40, 64, device="cuda")
    Wg, Wu = torch.zeros(64, 64, device="cuda"), torch.zeros(64, 64, device="cuda")
    i = torch.arange(40, device="cuda")
    big = torch.tensor(3.4e38, device="cuda")     # rounds to infinity in bf16
    X[i, i] = 1.0
    X[3, 3], Wg[3, 3], Wu[3, 3] = big, 2.0 ** -100, 2.0 ** -100
    X[4, 4], Wg[4, 4], Wu[4, 4] = 2.0 ** -100 * (1 + 2.0 ** -23), 2.0 ** 100, 2.0 ** 100
    X[5, 5], Wg[5, 5], Wu[5, 5] = 1 / 3, -1 / 7, 1 + 2.0 ** -23
    out, G, U = sga.gated_ff_fwd(X, Wg, Wu, "relu")
    x, g = X.double(), X.double() @ Wg.double()
    u = x @ Wu.double()
    assert ((G.double() - g).abs() <= 2.0 ** -22 * g.abs()).all() and ((U.double() - u).abs() <= 2.0 ** -22 * u.abs()).all()
    assert ((out.double() - torch.relu(g) * u).abs() <= 2.0 ** -21 * (torch.relu(g) * u).abs()).all()


@pytest.mark.parametrize("dt", [BF, F32])
def test_rows_that_are_not_finite_stay_alone(dt):
    X, Wg, Wu, dO = inputs(400, 100, 136, dt)
    a = sga.gated_ff_fwd(X, Wg, Wu)
    for v in (torch.nan, torch.inf):
        Y = X.clone()
        Y[133, 99] = v
        b = sga.gated_ff_fwd(Y, Wg, Wu)
        keep = torch.arange(400, device="cuda") != 133
        assert all(torch.equal(p[keep], q[keep]) for p, q in zip(a, b)) and not torch.isfinite(b[1][133]).any()
        E = dO.clone()
        E[133] = v
        c, d = sga.gated_ff_bwd(X, Wg, Wu, *a[1:], dO), sga.gated_ff_bwd(X, Wg, Wu, *a[1:], E)
        assert torch.equal(c[0][keep], d[0][keep]) and not torch.isfinite(d[0][133]).any()


def test_gradients_against_differences():
    X, Wg, Wu, dO = inputs(30, 24, 40, F32)
    f = lambda x, g, u: float((sga.gated_ff_fwd(x, g, u, "gelu")[0].double() * dO.double()).sum())
    _, G, U = sga.gated_ff_fwd(X, Wg, Wu, "gelu")
    grads = sga.gated_ff_bwd(X, Wg, Wu, G, U, dO, "gelu")
    r = torch.Generator(device="cuda").manual_seed(3)
    xs = (X, Wg, Wu)
    for i, d in enumerate(grads):
        v = torch.randn(xs[i].shape, generator=r, device="cuda")
        v /= v.norm()
        up, down = (f(*(x + s * 2.0 ** -6 * v if j == i else x for j, x in enumerate(xs))) for s in (1, -1))
        # (a step of 2^-6: its curvature is 2^-12 of the slope's size, the sums' roundings over it 2^-24 2^6)
        assert abs((up - down) * 2.0 ** 5 - float((d.double() * v.double()).sum())) < 2e-3 * float(d.double().norm())


@pytest.mark.parametrize("dt", [BF, F32])
def test_captured_overlapping_and_on_streams(dt):
    X, Wg, Wu, dO = inputs(1100, 320, 400, dt)

    def call():
        out, G, U = sga.gated_ff_fwd(X, Wg, Wu)
        return (out, G, U, *sga.gated_ff_bwd(X, Wg, Wu, G, U, dO))

    want = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    s = torch.cuda.Stream()
    for seed in (1, 5, 6):
        for t, n in zip((X, Wg, Wu, dO), inputs(1100, 320, 400, dt, seed)):
            t.copy_(n)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = call()
        graph.replay()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        want = call()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip(other, want))
    t = sga.gated_ff_fwd(X, Wg, Wu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(t[0], want[0]) and sga.gated_ff_device_error() == 0


@pytest.mark.parametrize("dt", [BF, F32])
def test_autograd(dt):
    X, Wg, Wu, dO = inputs(90, 40, 56, dt)
    leaves = [t.clone().requires_grad_() for t in (X, Wg, Wu)]
    out = sga.GatedFF.apply(*leaves, "gelu")
    out.backward(dO)
    o, G, U = sga.gated_ff_fwd(X, Wg, Wu, "gelu")
    grads = sga.gated_ff_bwd(X, Wg, Wu, G, U, dO, "gelu")
    assert torch.equal(out, o) and all(torch.equal(a.grad, b) for a, b in zip(leaves, grads))
    x = X.clone().requires_grad_()
    sga.GatedFF.apply(x, Wg, Wu, "gelu").backward(dO)
    assert torch.equal(x.grad, grads[0])
    w = Wu.clone().requires_grad_()
    sga.GatedFF.apply(X, Wg, w, "gelu").backward(dO)
    assert torch.equal(w.grad, grads[2])
    # transposed weights, and rows that do not begin on 16 bytes, are copied by the autograd function
    odd = torch.empty(90 * 40 + 1, device="cuda", dtype=dt)[1:].view(90, 40).copy_(X)
    got = sga.GatedFF.apply(odd, Wg.t().contiguous().t(), Wu, "gelu")
    assert torch.equal(got, o)


def test_refusals():
    X, Wg, Wu, dO = inputs(8, 16, 24, BF)
    with pytest.raises(ValueError, match="act"):
        sga.gated_ff_fwd(X, Wg, Wu, "tanh")
    with pytest.raises(ValueError, match="Wg must be"):
        sga.gated_ff_fwd(X, Wg[:15], Wu)
    with pytest.raises(ValueError, match="Wu must be"):
        sga.gated_ff_fwd(X, Wg, Wu[:, :8].contiguous())
    with pytest.raises(TypeError, match="Wu must be"):
        sga.gated_ff_fwd(X, Wg, Wu.float())
    with pytest.raises(TypeError, match="dtype"):
        sga.gated_ff_fwd(X.half(), Wg.half(), Wu.half())
    with pytest.raises(ValueError, match="contiguous"):
        sga.gated_ff_fwd(X.t().contiguous().t(), Wg, Wu)
    with pytest.raises(ValueError, match="16-byte"):
        sga.gated_ff_fwd(torch.empty(129, device="cuda", dtype=BF)[1:].view(8, 16), Wg, Wu)
    with pytest.raises(ValueError, match="save=False"):
        sga.gated_ff_fwd(X, Wg, Wu, save=False, G=dO)
    out, G, U = sga.gated_ff_fwd(X, Wg, Wu)
    with pytest.raises(ValueError, match="shares memory"):
        sga.gated_ff_fwd(X, Wg, Wu, G=G, U=G)
    with pytest.raises(ValueError, match="G must be"):
        sga.gated_ff_bwd(X, Wg, Wu, G[:7], U, dO)
    with pytest.raises(ValueError, match="input=False"):
        sga.gated_ff_bwd(X, Wg, Wu, G, U, dO, input=False, dX=X)
    with pytest.raises(ValueError, match="shares memory"):
        sga.gated_ff_bwd(X, Wg, Wu, G, U, dO, dX=X)
