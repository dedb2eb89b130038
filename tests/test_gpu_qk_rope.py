"""Norm and rotary positions of query and key heads against the 64-bit definition, elementwise bounds."""
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from layer_ref import rope_bwd_reference, rope_reference, within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def inputs(T, H, Hk, D, dt, seed=1, fused=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    if fused:
        x = n(T, H + 2 * Hk, D).to(dt)
        Q, K = x[:, :H], x[:, H:H + Hk]
    else:
        Q, K = n(T, H, D).to(dt), n(T, Hk, D).to(dt)
    return Q, K, n(D) * 0.3 + 1, n(D) * 0.3 + 1, n(T, H, D).to(dt), n(T, Hk, D).to(dt), g


def check(rot, T, H, Hk, D, dt, wdt=None, axes=1, pos=None, eps=1e-6, fused=False, seed=1):
    Q, K, wq, wk, dq, dk, g = inputs(T, H, Hk, D, dt, seed, fused)
    wq, wk = (wq.to(wdt), wk.to(wdt)) if wdt is not None else (None, None)
    if pos is None:
        pos = torch.randint(-50, 200000, (T, axes) if axes > 1 else (T,), generator=g, device="cuda")
    q, k, rq, rk = sga.qk_norm_rope_fwd(rot, Q, K, pos, wq, wk, eps)
    back = sga.qk_norm_rope_bwd(rot, Q, K, pos, wq, wk, rq, rk, dq, dk)
    assert all(a is None or torch.equal(a, b) for a, b in zip(back, sga.qk_norm_rope_bwd(rot, Q, K, pos, wq, wk, rq, rk, dq, dk)))
    for side, x, w, out, r, dout, dx, dw in (("q", Q, wq, q, rq, dq, back[0], back[2]), ("k", K, wk, k, rk, dk, back[1], back[3])):
        ref = rope_reference(rot, x, pos, w, eps)
        within(out, ref["out"], side)
        if eps is None:
            assert r is None
        else:
            within(r, ref["r"], side + " r")
        gr = rope_bwd_reference(rot, x, pos, w, r, dout)
        within(dx, gr["dx"], side + " dx")
        if w is None:
            assert dw is None
        else:
            within(dw, gr["dw"], side + " dw")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_widths_and_types(D, dt, wdt, interleaved):
    rot = sga.Rotary(D, interleaved=interleaved)
    for T, H, Hk in ((1, 1, 1), (37, 4, 2), (1000, 3, 1), (5003, 8, 8)):
        check(rot, T, H, Hk, D, dt, wdt)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D,dims", [(32, 16), (64, 48), (128, 16), (128, 112), (64, 0)])
def test_part_of_a_head_turned(D, dims, dt, interleaved):
    check(sga.Rotary(D, dims, base=500.0, interleaved=interleaved), 301, 5, 2, D, dt, dt)


@pytest.mark.parametrize("sections", [[16], [10, 22], [8, 12, 12], [0, 32], [8, 0, 8, 16]])
def test_several_axes(sections):
    n = sum(sections)
    for D in (32, 64, 128):
        if 2 * n <= D:
            for inter in (False, True):
                check(sga.Rotary(D, 2 * n, sections=sections, interleaved=inter), 257, 4, 2, D, BF, F32, axes=len(sections))


@pytest.mark.parametrize("dt", [BF, F32])
def test_rotation_alone_and_norm_alone(dt):
    check(sga.Rotary(64), 77, 4, 1, 64, dt, eps=None)                # no norm, no weights
    check(sga.Rotary(64), 77, 4, 1, 64, dt)                          # norm without weights
    check(sga.Rotary(128, 0), 77, 4, 1, 128, dt, F32, eps=1e-3)      # nothing turned
    check(sga.Rotary(32), 77, 2, 2, 32, dt, dt, eps=0.0)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_far_and_negative_positions(dtype):
    """fp32 angles would be off by radians at 2^30."""
    T = 64
    pos = torch.tensor([0, 1, -1, 2 ** 30, -2 ** 30, 2 ** 31 - 1, -2 ** 31, 999_999_937] * 8, dtype=dtype, device="cuda")
    for inter in (False, True):
        check(sga.Rotary(64, interleaved=inter), T, 2, 1, 64, F32, F32, pos=pos)
    if dtype == torch.int64:
        check(sga.Rotary(64), T, 2, 1, 64, F32, F32, pos=pos * 1000)


def test_frequencies_given():
    freqs = [-1.0, 3.5, 7.0, 0.0, 2.0 ** -20, 100.25, -1e-9, 6.283185307179586]
    check(sga.Rotary(32, 16, freqs=freqs), 90, 2, 1, 32, F32, F32)
    # whole turns a position turn nothing
    rot = sga.Rotary(32, 16, freqs=[2 * 3.141592653589793] * 8)
    Q, K, *_ = inputs(9, 1, 1, 32, F32)
    q, k, _, _ = sga.qk_norm_rope_fwd(rot, Q, K, torch.arange(9, device="cuda"), eps=None)
    assert torch.equal(q, Q) and torch.equal(k, K)


@pytest.mark.parametrize("dt", [BF, F32])
def test_slices_of_one_projection_equal_dense_ones(dt):
    check(sga.Rotary(64), 333, 6, 2, 64, dt, dt, fused=True)
    Q, K, wq, wk, dq, dk, _ = inputs(333, 6, 2, 64, dt, fused=True)
    rot, pos = sga.Rotary(64), torch.arange(333, device="cuda")
    a = sga.qk_norm_rope_fwd(rot, Q, K, pos, wq, wk)
    b = sga.qk_norm_rope_fwd(rot, Q.contiguous(), K.contiguous(), pos, wq, wk)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    c = sga.qk_norm_rope_bwd(rot, Q, K, pos, wq, wk, a[2], a[3], dq, dk)
    d = sga.qk_norm_rope_bwd(rot, Q.contiguous(), K.contiguous(), pos, wq, wk, a[2], a[3], dq, dk)
    assert all(torch.equal(x, y) for x, y in zip(c, d))
    one = Q[5:6], K[5:6]                     # one row of a slice
    e = sga.qk_norm_rope_fwd(rot, *one, pos[5:6], wq, wk)
    assert torch.equal(e[0], a[0][5:6]) and torch.equal(e[1], a[1][5:6])


def test_in_place():
    for dt in (BF, F32):
        Q, K, wq, wk, dq, dk, _ = inputs(1001, 4, 2, 64, dt)
        rot, pos = sga.Rotary(64, interleaved=True), torch.arange(1001, device="cuda", dtype=torch.int32)
        q, k, rq, rk = sga.qk_norm_rope_fwd(rot, Q, K, pos, wq, wk)
        gq, gk, wgq, wgk = sga.qk_norm_rope_bwd(rot, Q, K, pos, wq, wk, rq, rk, dq, dk)
        sga.qk_norm_rope_bwd(rot, Q, K, pos, wq, wk, rq, rk, dq, dk, dQ=dq, dK=dk)
        assert torch.equal(dq, gq) and torch.equal(dk, gk)
        sga.qk_norm_rope_fwd(rot, Q, K, pos, wq, wk, out_q=Q, out_k=K)
        assert torch.equal(Q, q) and torch.equal(K, k)


def test_many_heads_and_no_rows():
    check(sga.Rotary(32), 3, 600, 400, 32, BF, BF)
    check(sga.Rotary(128), 400, 1, 1, 128, F32, F32)
    rot = sga.Rotary(64)
    e = torch.empty(0, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    pos = torch.empty(0, dtype=torch.int64, device="cuda")
    q, k, rq, rk = sga.qk_norm_rope_fwd(rot, e, e, pos, w, w)
    assert q.shape == e.shape and rq.shape == (0, 2)
    out = sga.qk_norm_rope_bwd(rot, e, e, pos, w, w, rq, rk, e, e)
    assert (out[2] == 0).all() and (out[3] == 0).all()


def test_a_row_that_is_not_finite_stays_alone():
    rot = sga.Rotary(64, 32)
    Q, K, wq, wk, dq, dk, _ = inputs(40, 2, 2, 64, F32)
    pos = torch.arange(40, device="cuda")
    a = sga.qk_norm_rope_fwd(rot, Q, K, pos, wq, wk)
    Q2 = Q.clone()
    Q2[7, 1, 50] = torch.inf
    b = sga.qk_norm_rope_fwd(rot, Q2, K, pos, wq, wk)
    keep = torch.ones(40, 2, dtype=torch.bool, device="cuda")
    keep[7, 1] = False
    assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1], b[1])
    # without a norm an element that is not turned reaches nothing else
    c = sga.qk_norm_rope_fwd(rot, Q, K, pos, eps=None)[0]
    d = sga.qk_norm_rope_fwd(rot, Q2, K, pos, eps=None)[0]
    same = c == d
    assert same.sum() == same.numel() - 1 and torch.isinf(d[7, 1, 50])


def test_gradients_against_differences():
    """Of the mean of a function of both results, along random directions, in fp32: central differences of a step of 2^-6
    are off by their curvature (about 2^-12 of the slope) and by the roundings of the two sums over the step (2^-24 x 2^6 x
    the sum's size)."""
    rot = sga.Rotary(32, sections=[6, 10])
    Q, K, wq, wk, dq, dk, g = inputs(20, 3, 2, 32, F32)
    pos = torch.randint(0, 5000, (20, 2), generator=g, device="cuda")

    def f(Q, K, wq, wk):
        q, k, _, _ = sga.qk_norm_rope_fwd(rot, Q, K, pos, wq, wk)
        return float((q.double() * dq.double()).sum() + (k.double() * dk.double()).sum())

    _, _, rq, rk = sga.qk_norm_rope_fwd(rot, Q, K, pos, wq, wk)
    grads = sga.qk_norm_rope_bwd(rot, Q, K, pos, wq, wk, rq, rk, dq, dk)
    xs = (Q, K, wq, wk)
    for i, (x, d) in enumerate(zip(xs, grads)):
        v = torch.randn(x.shape, generator=g, device="cuda")
        v /= v.norm()
        up, down = (f(*(y + s * 2.0 ** -6 * v if j == i else y for j, y in enumerate(xs))) for s in (1, -1))
        slope, scale = (up - down) * 2.0 ** 5, float(d.double().norm())
        assert abs(slope - float((d.double() * v.double()).sum())) < 2e-3 * scale


def test_autograd_and_streams():
    rot = sga.Rotary(64)
    x = torch.randn(50, 8, 64, device="cuda").bfloat16().requires_grad_()
    wq, wk = (torch.rand(64, device="cuda").requires_grad_() for _ in range(2))
    pos = torch.arange(50, device="cuda")
    q, k = sga.QKNormRope.apply(x[:, :4], x[:, 4:6], pos, wq, wk, rot, 1e-6)
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    torch.autograd.backward((q, k), (dq, dk))
    xd = x.detach()
    r = sga.qk_norm_rope_fwd(rot, xd[:, :4], xd[:, 4:6], pos, wq.detach(), wk.detach())
    b = sga.qk_norm_rope_bwd(rot, xd[:, :4], xd[:, 4:6], pos, wq.detach(), wk.detach(), r[2], r[3], dq, dk)
    assert torch.equal(q, r[0]) and torch.equal(k, r[1])
    assert torch.equal(x.grad[:, :4], b[0]) and torch.equal(x.grad[:, 4:6], b[1]) and (x.grad[:, 6:] == 0).all()
    assert torch.equal(wq.grad, b[2]) and torch.equal(wk.grad, b[3])
    # heads that are not dense within a row are copied by the autograd function
    y = torch.randn(50, 64, 4, device="cuda").transpose(1, 2)
    q2, k2 = sga.QKNormRope.apply(y, y, pos, None, None, rot, None)
    assert torch.equal(q2, sga.qk_norm_rope_fwd(rot, y.contiguous(), y.contiguous(), pos, eps=None)[0]) and torch.equal(q2, k2)
    # tensors, and gradients, that do not begin on 16 bytes too
    z = torch.randn(2 * 50 * 4 * 64 + 1, device="cuda")
    a, g = z[1:1 + 50 * 256].view(50, 4, 64), z[1 + 50 * 256:].view(50, 4, 64)
    a.requires_grad_()
    q3, k3 = sga.QKNormRope.apply(a, a.detach(), pos, None, None, rot, 1e-6)
    (ga,) = torch.autograd.grad(q3, a, g)
    d = a.detach().clone()
    r3 = sga.qk_norm_rope_fwd(rot, d, d, pos)
    assert torch.equal(q3, r3[0]) and torch.equal(ga, sga.qk_norm_rope_bwd(rot, d, d, pos, None, None, r3[2], r3[3], g.clone(), torch.zeros_like(d))[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r2 = sga.qk_norm_rope_fwd(rot, xd[:, :4], xd[:, 4:6], pos, wq.detach(), wk.detach(), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(r2[0], r[0])


def test_captured():
    rot = sga.Rotary(128)
    Q, K, wq, wk, dq, dk, _ = inputs(300, 4, 2, 128, BF)
    pos = torch.arange(300, device="cuda")
    call = lambda: (lambda f: f[:2] + sga.qk_norm_rope_bwd(rot, Q, K, pos, wq, wk, f[2], f[3], dq, dk))(
        sga.qk_norm_rope_fwd(rot, Q, K, pos, wq, wk))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for seed in (2, 3):
        new = inputs(300, 4, 2, 128, BF, seed)
        for t, n in zip((Q, K, wq, wk, dq, dk), new):
            t.copy_(n)
        pos += seed * 1000
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, call()))


def test_refusals():
    rot = sga.Rotary(64)
    Q, K, wq, wk, dq, dk, _ = inputs(8, 2, 1, 64, F32)
    pos = torch.arange(8, device="cuda")
    f = sga.qk_norm_rope_fwd
    with pytest.raises(ValueError, match="K must be"):
        f(rot, Q, K[:7], pos)
    with pytest.raises(TypeError, match="K must be"):
        f(rot, Q, K.bfloat16(), pos)
    with pytest.raises(TypeError, match="pos"):
        f(rot, Q, K, pos.float())
    with pytest.raises(ValueError, match="pos"):
        f(rot, Q, K, pos[:7])
    with pytest.raises(ValueError, match="pos"):
        f(sga.Rotary(64, sections=[16, 16]), Q, K, pos)
    with pytest.raises(ValueError, match="both weights"):
        f(rot, Q, K, pos, wq)
    with pytest.raises(ValueError, match="weights need a norm"):
        f(rot, Q, K, pos, wq, wk, None)
    with pytest.raises(TypeError, match="weights"):
        f(rot, Q, K, pos, wq.bfloat16(), wk.bfloat16())
    with pytest.raises(ValueError, match="eps"):
        f(rot, Q, K, pos, wq, wk, -1.0)
    with pytest.raises(ValueError, match="eps"):
        f(rot, Q, K, pos, wq, wk, 1e-60)
    with pytest.raises(ValueError, match="heads must be dense"):
        f(rot, torch.randn(8, 64, 2, device="cuda").transpose(1, 2), K, pos)
    with pytest.raises(ValueError, match="heads must be dense"):
        f(rot, torch.randn(8 * 130 + 1, device="cuda")[1:1 + 8 * 128].view(8, 2, 64), K, pos)   # off 16 bytes
    with pytest.raises(ValueError, match="heads must be dense"):
        f(rot, torch.randn(8, 130, device="cuda").as_strided((8, 2, 64), (130, 64, 1)), K, pos)   # rows 520 bytes apart
    with pytest.raises(ValueError, match="must be"):
        f(sga.Rotary(32), Q, K, pos)
    with pytest.raises(ValueError, match="shares memory"):
        f(rot, Q, K, pos, out_q=Q, out_k=Q[:, :1].reshape(-1)[:0].new_empty(0).set_(Q.untyped_storage(), 0, (8, 1, 64)))
    buf = torch.randn(8, 6, 64, device="cuda")   # results among the rows of the slices that they are formed from
    with pytest.raises(ValueError, match="out_q shares memory with Q"):
        f(rot, buf[:, :2], buf[:, 2:3], pos, out_q=buf.view(-1)[-8 * 2 * 64:].view(8, 2, 64))
    _, _, rq, rk = f(rot, Q, K, pos, wq, wk)
    b = sga.qk_norm_rope_bwd
    with pytest.raises(ValueError, match="both rq and rk"):
        b(rot, Q, K, pos, wq, wk, rq, None, dq, dk)
    with pytest.raises(ValueError, match="weights need a norm"):
        b(rot, Q, K, pos, wq, wk, None, None, dq, dk)
    with pytest.raises(ValueError, match="dwq and dwk need"):
        b(rot, Q, K, pos, None, None, rq, rk, dq, dk, dwq=wq)
    with pytest.raises(ValueError, match="contiguous"):
        b(rot, Q, K, pos, wq, wk, rq, rk, torch.randn(8, 64, 2, device="cuda").transpose(1, 2), dk)
