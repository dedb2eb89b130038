"""The transformer-layer operators on arrays of more than 2^31 elements: the last rows are what the same call gives on
them alone."""
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from layer_ref import ff_bwd_reference, within
from test_gpu_dense_large import filled

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    yield
    torch.cuda.empty_cache()


def test_query_and_key_heads():
    T, H, HK, D = 140000, 124, 4, 128   # 2^31.05 elements of Q
    rot, pos = sga.Rotary(D), torch.arange(T, device="cuda")
    qkv, dq, dk = filled(T, H + 2 * HK, D), filled(T, H, D, seed=1), filled(T, HK, D, seed=2)
    Q, K = qkv[:, :H], qkv[:, H:H + HK]
    assert Q.numel() > 1 << 31
    w = torch.rand(D, device="cuda") + 0.5
    q, k, rq, rk = sga.qk_norm_rope_fwd(rot, Q, K, pos, w, w)
    dQ, dK, dwq, dwk = sga.qk_norm_rope_bwd(rot, Q, K, pos, w, w, rq, rk, dq, dk)
    s = slice(T - 500, None)
    a = sga.qk_norm_rope_fwd(rot, Q[s], K[s], pos[s], w, w)
    b = sga.qk_norm_rope_bwd(rot, Q[s], K[s], pos[s], w, w, a[2], a[3], dq[s], dk[s])
    assert all(torch.equal(x[s], y) for x, y in zip((q, k, rq, rk), a)) and torch.equal(dQ[s], b[0]) and torch.equal(dK[s], b[1])
    # dw of gradients that are zero but in the last rows
    dq[:T - 500] = 0
    dk[:T - 500] = 0
    c = sga.qk_norm_rope_bwd(rot, Q, K, pos, w, w, rq, rk, dq, dk)
    for x, y in ((c[2], b[2]), (c[3], b[3])):   # (the same terms in another order: 62,000 of them at most, about 1 each)
        assert ((x - y).abs() <= 2 * 62000 * 2.0 ** -24 * 500 * H).all() and (x - y).norm() <= 1e-4 * y.norm()


def test_windowed_attention():
    n, T, H, D = 100000, 1 << 20, 17, 128   # 2^31.09 elements of Q; sinks' walks cut into parts
    lens = [n] * (T // n) + [T % n]
    ptr = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    plan = sga.SeqPlan(ptr, H, D, kv_heads=1, causal=True, window=200, sinks=3)
    Q, K, V, dO = (filled(T, h, D, seed=s) for s, h in enumerate((H, 1, 1, H)))
    assert Q.numel() > 1 << 31
    out, lse = sga.seq_attn_fwd(plan, Q, K, V)
    dQ, dK, dV = sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO)
    assert plan.device_error() == 0
    # the last rows' own keys: the window before them, and the last sequence's sinks
    first = int(ptr[-2])
    for r in (T - 1, T - 130, first, first + 150, first + 4000):
        keys = torch.tensor(sorted(set(range(first, first + 3)) & set(range(first, r + 1)) | set(range(max(first, r - 199), r + 1))), device="cuda")
        s = torch.einsum("hd,jd->hj", Q[r].double(), K[keys, 0].double()) / D ** 0.5
        p = torch.softmax(s, -1)
        o = p @ V[keys, 0].double()
        assert ((out[r].double() - o).abs() <= 2.0 ** -7 * (p @ V[keys, 0].double().abs()) + 2.0 ** -8 * o.abs()).all(), r
        dp = dO[r].double() @ V[keys, 0].double().T
        ds = p * (dp - (dO[r].double() * out[r].double()).sum(-1, keepdim=True))
        want = ds @ K[keys, 0].double() / D ** 0.5
        bound = (2.0 ** -7 * (ds.abs() + p * dp.abs()) @ K[keys, 0].double().abs()) / D ** 0.5 + 2.0 ** -8 * want.abs() + 1e-3
        assert ((dQ[r].double() - want).abs() <= bound).all(), r
    # a sink of the last sequence gathers all of its rows
    rows = torch.arange(first, T, device="cuda")
    total = torch.zeros(D, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(total)
    for i in range(0, len(rows), 4096):
        r = rows[i:i + 4096]
        p = torch.exp(torch.einsum("ihd,d->ih", Q[r].double(), K[first, 0].double()) / D ** 0.5 - lse[r].double())
        total += torch.einsum("ih,ihd->d", p, dO[r].double())
        mag += torch.einsum("ih,ihd->d", p, dO[r].double().abs())
    assert ((dV[first, 0].double() - total).abs() <= 2.0 ** -7 * mag).all()


def test_feed_forward():
    T, F, M = 1 << 20, 64, 2056   # 2^31.006 elements of G
    X, Wg, Wu = filled(T, F), filled(F, M, seed=1) / 8, filled(F, M, seed=2) / 8
    out, G, U = sga.gated_ff_fwd(X, Wg, Wu)
    assert G.numel() > 1 << 31 and sga.gated_ff_device_error() == 0
    s = slice(T - 1000, None)
    a = sga.gated_ff_fwd(X[s].clone(), Wg, Wu)
    assert all(torch.equal(x[s], y) for x, y in zip((out, G, U), a))
    dO = torch.zeros_like(out)
    dO[s] = filled(1000, M, seed=3)
    grads = sga.gated_ff_bwd(X, Wg, Wu, G, U, dO)
    assert sga.gated_ff_device_error() == 0 and not grads[0][:T - 1000].any()
    ref = ff_bwd_reference(X[s], Wg, Wu, G[s], U[s], dO[s], "silu")   # (the other rows add zeros)
    for name, g in zip(("dX", "dWg", "dWu"), (grads[0][s], *grads[1:])):
        within(g, ref[name], name)
