"""The transformer-layer operators as a model uses them: norm -> one projection to queries, keys and values -> norm and
rotary positions of their heads -> windowed attention -> norm -> gated feed-forward, with gradients to every parameter,
against the same layer in 64 bits; captured; and beside other streams."""
import numpy as np
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from layer_ref import visible

pytestmark = pytest.mark.gpu

LENS, H, HK, D, M, WINDOW, SINKS = [150, 1, 70, 0, 333], 4, 2, 32, 344, 40, 2
C = H * D


def parameters(dtype):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    p = {"w1": 1 + 0.1 * r(C), "w2": 1 + 0.1 * r(C), "Wqkv": r(C, (H + 2 * HK) * D) / C ** 0.5, "wq": 1 + 0.1 * r(D), "wk": 1 + 0.1 * r(D),
         "Wo": r(C, C) / C ** 0.5, "Wg": r(C, M) / C ** 0.5, "Wu": r(C, M) / C ** 0.5, "Wd": r(M, C) / M ** 0.5}
    return {n: t.to("cuda", dtype).requires_grad_() for n, t in p.items()}


def batch(dtype, seed=2):
    ptr = np.concatenate([[0], np.cumsum(LENS)])
    x = torch.randn(int(ptr[-1]), C, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
    pos = np.concatenate([np.stack([np.arange(n) // 12, np.arange(n) % 12], 1) + [90000, 0] for n in LENS])
    return x.to("cuda", dtype), torch.as_tensor(ptr, dtype=torch.int32, device="cuda"), torch.as_tensor(pos, device="cuda")


def layer(p, x, pos, rot, plan):
    T = x.shape[0]
    qkv = (sga.LayerNorm.apply(x, p["w1"]) @ p["Wqkv"]).view(T, H + 2 * HK, D)
    q, k = sga.QKNormRope.apply(qkv[:, :H], qkv[:, H:H + HK], pos, p["wq"], p["wk"], rot, 1e-6)
    x = x + sga.SeqAttention.apply(q, k, qkv[:, H + HK:], plan).reshape(T, C) @ p["Wo"]
    return x + sga.GatedFF.apply(sga.LayerNorm.apply(x, p["w2"]), p["Wg"], p["Wu"], "gelu") @ p["Wd"]


def layer64(p, x, pos, rot):
    T, seen = x.shape[0], torch.block_diag(*[visible(n, True, WINDOW, SINKS).double() for n in LENS if n]).bool()
    norm = lambda t, w: torch.nn.functional.layer_norm(t, (C,), w)
    qkv = (norm(x, p["w1"]) @ p["Wqkv"]).view(T, H + 2 * HK, D)
    f = torch.tensor(rot.freqs, dtype=torch.float64, device="cuda")
    which = torch.tensor([a for a, n in enumerate(rot.sections) for _ in range(n)], device="cuda")
    turn = torch.polar(torch.ones(T, D // 2, dtype=torch.float64, device="cuda"), pos.double()[:, which] * f)[:, None]

    def heads(t, w):
        t = t * ((t * t).mean(-1, keepdim=True) + 1e-6) ** -0.5 * w
        z = torch.complex(t[..., :D // 2], t[..., D // 2:]) * turn
        return torch.cat([z.real, z.imag], -1)

    q, k, v = heads(qkv[:, :H], p["wq"]), heads(qkv[:, H:H + HK], p["wk"]), qkv[:, H + HK:]
    k, v = (t.repeat_interleave(H // HK, 1) for t in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, k).div(D ** 0.5).masked_fill(~seen, -torch.inf)
    x = x + torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v).reshape(T, C) @ p["Wo"]
    y = norm(x, p["w2"])
    return x + (torch.nn.functional.gelu(y @ p["Wg"]) * (y @ p["Wu"])) @ p["Wd"]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_layer_and_its_gradients(dtype):
    """fp32: each operator is within about (sum's length) 2^-24 of its terms (their own tests); a few hundred terms and
    some ten stages, whose errors enter the gradients twice, stay under 2 x 10 x 400 x 2^-24 = 5e-4 of a tensor's norm, and
    the products in between add as much.  bf16: every stage's result is rounded by at most 2^-8 of itself, about 2^-9 of a
    tensor's norm; twelve stages, twice, at random, sqrt(24) 2^-9 = 1e-2, times up to three where a gradient is a
    difference of terms larger than itself."""
    p, p64 = parameters(dtype), {n: t.detach().double().requires_grad_() for n, t in parameters(dtype).items()}
    x, ptr, pos = batch(dtype)
    rot = sga.Rotary(D, sections=[8, 8])
    plan = sga.SeqPlan(ptr, H, D, dtype, kv_heads=HK, causal=True, window=WINDOW, sinks=SINKS)
    x64 = x.double().requires_grad_()
    x.requires_grad_()
    G = torch.randn(x.shape, generator=torch.Generator().manual_seed(5), dtype=torch.float64).to("cuda", dtype)
    out = layer(p, x, pos, rot, plan)
    out.backward(G)
    ref = layer64(p64, x64, pos, rot)
    ref.backward(G.double())
    for name, a, b in [("out", out, ref), ("x", x.grad, x64.grad)] + [(n, p[n].grad, p64[n].grad) for n in p]:
        a, b = a.detach().double(), b.detach()
        assert float((a - b).norm()) <= (1e-3 if dtype == torch.float32 else 3e-2) * float(b.norm()), name
    assert plan.device_error() == 0 and sga.gated_ff_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_captured_layer_equals_the_eager_one(dtype):
    x, ptr, pos = batch(dtype)
    rot = sga.Rotary(D, sections=[8, 8])
    plan = sga.SeqPlan(ptr, H, D, dtype, kv_heads=HK, causal=True, window=WINDOW, sinks=SINKS)
    G = torch.randn(x.shape, device="cuda").to(dtype)

    def step():
        p = {n: t.detach().requires_grad_() for n, t in held.items()}   # (fresh leaves: no eager graph of them lives)
        out = layer(p, x, pos, rot, plan)
        return (out.detach(), *torch.autograd.grad(out, list(p.values()), G))

    held = {n: t.detach() for n, t in parameters(dtype).items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (2, 3):
        x.copy_(batch(dtype, seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(kept, step()))
    assert plan.device_error() == 0 and sga.gated_ff_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_chains_whose_kernels_overlap_equal_the_calls_one_by_one(dtype):
    """Kernels of a chain start while the one before ends, here and on a second stream at the same time."""
    x, ptr, pos = batch(dtype)
    T = x.shape[0]
    rot = sga.Rotary(D, sections=[8, 8], interleaved=True)
    plan = sga.SeqPlan(ptr, H, D, dtype, kv_heads=HK, causal=False, window=WINDOW, sinks=SINKS)
    p = {n: t.detach() for n, t in parameters(dtype).items()}
    qkv = torch.randn(T, H + 2 * HK, D, device="cuda").to(dtype)
    v = qkv[:, H + HK:].contiguous()

    def chain(sync):
        wait = torch.cuda.synchronize if sync else lambda: None
        q, k, rq, rk = sga.qk_norm_rope_fwd(rot, qkv[:, :H], qkv[:, H:H + HK], pos, p["wq"], p["wk"])
        wait()
        o, lse = sga.seq_attn_fwd(plan, q, k, v)
        wait()
        h, G, U = sga.gated_ff_fwd(o.view(T, C), p["Wg"], p["Wu"])
        wait()
        do, dwg, dwu = sga.gated_ff_bwd(o.view(T, C), p["Wg"], p["Wu"], G, U, h)
        wait()
        dq, dk, dv = sga.seq_attn_bwd(plan, q, k, v, o, lse, do.view(T, H, D))
        wait()
        back = sga.qk_norm_rope_bwd(rot, qkv[:, :H], qkv[:, H:H + HK], pos, p["wq"], p["wk"], rq, rk, dq, dk)
        wait()
        return (q, k, o, lse, h, do, dwg, dwu, dv, *back)

    want = chain(True)
    s = torch.cuda.Stream()
    for _ in range(5):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = chain(False)
        mine = chain(False)
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(mine, want)) and all(torch.equal(a, b) for a, b in zip(other, want))
