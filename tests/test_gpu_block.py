"""The dense operators and the edge attention as a model uses them: token
embedding -> norm -> (edge attention over the graph + attention over the whole
graph) -> norm, with gradients to every parameter, against the same model in
64 bits."""
import numpy as np
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga

pytestmark = pytest.mark.gpu

LENS, V, H, HK, D = [37, 1, 70, 0, 130, 12], 23, 4, 2, 32
C = H * D


def batch(seed=0):
    """Random graphs, one behind the other: node tokens, CSR over all nodes, sequence pointers."""
    rng = np.random.default_rng(seed)
    ptr = np.concatenate([[0], np.cumsum(LENS)])
    rows = [np.sort(rng.integers(b, e, rng.integers(1, 6))) for b, e in zip(ptr[:-1], ptr[1:]) for _ in range(e - b)]
    indptr = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(np.int32)
    cu = lambda x, t=torch.int32: torch.as_tensor(np.asarray(x), dtype=t, device="cuda")
    return cu(rng.integers(0, V, ptr[-1]), torch.int64), cu(indptr), cu(np.concatenate(rows)), cu(ptr)


def parameters(dtype):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    p = {"table": r(V, C) * 0.3, "w1": 1 + 0.1 * r(C), "b1": 0.1 * r(C), "w2": 1 + 0.1 * r(C), "b2": 0.1 * r(C),
         "Wq": r(C, C) / C ** 0.5, "Wk": r(C, HK * D) / C ** 0.5, "Wv": r(C, HK * D) / C ** 0.5,
         "Wl": r(C, 3 * C) / C ** 0.5}
    return {n: t.to("cuda", dtype).requires_grad_() for n, t in p.items()}


def model(p, ids, seq_plan, plan):
    x = sga.Embedding.apply(ids, p["table"], C ** 0.5)
    y = sga.LayerNorm.apply(x, p["w1"], p["b1"])
    T = ids.numel()
    q, k, v = (y @ p[n] for n in ("Wq", "Wk", "Wv"))
    whole = sga.SeqAttention.apply(q.view(T, H, D), k.view(T, HK, D), v.view(T, HK, D), seq_plan)
    lq, lk, lv = (t.reshape(T, H, D) for t in (y @ p["Wl"]).split(C, 1))
    local = sga.GTAttention.apply(lq, lk, lv, plan)
    return sga.LayerNorm.apply(x + whole.reshape(T, C) + local.reshape(T, C), p["w2"], p["b2"])


def model64(p, ids, indptr, indices, ptr):
    x = p["table"][ids] * C ** 0.5
    norm = lambda t, w, b: torch.nn.functional.layer_norm(t, (C,), w, b, 1e-5)
    y = norm(x, p["w1"], p["b1"])
    T = ids.numel()
    seq = torch.searchsorted(ptr.long(), torch.arange(T, device="cuda"), right=True)
    same = seq[:, None] == seq[None]
    edges = torch.zeros(T, T, dtype=torch.float64, device="cuda")   # how often an edge is listed
    dst = torch.repeat_interleave(torch.arange(T, device="cuda"), (indptr[1:] - indptr[:-1]).long())
    edges.index_put_((dst, indices.long()), torch.ones(len(dst), dtype=torch.float64, device="cuda"), accumulate=True)

    def attend(q, k, v, count):
        k, v = (t.repeat_interleave(H // t.shape[1], 1) for t in (k, v))
        e = torch.exp(torch.einsum("ihd,jhd->hij", q, k) / D ** 0.5) * count
        return torch.einsum("hij,jhd->ihd", e / e.sum(-1, keepdim=True), v).reshape(T, C)

    whole = attend((y @ p["Wq"]).view(T, H, D), (y @ p["Wk"]).view(T, HK, D), (y @ p["Wv"]).view(T, HK, D), same.double())
    local = attend(*(t.reshape(T, H, D) for t in (y @ p["Wl"]).split(C, 1)), edges)
    return norm(x + whole + local, p["w2"], p["b2"])


def test_a_layer_and_its_gradients():
    """fp32 throughout.  Each operator is within about (sum's length) 2^-24 of
    its terms (their own tests); a few hundred terms and some ten stages, whose
    errors enter the gradients twice, stay under 2 x 10 x 400 x 2^-24 = 5e-4 of
    a tensor's norm, and the products in between add as much."""
    ids, indptr, indices, ptr = batch()
    tf32 = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        p, p64 = parameters(torch.float32), parameters(torch.float64)
        seq_plan = sga.SeqPlan(ptr, H, D, torch.float32, kv_heads=HK, causal=False)
        plan = sga.Plan(indptr, indices, H, D, torch.float32)
        G = torch.randn(ids.numel(), C, generator=torch.Generator().manual_seed(2), dtype=torch.float64).cuda()
        out = model(p, ids, seq_plan, plan)
        (out * G.float()).sum().backward()
        ref = model64(p64, ids, indptr, indices, ptr)
        (ref * G).sum().backward()
    finally:
        torch.backends.cuda.matmul.allow_tf32 = tf32
    pairs = [("out", out.detach(), ref.detach())] + [(n, p[n].grad, p64[n].grad) for n in p]
    for name, a, b in pairs:
        assert float((a.double() - b).norm()) <= 1e-3 * float(b.norm()), name
    assert seq_plan.device_error() == 0 and plan.device_error() == 0 and sga.embed_device_error() == 0


def test_a_captured_layer():
    """The forward pass in bf16, captured and replayed on new tokens."""
    ids, indptr, indices, ptr = batch(3)
    p = {n: t.detach() for n, t in parameters(torch.bfloat16).items()}
    seq_plan, plan = sga.SeqPlan(ptr, H, D, kv_heads=HK, causal=False), sga.Plan(indptr, indices, H, D)
    with torch.no_grad():
        model(p, ids, seq_plan, plan)   # (libraries initialised before the capture)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = model(p, ids, seq_plan, plan)
        ids.copy_((ids * 7 + 5) % V)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, model(p, ids, seq_plan, plan))


@pytest.mark.parametrize("dtype,heads,kv,width", [(torch.bfloat16, 4, 2, 64), (torch.bfloat16, 2, 2, 128),
                                                  (torch.bfloat16, 4, 1, 32), (torch.float32, 4, 2, 32)])
def test_calls_in_a_row_equal_calls_apart(dtype, heads, kv, width):
    """Kernels start while the one before them ends: a chain of calls, each on the
    results of earlier ones and into buffers that earlier ones read, gives bit
    for bit what the same calls give one by one, and captured."""
    lens, c, rows = [300, 1, 70, 129, 700], heads * width, 90
    T = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)
    ptr = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    seqs = sga.SeqPlan(ptr, heads, width, dtype, kv_heads=kv, causal=True)
    few, many = (torch.randint(0, n, (T,), generator=gen, device="cuda") for n in (rows, 70000))
    tables, w, b, dO = (r(rows, c), r(70000, c)), r(c), r(c), r(T, heads, width)
    indptr = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    edge = sga.Plan(indptr, indptr[:-1].flip(0).contiguous(), heads, width, dtype)
    x, y, dx, o, dq, e = (torch.empty(T, c, device="cuda", dtype=dtype) for _ in range(6))
    k, v, dk, dv = (torch.empty(T, kv, width, device="cuda", dtype=dtype) for _ in range(4))
    mean, rstd, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, heads, device="cuda")
    dw, db, dts = torch.empty_like(w), torch.empty_like(b), [torch.empty_like(t) for t in tables]
    h = lambda t: t.view(T, heads, width)
    steps = []
    for i, ids in enumerate((few, many)):
        steps += [
            lambda i=i, ids=ids: sga.embed_fwd(ids, tables[i], out=x),
            lambda: sga.layer_norm_fwd(x, w, b, out=y, mean=mean, rstd=rstd),
            lambda: k.copy_(h(y)[:, :kv]), lambda: v.copy_(h(x)[:, -kv:]),
            lambda: sga.seq_attn_fwd(seqs, h(y), k, v, out=h(o), lse=lse),
            lambda: sga.seq_attn_bwd(seqs, h(y), k, v, h(o), lse, dO, dQ=h(dq), dK=dk, dV=dv),
            lambda: sga.seq_attn_fwd(seqs, h(dq), dk, dv, out=h(e)),
            lambda: sga.seq_attn_fwd(seqs, h(o), dk, v, out=h(dx)),
            lambda: sga.layer_norm_bwd(x, w, mean, rstd, dq, dX=dx, dweight=dw, dbias=db),
            lambda: sga.layer_norm_fwd(dx, dw, db, out=dq),
            lambda i=i, ids=ids: sga.embed_bwd(ids, dx, len(tables[i]), dTable=dts[i]),
            lambda i=i: sga.embed_fwd(few, dts[i], out=x),
            lambda: e.add_(sga.gt_attn_fwd(edge, h(x), h(dq), h(y))[0].view(T, c)),
            lambda: sga.layer_norm_fwd(e, w, b, out=e),
        ]
    results = [x, y, dx, o, dq, e, k, v, dk, dv, mean, rstd, lse, dw, db, *dts]

    def run(apart):
        for step in steps:
            step()
            if apart:
                torch.cuda.synchronize()

    run(True)
    want = [t.clone() for t in results]
    assert all(torch.isfinite(t.float()).all() for t in want)
    for _ in range(5):
        for t in results:
            t.fill_(1)
        run(False)
        torch.cuda.synchronize()
        assert all(torch.equal(t, u) for t, u in zip(results, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(False)
        run(False)
    for _ in range(3):
        for t in results:
            t.fill_(1)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, u) for t, u in zip(results, want))
    assert seqs.device_error() == 0 and edge.device_error() == 0 and sga.embed_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forked_streams(dtype):
    """Calls on two streams that fork and join, eager and in one captured graph:
    a call waits for what its stream waits for, not for the kernel before it only."""
    T, c, rows = 1200, 128, 50
    gen = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)
    seqs = sga.SeqPlan(torch.tensor([0, 500, 501, T], dtype=torch.int32, device="cuda"), 2, 64, dtype, causal=False)
    ids, table, w, b = torch.randint(0, rows, (T,), generator=gen, device="cuda"), r(rows, c), r(c), r(c)
    x, y, z, o, dt = (torch.empty(n, c, device="cuda", dtype=dtype) for n in (T, T, T, T, rows))
    h = lambda t: t.view(T, 2, 64)
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        sga.embed_fwd(ids, table, out=x)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            sga.layer_norm_fwd(x, w, b, out=y)           # beside the attention on the main stream
        sga.seq_attn_fwd(seqs, h(x), h(x), h(x), out=h(z))
        main.wait_stream(side)
        sga.seq_attn_fwd(seqs, h(y), h(z), h(x), out=h(o))   # of both
        side.wait_stream(main)
        with torch.cuda.stream(side):
            sga.embed_bwd(ids, o, rows, dTable=dt)
            sga.layer_norm_fwd(o, w, b, out=y)
        main.wait_stream(side)
        sga.layer_norm_fwd(y, w, b, out=x)

    results = (x, y, z, o, dt)
    run()
    torch.cuda.synchronize()
    sga.embed_fwd(ids, table, out=x)
    torch.cuda.synchronize()
    ref = [sga.layer_norm_fwd(x, w, b)[0], sga.seq_attn_fwd(seqs, h(x), h(x), h(x))[0]]
    torch.cuda.synchronize()
    ref.append(sga.seq_attn_fwd(seqs, h(ref[0]), ref[1], h(x))[0].view(T, c))
    torch.cuda.synchronize()
    y2 = sga.layer_norm_fwd(ref[2], w, b)[0]
    torch.cuda.synchronize()
    want = (sga.layer_norm_fwd(y2, w, b)[0], y2, ref[1].view(T, c), ref[2], sga.embed_bwd(ids, ref[2], rows))
    torch.cuda.synchronize()
    for _ in range(5):
        for t in results:
            t.fill_(1)
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(t, u) for t, u in zip(results, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(5):
        for t in results:
            t.fill_(1)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, u) for t, u in zip(results, want))
    assert seqs.device_error() == 0 and sga.embed_device_error() == 0
