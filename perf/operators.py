"""Measured cases of the operators around the edge-attention layers: attention over packed sequences, layer norm
and embedding lookup, each forward and backward.

`own` False: the plain forms, in elementary torch operations.  `own` True: the package's kernels.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # global attention inside each graph of a batch of molecules: 9 to 38 atoms a graph, every pair visible
        {"name": "attn_fwd_molecules", "op": "attn_fwd", "lens": _spread(9, 38, 128, 1), "heads": 4, "kv_heads": 4, "dim": 64,
         "causal": False, "dtype": "bf16"},
        # long node or token sequences in one packed batch, causal, four query heads to a key head
        {"name": "attn_fwd_long", "op": "attn_fwd", "lens": "16384,1501,1", "heads": 8, "kv_heads": 2, "dim": 128,
         "causal": True, "dtype": "bf16"},
        # training step of the global attention on small graphs in fp32, odd lengths, one of a single node
        {"name": "attn_bwd_graphs_f32", "op": "attn_bwd", "lens": "333,1,70,512,129", "heads": 4, "kv_heads": 4, "dim": 32,
         "causal": False, "dtype": "f32"},
        # training step on long sequences, causal, grouped heads
        {"name": "attn_bwd_long", "op": "attn_bwd", "lens": "8192,4099,1,600", "heads": 8, "kv_heads": 4, "dim": 128,
         "causal": True, "dtype": "bf16"},
        # norm between two layers of a small graph (4 heads of 64)
        {"name": "norm_fwd_small", "op": "norm_fwd", "rows": 2708, "width": 256, "dtype": "bf16", "weight": "f32"},
        # the same on a graph of a million nodes
        {"name": "norm_fwd_rmat", "op": "norm_fwd", "rows": 1048576, "width": 256, "dtype": "bf16", "weight": "bf16"},
        # gradient of a norm of an odd width, fp32
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 4099, "width": 301, "dtype": "f32", "weight": "f32"},
        # gradient of the norm of a large graph (4 heads of 128), fp32 master weights
        {"name": "norm_bwd_large", "op": "norm_bwd", "rows": 169343, "width": 512, "dtype": "bf16", "weight": "f32"},
        # atom types of a batch of molecules
        {"name": "embed_fwd_atoms", "op": "embed_fwd", "tokens": 3001, "vocab": 119, "width": 256, "dtype": "f32", "ids": "int64"},
        # node tokens from a large vocabulary, Zipf frequencies
        {"name": "embed_fwd_tokens", "op": "embed_fwd", "tokens": 524288, "vocab": 50257, "width": 512, "dtype": "bf16", "ids": "int64"},
        # gradient of the atom types: few rows, each with many tokens
        {"name": "embed_bwd_atoms", "op": "embed_bwd", "tokens": 30011, "vocab": 119, "width": 100, "dtype": "f32", "ids": "int32"},
        # gradient of the large vocabulary: a few rows hold a large part of the tokens, many rows none
        {"name": "embed_bwd_tokens", "op": "embed_bwd", "tokens": 524288, "vocab": 50257, "width": 512, "dtype": "bf16", "ids": "int64"},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attn_fwd", "attn_bwd", "norm_fwd", "norm_bwd", "embed_fwd", "embed_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    case = {"op": op, "dtype": dtype}
    if op.startswith("attn"):
        dim = rng.choice([32, 64, 128])
        kv = rng.choice([1, 2, 4])
        heads = kv * rng.choice([1, 2, 4])
        longest = log(4, 8192)
        seqs = max(1, min(128, log(1, 128), 16384 // longest))
        lens = [log(1, longest) for _ in range(seqs - 1)] + [longest]
        rng.shuffle(lens)
        case |= {"heads": heads, "kv_heads": kv, "dim": dim, "causal": rng.random() < 0.6}
        while True:   # no more work than the largest listed case (in fp32, which runs off the tensor cores, an eighth)
            case["lens"] = ",".join(map(str, lens))
            if work(case)["flops"] <= (5e11 if dtype == "bf16" else 6e10):
                break
            lens = [(n + 1) // 2 for n in lens]
    elif op.startswith("norm"):
        width = rng.choice([rng.randrange(1, 2049), 8 * rng.randrange(1, 513)])
        case |= {"rows": log(1, max(2, (1 << 27) // width)), "width": width, "weight": rng.choice([dtype, "f32"])}
    else:
        width = rng.choice([rng.randrange(1, 513), 8 * rng.randrange(1, 129)])
        case |= {"tokens": log(1, max(2, (1 << 27) // width)), "vocab": log(1, 100000), "width": width,
                 "ids": rng.choice(["int32", "int64"])}
    return case


def _spread(lo, hi, n, seed):
    """n lengths in [lo, hi] as a text, the same every time."""
    r = np.random.default_rng(seed)
    return ",".join(str(x) for x in r.integers(lo, hi + 1, n))


def _lengths(case):
    return [int(x) for x in case["lens"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, mean=0.0, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    st = dict(case)
    if case["op"].startswith("attn"):
        lens = _lengths(case)
        T, H, Hk, D = sum(lens), case["heads"], case["kv_heads"], case["dim"]
        st["longest"] = max(lens)
        st["seq_ptr"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        st["Q"], st["K"], st["V"] = normal(T, H, D), normal(T, Hk, D), normal(T, Hk, D)
        if case["op"] == "attn_bwd":
            st["dOut"] = normal(T, H, D)
            st["out"], st["lse"] = _attn_fwd(st)
        if own:   # the handle of a batch's lengths, made once and used by every layer of the model
            import sparse_graph_attention_csr_gb300 as sga
            st["plan"] = sga.SeqPlan(st["seq_ptr"], H, D, dt, kv_heads=Hk, causal=case["causal"])
    elif case["op"].startswith("norm"):
        n, c, wt = case["rows"], case["width"], DTYPES[case["weight"]]
        st["X"] = normal(n, c, mean=0.3, std=1.7)
        st["w"], st["b"] = normal(c, dtype=wt, mean=1.0, std=0.1), normal(c, dtype=wt, std=0.1)
        if case["op"] == "norm_bwd":
            st["dOut"] = normal(n, c)
            _, st["mean"], st["rstd"] = _norm_fwd(st)
    else:
        t, v, c = case["tokens"], case["vocab"], case["width"]
        u = torch.rand(t, generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(v + 1)) - 1).floor().clamp(0, v - 1)   # frequency of id k falls as 1 / (k + 1)
        st["ids"] = ids.to(torch.int32 if case["ids"] == "int32" else torch.int64)
        st["scale"] = math.sqrt(c)
        if case["op"] == "embed_fwd":
            st["table"] = normal(v, c, std=0.05)
        else:
            st["dOut"] = normal(t, c)
    return st


def run(st):
    if own:
        return _own(st)
    return {"attn_fwd": _attn_fwd, "attn_bwd": _attn_bwd, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd,
            "embed_fwd": _embed_fwd, "embed_bwd": _embed_bwd}[st["op"]](st)


def _own(st):
    import sparse_graph_attention_csr_gb300 as sga
    op = st["op"]
    if op == "attn_fwd":
        return sga.seq_attn_fwd(st["plan"], st["Q"], st["K"], st["V"])
    if op == "attn_bwd":
        return sga.seq_attn_bwd(st["plan"], st["Q"], st["K"], st["V"], st["out"], st["lse"], st["dOut"])
    if op == "norm_fwd":
        return sga.layer_norm_fwd(st["X"], st["w"], st["b"], eps=1e-5)
    if op == "norm_bwd":
        return sga.layer_norm_bwd(st["X"], st["w"], st["mean"], st["rstd"], st["dOut"])
    if op == "embed_fwd":
        return sga.embed_fwd(st["ids"], st["table"], scale=st["scale"])
    return sga.embed_bwd(st["ids"], st["dOut"], st["vocab"], scale=st["scale"])


# ---- plain forms ------------------------------------------------------------


def _grid(st):
    """Every sequence padded to the longest: the packed row of (sequence, position), whether there is one, and each
    packed row's sequence and position."""
    ptr = st["seq_ptr"].long()
    pos = torch.arange(st["longest"], device="cuda")
    row = ptr[:-1, None] + pos[None]
    there = row < ptr[1:, None]
    t = torch.arange(st["Q"].shape[0], device="cuda")
    seq = torch.searchsorted(ptr, t, right=True) - 1
    return torch.where(there, row, torch.zeros_like(row)), there, seq, t - ptr[seq]


def _visible(st, there):
    m = there[:, None, :].expand(-1, st["longest"], -1)
    if st["causal"]:
        pos = torch.arange(st["longest"], device="cuda")
        m = m & (pos[None, :] <= pos[:, None])[None]
    return m[:, None, None]


def _heads(x, row, kv_heads):
    """[T, h, D] -> [sequence, kv head, heads of the group, position, D] in fp32."""
    b, n = row.shape
    return x.float()[row].view(b, n, kv_heads, -1, x.shape[-1]).permute(0, 2, 3, 1, 4)


def _packed(y, seq, pos):
    """The inverse of _heads: [sequence, kv head, group, position, D] -> [T, h, D]."""
    b, k, r, n, d = y.shape
    return y.reshape(b, k * r, n, d)[seq, :, pos]


def _attn_fwd(st):
    row, there, seq, pos = _grid(st)
    kv = st["kv_heads"]
    q, k, v = (_heads(st[n], row, kv) for n in ("Q", "K", "V"))
    s = (q / math.sqrt(st["dim"])) @ k.transpose(-1, -2)
    s = torch.where(_visible(st, there), s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    s = torch.exp(s - top)
    total = s.sum(-1, keepdim=True)
    out = (s @ v) / total
    lse = top + torch.log(total)
    return _packed(out, seq, pos).to(st["Q"].dtype), _packed(lse, seq, pos)[..., 0]


def _attn_bwd(st):
    row, there, seq, pos = _grid(st)
    kv, scale = st["kv_heads"], 1.0 / math.sqrt(st["dim"])
    q, k, v, o, do = (_heads(st[n], row, kv) for n in ("Q", "K", "V", "out", "dOut"))
    lse = _heads(st["lse"][..., None], row, kv)
    live = there[:, None, None, :, None]
    p = torch.exp((q * scale) @ k.transpose(-1, -2) - lse)
    p = torch.where(_visible(st, there) & live, p, 0.0)
    dv = (p.transpose(-1, -2) @ do).sum(2, keepdim=True)
    p *= do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True)
    dq = (p @ k) * scale
    dk = (p.transpose(-1, -2) @ q).sum(2, keepdim=True) * scale
    return tuple(_packed(x, seq, pos).to(st["Q"].dtype) for x in (dq, dk, dv))


def _norm_fwd(st):
    x = st["X"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(1) + 1e-5)
    y = c * rstd[:, None] * st["w"].float() + st["b"].float()
    return y.to(st["X"].dtype), mean, rstd


def _norm_bwd(st):
    x, dy = st["X"].float(), st["dOut"].float()
    xhat = (x - st["mean"][:, None]) * st["rstd"][:, None]
    g = dy * st["w"].float()
    dx = st["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    dw, db = (dy * xhat).sum(0, dtype=torch.float64), dy.sum(0, dtype=torch.float64)
    return dx.to(st["X"].dtype), dw.to(st["w"].dtype), db.to(st["w"].dtype)


def _embed_fwd(st):
    return (st["table"][st["ids"].long()].float() * st["scale"]).to(st["table"].dtype)


def _embed_bwd(st):
    d = st["dOut"]
    total = torch.zeros(st["vocab"], d.shape[1], dtype=torch.float64, device="cuda")
    total.index_add_(0, st["ids"].long(), d.double())
    return (total * st["scale"]).to(d.dtype)


# ---- what a pass cannot do without ------------------------------------------


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("attn"):
        lens = _lengths(case)
        T, H, Hk, D = sum(lens), case["heads"], case["kv_heads"], case["dim"]
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens) * H
        q, kv, stat = T * H * D * e, T * Hk * D * e, T * H * 4
        if op == "attn_fwd":
            return {"bytes": 2 * q + 2 * kv + stat, "flops": 4 * D * pairs}
        return {"bytes": 4 * q + 4 * kv + stat, "flops": 10 * D * pairs}
    if op.startswith("norm"):
        n, c = case["rows"], case["width"]
        we = 2 if case["weight"] == "bf16" else 4
        if op == "norm_fwd":
            return {"bytes": 2 * n * c * e + 8 * n + 2 * c * we, "flops": 8 * n * c}
        return {"bytes": 3 * n * c * e + 8 * n + 3 * c * we, "flops": 13 * n * c}
    t, v, c = case["tokens"], case["vocab"], case["width"]
    ids = t * (4 if case["ids"] == "int32" else 8)
    if op == "embed_fwd":
        return {"bytes": ids + min(t, v) * c * e + t * c * e, "flops": t * c}
    return {"bytes": ids + t * c * e + v * c * e, "flops": t * c}


# ---- the definitions in 64 bits ---------------------------------------------


def exact(case, seed):
    st = _inputs(case, seed)
    return {"attn_fwd": _exact_attn, "attn_bwd": _exact_attn, "norm_fwd": _exact_norm, "norm_bwd": _exact_norm,
            "embed_fwd": _exact_embed, "embed_bwd": _exact_embed}[case["op"]](case, st)


def _inputs(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _exact_attn(case, st):
    """Row by row of the definition: each sequence's keys alone, one sequence and head at a time, in blocks of rows."""
    lens = _lengths(case)
    H, Hk, D, back = case["heads"], case["kv_heads"], case["dim"], case["op"] == "attn_bwd"
    if work(case)["flops"] * (2 if case["causal"] else 1) > 6e12:
        return None
    f = {n: st[n].double() for n in ("Q", "K", "V") + (("dOut",) if back else ())}
    out, lse = torch.zeros_like(f["Q"]), torch.zeros(sum(lens), H, dtype=torch.float64, device="cuda")
    grad = {n: torch.zeros_like(f[n]) for n in ("Q", "K", "V")}
    at = 0
    for n in lens:
        for h in range(H):
            kh = h // (H // Hk)
            K, V = f["K"][at:at + n, kh], f["V"][at:at + n, kh]
            for i0 in range(0, n, 2048):
                i1 = min(n, i0 + 2048)
                m = i1 if case["causal"] else n
                rows = slice(at + i0, at + i1)
                logits = torch.einsum("id,jd->ij", f["Q"][rows, h], K[:m]) * D ** -0.5
                if case["causal"]:
                    logits.masked_fill_(torch.ones(i1 - i0, m, dtype=torch.bool, device="cuda").triu(i0 + 1), -math.inf)
                z = torch.logsumexp(logits, 1)
                w = torch.exp(logits - z[:, None])
                o = torch.einsum("ij,jd->id", w, V[:m])
                out[rows, h], lse[rows, h] = o, z
                if back:
                    do = f["dOut"][rows, h]
                    grad["V"][at:at + m, kh] += torch.einsum("ij,id->jd", w, do)
                    ds = w * (torch.einsum("id,jd->ij", do, V[:m]) - (do * o).sum(1)[:, None]) * D ** -0.5
                    grad["Q"][rows, h] = torch.einsum("ij,jd->id", ds, K[:m])
                    grad["K"][at:at + m, kh] += torch.einsum("ij,id->jd", ds, f["Q"][rows, h])
        at += n
    return (grad["Q"], grad["K"], grad["V"]) if back else (out, lse)


def _exact_norm(case, st):
    """The forward of the definition, and its gradient by differentiating it in 64 bits (rows in blocks)."""
    x, w, b = st["X"].double(), st["w"].double(), st["b"].double()
    c = x.shape[1]
    if case["op"] == "norm_fwd":
        mean = x.sum(1) / c
        var = (x ** 2).sum(1) / c - mean ** 2
        rstd = (var.clamp_min(0) + 1e-5) ** -0.5
        return (x - mean[:, None]) * rstd[:, None] * w + b, mean, rstd
    dx, dw, db = torch.empty_like(x), torch.zeros_like(w), torch.zeros_like(b)
    for i in range(0, x.shape[0], 1 << 18):
        xi, wi, bi = x[i:i + (1 << 18)].clone().requires_grad_(), w.clone().requires_grad_(), b.clone().requires_grad_()
        with torch.enable_grad():
            d = xi - xi.sum(1, keepdim=True) / c
            y = d / torch.sqrt((d * d).sum(1, keepdim=True) / c + 1e-5) * wi + bi
            gx, gw, gb = torch.autograd.grad(y, (xi, wi, bi), st["dOut"][i:i + (1 << 18)].double())
        dx[i:i + (1 << 18)] = gx
        dw += gw
        db += gb
    return dx, dw, db


def _exact_embed(case, st):
    ids = st["ids"].long()
    if case["op"] == "embed_fwd":
        return torch.index_select(st["table"].double(), 0, ids) * st["scale"]
    order = torch.argsort(ids, stable=True)
    sums = torch.zeros(case["vocab"] + 1, case["width"], dtype=torch.float64, device="cuda")
    counts = torch.bincount(ids, minlength=case["vocab"])
    ends = torch.cumsum(counts, 0)
    for c0 in range(0, case["width"], 64):   # running totals over the sorted tokens, differences at the ends
        run_ = torch.cumsum(st["dOut"][:, c0:c0 + 64].double()[order], 0)
        run_ = torch.cat([torch.zeros_like(run_[:1]), run_])
        sums[:-1, c0:c0 + 64] = run_[ends] - run_[ends - counts]
    return sums[:-1] * st["scale"]
