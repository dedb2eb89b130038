"""Measured cases of the operators of a transformer layer over packed sequences: the norm of query and key heads with
their rotary positions, attention with a sliding window and first rows that stay visible, and the gated product of a
feed-forward block, each forward and backward.

`own` False: the plain forms, in elementary torch operations.  `own` True: the package's kernels.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128   # rows that the plain form of windowed attention takes together


def listed():
    return [
        # next tokens of 37 sequences far into their contexts, one row each, in fp32: latency
        {"name": "qk_fwd_tokens", "op": "qk_fwd", "lens": "1," * 36 + "1", "heads": 4, "kv_heads": 2, "dim": 64, "axes": "",
         "interleaved": False, "fused": False, "dtype": "f32"},
        # a training batch of long sequences, queries and keys as slices of one projection's result
        {"name": "qk_fwd_long", "op": "qk_fwd", "lens": "65536,4099,1", "heads": 16, "kv_heads": 4, "dim": 128, "axes": "",
         "interleaved": False, "fused": True, "dtype": "bf16"},
        # gradient for nodes with three coordinates (time, height, width), neighbouring elements paired, fp32
        {"name": "qk_bwd_axes", "op": "qk_bwd", "lens": "30011", "heads": 4, "kv_heads": 4, "dim": 64, "axes": "8,12,12",
         "interleaved": True, "fused": False, "dtype": "f32"},
        # gradient of the long training batch
        {"name": "qk_bwd_long", "op": "qk_bwd", "lens": "65536,4099,1", "heads": 16, "kv_heads": 4, "dim": 128, "axes": "",
         "interleaved": False, "fused": True, "dtype": "bf16"},
        # neighbourhoods along chains of 9 to 300 nodes with two global nodes at the head of each, both directions
        {"name": "window_fwd_chains", "op": "win_fwd", "lens": _spread(9, 300, 64, 1), "heads": 4, "kv_heads": 4, "dim": 64,
         "causal": False, "window": 17, "sinks": 2, "dtype": "bf16"},
        # long sequences, four query heads to a key head, a window that ends inside tiles
        {"name": "window_fwd_long", "op": "win_fwd", "lens": "32768,1501,1", "heads": 8, "kv_heads": 2, "dim": 128,
         "causal": True, "window": 1000, "sinks": 4, "dtype": "bf16"},
        # training step of a windowed layer in fp32, odd lengths
        {"name": "window_bwd_f32", "op": "win_bwd", "lens": "1045,1,333,2049", "heads": 4, "kv_heads": 2, "dim": 32,
         "causal": False, "window": 129, "sinks": 1, "dtype": "f32"},
        # training step on long sequences
        {"name": "window_bwd_long", "op": "win_bwd", "lens": "16384,8191,1,600", "heads": 8, "kv_heads": 4, "dim": 128,
         "causal": True, "window": 1024, "sinks": 4, "dtype": "bf16"},
        # feed-forward block of a layer on a small graph (4 heads of 64)
        {"name": "ff_fwd_small", "op": "ff_fwd", "rows": 2708, "width": 256, "hidden": 680, "act": "gelu", "dtype": "bf16"},
        # the same of a wide layer on long sequences
        {"name": "ff_fwd_large", "op": "ff_fwd", "rows": 32769, "width": 2048, "hidden": 5632, "act": "silu", "dtype": "bf16"},
        # training step in fp32, every size odd
        {"name": "ff_bwd_odd", "op": "ff_bwd", "rows": 4099, "width": 301, "hidden": 803, "act": "gelu", "dtype": "f32"},
        # training step of a layer of 4 heads of 256 on long sequences
        {"name": "ff_bwd_large", "op": "ff_bwd", "rows": 16384, "width": 1024, "hidden": 2816, "act": "silu", "dtype": "bf16"},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["qk_fwd", "qk_bwd", "win_fwd", "win_bwd", "ff_fwd", "ff_bwd"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op.startswith("ff"):
        rows, width, hidden = log(1, 65536), log(8, 4096), log(8, 8192)
        if rng.random() < 0.6:   # whole 16 bytes a row, as models have them
            width, hidden = width // 8 * 8, hidden // 8 * 8
        limit = 3e11 if case["dtype"] == "bf16" else 5e10
        while rows > 1 and 12 * rows * width * hidden > limit:
            rows = (rows + 1) // 2
        return case | {"rows": rows, "width": width, "hidden": hidden, "act": rng.choice(["silu", "gelu", "relu"])}
    dim = rng.choice([32, 64, 128])
    kv = rng.choice([1, 2, 4])
    heads = kv * rng.choice([1, 2, 4])
    longest = log(1, 32768)
    seqs = max(1, min(128, log(1, 128), 32768 // longest))
    lens = [log(1, longest) for _ in range(seqs - 1)] + [longest]
    rng.shuffle(lens)
    case |= {"heads": heads, "kv_heads": kv, "dim": dim}
    if op.startswith("qk"):
        pairs = dim // 2
        axes = rng.choice(["", "", "%d,%d" % (pairs // 2, pairs - pairs // 2), "%d,%d,%d" % (pairs // 4, 3 * pairs // 8, 3 * pairs // 8)])
        case |= {"axes": axes, "interleaved": rng.random() < 0.5, "fused": rng.random() < 0.5}
    else:
        case |= {"causal": rng.random() < 0.6, "window": log(1, 4096), "sinks": rng.choice([0, 1, 4, log(1, 200)])}
        limit = 1.2e8 if case["dtype"] == "bf16" else 3e7   # pairs of a row and a key
        while heads * sum(lens) * min(max(lens), case["window"] * (1 if case["causal"] else 2)) > limit:
            lens = [(n + 1) // 2 for n in lens]
    case["lens"] = ",".join(map(str, lens))
    return case


def _spread(lo, hi, n, seed):
    """n lengths in [lo, hi] as a text, the same every time."""
    r = np.random.default_rng(seed)
    return ",".join(str(x) for x in r.integers(lo, hi + 1, n))


def _lengths(case):
    return [int(x) for x in case["lens"].split(",")]


def _axes(case):
    return [int(x) for x in case["axes"].split(",")] if case["axes"] else None


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, mean=0.0, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    st = dict(case)
    if case["op"].startswith("qk"):
        lens, H, Hk, D = _lengths(case), case["heads"], case["kv_heads"], case["dim"]
        T = sum(lens)
        if case["fused"]:   # one projection's result: query, key and value heads of a row side by side
            qkv = normal(T, H + 2 * Hk, D, std=1.3)
            st["Q"], st["K"] = qkv[:, :H], qkv[:, H:H + Hk]
        else:
            st["Q"], st["K"] = normal(T, H, D, std=1.3), normal(T, Hk, D, std=1.3)
        st["wq"], st["wk"] = normal(D, mean=1.0, std=0.1), normal(D, mean=1.0, std=0.1)
        # positions run on in each sequence, from where its context has got to
        first = torch.randint(0, 200000, (len(lens),), generator=g, device="cuda")
        seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"))
        begin = torch.tensor(np.concatenate([[0], np.cumsum(lens)[:-1]]), device="cuda")
        pos = torch.arange(T, device="cuda") - begin[seq]
        if case["axes"]:    # a grid of 24 columns and rows, time behind them
            cols = torch.stack([pos // 576 + first[seq], pos // 24 % 24, pos % 24], 1)
            st["pos"] = cols[:, :len(_axes(case))].contiguous()
        else:
            st["pos"] = pos + first[seq]
        st["eps"], st["base"] = 1e-6, 10000.0
        if case["op"] == "qk_bwd":
            st["dQo"], st["dKo"] = normal(T, H, D), normal(T, Hk, D)
            _, _, st["rq"], st["rk"] = _qk_fwd(st)
        if own:   # the table of a model's frequencies, made once
            import sparse_graph_attention_csr_gb300 as sga
            st["rot"] = sga.Rotary(D, base=st["base"], sections=_axes(case), interleaved=case["interleaved"])
    elif case["op"].startswith("win"):
        lens, H, Hk, D = _lengths(case), case["heads"], case["kv_heads"], case["dim"]
        T = sum(lens)
        st["seq_ptr"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        st["reach"] = min(case["window"], max(lens))
        st["Q"], st["K"], st["V"] = normal(T, H, D), normal(T, Hk, D), normal(T, Hk, D)
        if case["op"] == "win_bwd":
            st["dOut"] = normal(T, H, D)
            st["out"], st["lse"] = _win_fwd(st)
        if own:   # the handle of a batch's lengths, made once and used by every layer of the model
            import sparse_graph_attention_csr_gb300 as sga
            st["plan"] = sga.SeqPlan(st["seq_ptr"], H, D, dt, kv_heads=Hk, causal=case["causal"], window=case["window"],
                                     sinks=case["sinks"])
    else:
        n, c, m = case["rows"], case["width"], case["hidden"]
        st["X"] = normal(n, c)
        st["Wg"], st["Wu"] = normal(c, m, std=c ** -0.5), normal(c, m, std=c ** -0.5)
        if case["op"] == "ff_bwd":
            st["dOut"] = normal(n, m)
            _, st["G"], st["U"] = _ff_fwd(st)
    return st


def run(st):
    if own:
        return _own(st)
    return {"qk_fwd": _qk_fwd, "qk_bwd": _qk_bwd, "win_fwd": _win_fwd, "win_bwd": _win_bwd, "ff_fwd": _ff_fwd,
            "ff_bwd": _ff_bwd}[st["op"]](st)


def _own(st):
    import sparse_graph_attention_csr_gb300 as sga
    op = st["op"]
    if op == "qk_fwd":
        return sga.qk_norm_rope_fwd(st["rot"], st["Q"], st["K"], st["pos"], st["wq"], st["wk"], eps=st["eps"])
    if op == "qk_bwd":
        return sga.qk_norm_rope_bwd(st["rot"], st["Q"], st["K"], st["pos"], st["wq"], st["wk"], st["rq"], st["rk"],
                                    st["dQo"], st["dKo"])
    if op == "win_fwd":
        return sga.seq_attn_fwd(st["plan"], st["Q"], st["K"], st["V"])
    if op == "win_bwd":
        # (the plain form's out and lse of a single block of rows are views)
        return sga.seq_attn_bwd(st["plan"], st["Q"], st["K"], st["V"], st["out"].contiguous(), st["lse"].contiguous(), st["dOut"])
    if op == "ff_fwd":
        return sga.gated_ff_fwd(st["X"], st["Wg"], st["Wu"], act=st["act"])
    return sga.gated_ff_bwd(st["X"], st["Wg"], st["Wu"], st["G"], st["U"], st["dOut"], act=st["act"])


# ---- plain forms ------------------------------------------------------------


def _turns(st):
    """cos and sin [T, 1, D / 2] of every row's angles, formed in 64 bits."""
    pairs = st["dim"] // 2
    freq = st["base"] ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)
    pos = st["pos"].double()
    if st["axes"]:
        axis = torch.repeat_interleave(torch.arange(pos.shape[1], device="cuda"), torch.tensor(_axes(st), device="cuda"))
        angle = pos[:, axis] * freq
    else:
        angle = pos[:, None] * freq
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _rotate(x, cos, sin, interleaved):
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)
    y = (a * cos - b * sin, a * sin + b * cos)
    return torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)


def _qk_fwd(st):
    cos, sin = _turns(st)

    def half(x, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1) + st["eps"])
        return _rotate(x * r[..., None] * w.float(), cos, sin, st["interleaved"]).to(st["Q"].dtype), r

    (q, rq), (k, rk) = half(st["Q"], st["wq"]), half(st["K"], st["wk"])
    return q, k, rq, rk


def _qk_bwd(st):
    cos, sin = _turns(st)

    def half(x, w, r, dy):
        xhat = x.float() * r[..., None]
        dn = _rotate(dy.float(), cos, -sin, st["interleaved"])
        g = dn * w.float()
        dx = r[..., None] * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        return dx.to(x.dtype), (dn * xhat).sum((0, 1), dtype=torch.float64).to(w.dtype)

    (dq, dwq), (dk, dwk) = half(st["Q"], st["wq"], st["rq"], st["dQo"]), half(st["K"], st["wk"], st["rk"], st["dKo"])
    return dq, dk, dwq, dwk


def _near(st):
    """The rows in blocks: the rows of each [n, BLOCK], the keys of each [n, m] (those that the window of one of its rows
    may reach, and the first rows of its first row's sequence; both ways as many behind its last row as there are first
    rows, since those of a sequence that begins there, or shortly before, may lie behind its windows), and which pairs are
    visible [n, BLOCK, m]."""
    ptr = st["seq_ptr"].long()
    dev = ptr.device
    T, w = st["Q"].shape[0], st["reach"]
    n = (T + BLOCK - 1) // BLOCK
    first = torch.arange(n, device=dev)[:, None] * BLOCK
    row = first + torch.arange(BLOCK, device=dev)
    near = first + torch.arange(1 - w, BLOCK + (0 if st["causal"] else max(w, min(st["sinks"], T)) - 1), device=dev)
    begin = ptr[torch.searchsorted(ptr, first, right=True) - 1]
    head = begin + torch.arange(st["sinks"], device=dev)
    key = torch.cat([near, torch.where(head < near[:, :1], head, -torch.ones_like(head))], 1)
    there = (row < T)[..., None] & ((key >= 0) & (key < T))[:, None]
    row, key = row.clamp(0, T - 1), key.clamp(0, T - 1)
    rseq, kseq = torch.searchsorted(ptr, row, right=True) - 1, torch.searchsorted(ptr, key, right=True) - 1
    apart = row[..., None] - key[:, None]
    seen = (apart.abs() < st["window"]) | (key - ptr[kseq] < st["sinks"])[:, None]
    if st["causal"]:
        seen &= apart >= 0
    return row, key, there & seen & (rseq[..., None] == kseq[:, None])


def _heads(x, at, kv_heads):
    """[T, h, D] at [n, m] -> [n, kv head, heads of the group, m, D] in fp32."""
    n, m = at.shape
    return x[at].float().view(n, m, kv_heads, -1, x.shape[-1]).permute(0, 2, 3, 1, 4)


def _packed(y, T):
    """[n, kv head, group, BLOCK, D] -> [T, h, D]."""
    n, k, r, b, d = y.shape
    return y.permute(0, 3, 1, 2, 4).reshape(n * b, k * r, d)[:T]


def _added(y, key, T):
    """[n, kv head, 1, m, D] summed over the keys' rows -> [T, kv head, D]."""
    n, k, _, m, d = y.shape
    return torch.zeros(T, k, d, device=y.device).index_add_(0, key.flatten(), y[:, :, 0].permute(0, 2, 1, 3).reshape(n * m, k, d))


def _win_fwd(st):
    row, key, seen = _near(st)
    kv, T = st["kv_heads"], st["Q"].shape[0]
    q, k, v = _heads(st["Q"], row, kv), _heads(st["K"], key, kv), _heads(st["V"], key, kv)
    s = (q / math.sqrt(st["dim"])) @ k.transpose(-1, -2)
    s = torch.where(seen[:, None, None], s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    s = torch.exp(s - top)
    total = s.sum(-1, keepdim=True)
    return _packed((s @ v) / total, T).to(st["Q"].dtype), _packed(top + torch.log(total), T)[..., 0]


def _win_bwd(st):
    row, key, seen = _near(st)
    kv, T, scale = st["kv_heads"], st["Q"].shape[0], 1.0 / math.sqrt(st["dim"])
    q, do, o = (_heads(st[n], row, kv) for n in ("Q", "dOut", "out"))
    k, v = _heads(st["K"], key, kv), _heads(st["V"], key, kv)
    lse = _heads(st["lse"][..., None], row, kv)
    p = torch.exp((q * scale) @ k.transpose(-1, -2) - lse)
    p = torch.where(seen[:, None, None], p, 0.0)
    dv = (p.transpose(-1, -2) @ do).sum(2, keepdim=True)
    p *= do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True)
    dq = (p @ k) * scale
    dk = (p.transpose(-1, -2) @ q).sum(2, keepdim=True) * scale
    dt = st["Q"].dtype
    return _packed(dq, T).to(dt), _added(dk, key, T).to(dt), _added(dv, key, T).to(dt)


def _act(g, name):
    """The activation and its derivative."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        c = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    on = (g > 0).to(g.dtype)
    return g * on, on


def _ff_fwd(st):
    x, dt = st["X"].float(), st["X"].dtype
    g, u = x @ st["Wg"].float(), x @ st["Wu"].float()
    return (_act(g, st["act"])[0] * u).to(dt), g.to(dt), u.to(dt)


def _ff_bwd(st):
    x, dt = st["X"].float(), st["X"].dtype
    a, slope = _act(st["G"].float(), st["act"])
    do = st["dOut"].float()
    dg, du = do * st["U"].float() * slope, do * a
    dx = dg @ st["Wg"].float().T + du @ st["Wu"].float().T
    return dx.to(dt), (x.T @ dg).to(dt), (x.T @ du).to(dt)


# ---- what a pass cannot do without ------------------------------------------


def _pairs(n, window, sinks, causal):
    """Visible pairs of one sequence of n rows."""
    i = np.arange(n, dtype=np.int64)
    lo, hi = np.maximum(0, i - window + 1), i + 1 if causal else np.minimum(n, i + window)
    return int((hi - lo + np.minimum(sinks, lo)).sum() + (0 if causal else np.maximum(0, min(sinks, n) - hi).sum()))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("ff"):
        n, c, m = case["rows"], case["width"], case["hidden"]
        if op == "ff_fwd":
            return {"bytes": (n * c + 2 * c * m + 3 * n * m) * e, "flops": 4 * n * c * m}
        return {"bytes": (2 * n * c + 4 * c * m + 3 * n * m) * e, "flops": 8 * n * c * m}
    lens = _lengths(case)
    T, H, Hk, D = sum(lens), case["heads"], case["kv_heads"], case["dim"]
    if op.startswith("qk"):
        x, stat, pos = T * (H + Hk) * D * e, T * (H + Hk) * 4, T * 8 * max(1, len(_axes(case) or []))
        return {"bytes": (2 if op == "qk_fwd" else 3) * x + stat + pos, "flops": (8 if op == "qk_fwd" else 14) * T * (H + Hk) * D}
    pairs = sum(_pairs(n, case["window"], case["sinks"], case["causal"]) for n in lens) * H
    q, kv, stat = T * H * D * e, T * Hk * D * e, T * H * 4
    if op == "win_fwd":
        return {"bytes": 2 * q + 2 * kv + stat, "flops": 4 * D * pairs}
    return {"bytes": 4 * q + 4 * kv + stat, "flops": 10 * D * pairs}


# ---- the definitions in 64 bits ---------------------------------------------


def exact(case, seed):
    st = _inputs(case, seed)
    return {"qk": _exact_qk, "wi": _exact_win, "ff": _exact_ff}[case["op"][:2]](case, st)


def _inputs(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _exact_qk(case, st):
    """The definition with a pair of elements as a complex number, turned by exp(i angle); its gradient by differentiation."""
    D, back = case["dim"], case["op"] == "qk_bwd"
    pos = st["pos"].double()
    pos = pos[:, None] if pos.dim() == 1 else pos
    which = [a for a, n in enumerate(_axes(case) or [D // 2]) for _ in range(n)]
    angle = torch.stack([pos[:, which[i]] * math.exp(-2.0 * i / D * math.log(st["base"])) for i in range(D // 2)], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def forward(x, w):
        r = (torch.einsum("thd,thd->th", x, x) / D + st["eps"]) ** -0.5
        y = torch.einsum("thd,th,d->thd", x, r, w)
        if case["interleaved"]:
            y = torch.view_as_real(torch.view_as_complex(y.reshape(*y.shape[:-1], D // 2, 2)) * turn).reshape(y.shape)
        else:
            z = torch.complex(y[..., :D // 2], y[..., D // 2:]) * turn
            y = torch.cat([z.real, z.imag], -1)
        return y, r

    outs = []
    for x, w, dy in ((st["Q"], st["wq"], st.get("dQo")), (st["K"], st["wk"], st.get("dKo"))):
        x, w = x.double().contiguous(), w.double()
        if not back:
            outs.append(forward(x, w))
            continue
        with torch.enable_grad():
            x.requires_grad_(), w.requires_grad_()
            outs.append(torch.autograd.grad(forward(x, w)[0], (x, w), dy.double()))
    return outs[0][0], outs[1][0], outs[0][1], outs[1][1]


def _exact_win(case, st):
    """Row by row of the definition: one sequence and head at a time, in blocks of rows against the keys that are near, and
    the sequence's first rows where those lie before them."""
    lens, w, s, causal = _lengths(case), case["window"], case["sinks"], case["causal"]
    H, Hk, D, back = case["heads"], case["kv_heads"], case["dim"], case["op"] == "win_bwd"
    if sum(n * min(n, 2 * w + 512) for n in lens) * H * D * (10 if back else 4) > 6e12 or len(lens) * H > 2000:
        return None
    f = {n: st[n].double() for n in ("Q", "K", "V") + (("dOut",) if back else ())}
    out, lse = torch.zeros_like(f["Q"]), torch.zeros(sum(lens), H, dtype=torch.float64, device="cuda")
    grad = {n: torch.zeros_like(f[n]) for n in ("Q", "K", "V")}
    at = 0
    for n in lens:
        for i0 in range(0, n, 1024):
            i1 = min(n, i0 + 1024)
            j0, j1 = max(0, i0 - w + 1), i1 if causal else min(n, i1 + w - 1)
            i = torch.arange(i0, i1, device="cuda")
            j = torch.cat([torch.arange(0, min(s, j0), device="cuda"), torch.arange(j0, max(j1, min(s, n) if not causal else 0), device="cuda")])
            hidden = ~(((i[:, None] - j).abs() < w) | (j < s))
            if causal:
                hidden |= j > i[:, None]
            rows, keys = at + i, at + j
            for h in range(H):
                kh = h // (H // Hk)
                K, V = f["K"][keys, kh], f["V"][keys, kh]
                logits = torch.einsum("id,jd->ij", f["Q"][rows, h], K) * D ** -0.5
                logits.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(logits, 1)
                a = torch.exp(logits - z[:, None])
                o = torch.einsum("ij,jd->id", a, V)
                out[rows, h], lse[rows, h] = o, z
                if back:
                    do = f["dOut"][rows, h]
                    grad["V"][keys, kh] += torch.einsum("ij,id->jd", a, do)
                    ds = a * (torch.einsum("id,jd->ij", do, V) - (do * o).sum(1)[:, None]) * D ** -0.5
                    grad["Q"][rows, h] = torch.einsum("ij,jd->id", ds, K)
                    grad["K"][keys, kh] += torch.einsum("ij,id->jd", ds, f["Q"][rows, h])
        at += n
    return (grad["Q"], grad["K"], grad["V"]) if back else (out, lse)


def _exact_ff(case, st):
    """The definition, and the gradients of its product at the given projections by differentiation."""
    if 8 * case["rows"] * case["width"] * case["hidden"] > 6e12:
        return None
    f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu}[case["act"]]
    x, wg, wu = (st[n].double() for n in ("X", "Wg", "Wu"))
    if case["op"] == "ff_fwd":
        g, u = torch.einsum("nc,cm->nm", x, wg), torch.einsum("nc,cm->nm", x, wu)
        return f(g) * u, g, u
    with torch.enable_grad():
        g, u = st["G"].double().requires_grad_(), st["U"].double().requires_grad_()
        dg, du = torch.autograd.grad(f(g) * u, (g, u), st["dOut"].double())
    dx = torch.einsum("nm,cm->nc", dg, wg) + torch.einsum("nm,cm->nc", du, wu)
    return dx, torch.einsum("nc,nm->cm", x, dg), torch.einsum("nc,nm->cm", x, du)
