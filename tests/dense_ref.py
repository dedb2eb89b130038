"""64-bit references of packed-sequence attention, layer norm and embedding,
each with an elementwise bound on the error of a kernel that computes in fp32
and rounds where the dtype says.

Units of rounding: U = 2^-24 for an fp32 operation, R = 2^-8 for a value
rounded to bf16 (0 in fp32).  A sum of n terms in any order is off by at most
(n + 4) U times the sum of their magnitudes (the 4 covers the scale, the
approximate exp2 and its argument)."""
import torch

U = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def seq_reference(seq_ptr, Q, K, V, scale, causal, dOut=None, out_used=None):
    """{name: (value, bound)} in float64 for out, lse and, with dOut, dQ, dK, dV.
    Row by row of the definition: each sequence and head by itself.  The
    gradients' bound takes the forward's rounded out (out_used), from which the
    kernels form Delta."""
    dt, R = Q.dtype, (0.0 if Q.dtype == torch.float32 else ROUND[Q.dtype])
    last = ROUND[dt]
    T, H, D = Q.shape
    g = H // K.shape[1]
    q, k, v = (t.double() for t in (Q, K, V))
    z = lambda t: torch.zeros_like(t)
    out, out_b, lse, lse_b = z(q), z(q), z(q[..., 0]), z(q[..., 0])
    res = {"out": (out, out_b), "lse": (lse, lse_b)}
    if dOut is not None:
        do, ou = dOut.double(), out_used.double()
        dQ, dQb, dK, dKb, dV, dVb = z(q), z(q), z(k), z(k), z(v), z(v)
        res |= {"dQ": (dQ, dQb), "dK": (dK, dKb), "dV": (dV, dVb)}
    ptr = [int(x) for x in seq_ptr]
    for b, e in zip(ptr[:-1], ptr[1:]):
        n = e - b
        if n == 0:
            continue
        vis = torch.ones(n, n, dtype=torch.bool, device=Q.device)
        if causal:
            vis = vis.tril()
        for h in range(H):
            qi, ki, vi = q[b:e, h], k[b:e, h // g], v[b:e, h // g]
            s = torch.where(vis, scale * (qi @ ki.T), -torch.inf)
            ls = torch.logsumexp(s, 1)
            p = torch.exp(s - ls[:, None])
            # a score's error; the exponential's argument is as large as the scores are apart
            ds = (D + 4) * U * scale * (qi.abs() @ ki.abs().T) + 8 * U * (1 + ls.abs()[:, None])
            ds = torch.where(vis, ds, 0.0)
            top = ds.amax(1)
            o = p @ vi
            out[b:e, h], lse[b:e, h] = o, ls
            lse_b[b:e, h] = top + (n + 8) * U * (1 + ls.abs())
            # P rounded (R), its error and the sum's (2 top), the product's sum
            rel = R + 2 * top + 2 * (n + 8) * U
            out_b[b:e, h] = rel[:, None] * (p @ vi.abs()) + last * o.abs() + 1e-30
            if dOut is None:
                continue
            doi, oi = do[b:e, h], ou[b:e, h]
            dp = doi @ vi.T
            delta = (doi * o).sum(1)
            d_delta = (doi.abs() * (oi - o).abs()).sum(1) + (D + 4) * U * (doi.abs() * oi.abs()).sum(1)
            # lse is the kernel's own, within lse_b
            pe = p * (ds + lse_b[b:e, h][:, None] + 8 * U * (1 + ls.abs()[:, None]))
            dsv = p * (dp - delta[:, None])
            dse = (R + 4 * U) * dsv.abs() + pe * (dp - delta[:, None]).abs() + \
                p * ((D + 4) * U * (doi.abs() @ vi.abs().T) + d_delta[:, None])
            sums = (n * g + 8) * U
            dQ[b:e, h] = scale * (dsv @ ki)
            dQb[b:e, h] = scale * (dse @ ki.abs() + sums * (dsv.abs() @ ki.abs()))
            dK[b:e, h // g] += scale * (dsv.T @ qi)
            dKb[b:e, h // g] += scale * (dse.T @ qi.abs() + sums * (dsv.abs().T @ qi.abs()))
            dV[b:e, h // g] += p.T @ doi
            dVb[b:e, h // g] += (R * p + pe + sums * p).T @ doi.abs()
    if dOut is not None:
        for x, xb in ((dQ, dQb), (dK, dKb), (dV, dVb)):
            xb += last * (x.abs() + xb) + 1e-30
    return res


def norm_reference(X, weight, bias, eps, dOut=None):
    """{name: (value, bound)} of out, mean, rstd and, with dOut, dX, dweight, dbias."""
    last = ROUND[X.dtype]
    C = X.shape[-1]
    x = X.double().reshape(-1, C)
    w = torch.ones(C, dtype=torch.float64, device=X.device) if weight is None else weight.double()
    b = torch.zeros_like(w) if bias is None else bias.double()
    n = C + 8
    mean = x.mean(1)
    mean_b = n * U * x.abs().mean(1)
    c = x - mean[:, None]
    var = (c * c).mean(1)
    rstd = (var + eps) ** -0.5
    # (x - mean): off by mean_b and a rounding; the variance by twice that times |c|, and its sum
    cb = mean_b[:, None] + U * c.abs()
    var_b = (2 * c.abs() * cb + cb * cb).mean(1) + n * U * var
    # d(rstd) <= var_b / (var + eps)^1.5 / 2; where var_b is not small the plain interval bound
    low = torch.clamp(var - var_b, min=0) + eps
    rstd_b = (low ** -0.5 - rstd) + 8 * U * low ** -0.5 if eps > 0 else 0.5 * var_b * rstd ** 3 * 2 + 8 * U * rstd
    xh = c * rstd[:, None]
    xh_b = cb * (rstd + rstd_b)[:, None] + c.abs() * rstd_b[:, None] + 4 * U * xh.abs()
    y = xh * w + b
    y_b = xh_b * w.abs() + 4 * U * ((xh * w).abs() + b.abs())
    y_b = y_b + last * (y.abs() + y_b) + 1e-30
    lead = X.shape[:-1]
    res = {"out": (y.reshape(X.shape), y_b.reshape(X.shape)), "mean": (mean.reshape(lead), (mean_b + 1e-30).reshape(lead)),
           "rstd": (rstd.reshape(lead), rstd_b.reshape(lead))}
    if dOut is not None:
        dy = dOut.double().reshape(-1, C)
        N = dy.shape[0]
        g = dy * w
        c1, c2 = g.mean(1), (g * xh).mean(1)
        c1_b = n * U * g.abs().mean(1)
        c2_b = n * U * (g * xh).abs().mean(1) + (g.abs() * xh_b).mean(1)
        dx = rstd[:, None] * (g - c1[:, None] - xh * c2[:, None])
        mag = g.abs() + c1.abs()[:, None] + (xh * c2[:, None]).abs()
        dx_b = rstd[:, None] * (6 * U * mag + c1_b[:, None] + xh_b * c2.abs()[:, None] + (xh.abs() + xh_b) * c2_b[:, None]) + \
            rstd_b[:, None] * (mag + c1_b[:, None] + (xh.abs() + xh_b) * c2_b[:, None])
        dx_b = dx_b + last * (dx.abs() + dx_b) + 1e-30
        wl = ROUND[weight.dtype] if weight is not None else U
        dw, db = (dy * xh).sum(0), dy.sum(0)
        dw_b = (N + 8) * U * (dy * xh).abs().sum(0) + (dy.abs() * xh_b).sum(0)
        db_b = (N + 8) * U * dy.abs().sum(0)
        res |= {"dX": (dx.reshape(X.shape), dx_b.reshape(X.shape)),
                "dweight": (dw, dw_b + wl * (dw.abs() + dw_b) + 1e-30), "dbias": (db, db_b + wl * (db.abs() + db_b) + 1e-30)}
    return res


def embed_bwd_reference(ids, dOut, V, scale, padding_idx=None):
    C = dOut.shape[-1]
    d, i = dOut.double().reshape(-1, C), ids.reshape(-1).long()
    ok = (i >= 0) & (i < V)
    if padding_idx is not None:
        ok &= i != padding_idx
    d, i = d[ok], i[ok]
    val = torch.zeros(V, C, dtype=torch.float64, device=d.device).index_add_(0, i, d) * scale
    mag = torch.zeros(V, C, dtype=torch.float64, device=d.device).index_add_(0, i, d.abs()) * abs(scale)
    count = torch.bincount(i, minlength=V)[:V].double()[:, None]
    b = (count + 4) * U * mag
    return val, b + ROUND[dOut.dtype] * (val.abs() + b) + 1e-30


def within(got, ref, name=""):
    value, bound = ref
    assert got.shape == value.shape, f"{name}: {tuple(got.shape)} vs {tuple(value.shape)}"
    err = (got.double() - value).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{name}: {int(bad.sum())}/{bad.numel()} outside, worst {float((err / bound).nan_to_num(torch.inf).max()):.3g} "
                           f"of the bound at {tuple(int(x) for x in bad.nonzero()[0])}")
