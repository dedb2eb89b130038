"""64-bit references of the transformer-layer operators (norm and rotary positions of heads, windowed attention, the
gated feed-forward product), each with an elementwise bound on the error of a kernel that computes in fp32 and rounds
where the dtype says.

Units of rounding: U = 2^-24 for an fp32 operation, `last` for the result's own rounding (2^-8 in bf16).  A sum of n
terms in any order is off by at most (n + 4) U times the sum of their magnitudes."""
import math

import torch

from dense_ref import ROUND, U, within  # noqa: F401

LOW = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}


def angles(rot, pos):
    """[T, 1, pairs] angles in 64 bits, and the bound on the kernel's: its stored frequency (two roundings in 64 bits, 2^-64
    turns), half turns in fp32 (U pi) and sincospi (2 ulp of at most 1)."""
    f = torch.tensor(rot.freqs, dtype=torch.float64, device=pos.device)
    which = torch.tensor([a for a, n in enumerate(rot.sections or [rot.dims // 2]) for _ in range(n)], device=pos.device, dtype=torch.long)
    p = pos.double().reshape(pos.shape[0], -1)[:, which]
    ang = (p * f)[:, None]
    return ang, (p.abs() * (f.abs() * 2.0 ** -51 + 2.0 ** -61))[:, None] + (math.pi + 4) * U


def turned(rot, x, xb, pos, back=False):
    """x [T, h, D] turned, and its bound from x's."""
    ang, ab = angles(rot, pos)
    c, s = torch.cos(ang), torch.sin(-ang if back else ang)
    R, h = rot.dims, rot.dims // 2
    a, b = (slice(0, R, 2), slice(1, R, 2)) if rot.interleaved else (slice(0, h), slice(h, R))
    y, yb = x.clone(), xb.clone()
    u, v = x[..., a], x[..., b]
    mag = u.abs() + v.abs()
    err = (ab + 3 * U) * (mag + xb[..., a] + xb[..., b])
    y[..., a], y[..., b] = u * c - v * s, u * s + v * c
    yb[..., a] = c.abs() * xb[..., a] + s.abs() * xb[..., b] + err
    yb[..., b] = s.abs() * xb[..., a] + c.abs() * xb[..., b] + err
    return y, yb


def rope_reference(rot, x, pos, w, eps):
    """{out, r: (value, bound)} of one side (queries or keys)."""
    D, last = x.shape[-1], ROUND[x.dtype]
    v = x.double()
    if eps is None:
        y, yb = v, torch.zeros_like(v)
        r = None
    else:
        ww = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
        r = ((v * v).mean(-1) + eps) ** -0.5
        rel = (D / 2 + 6) * U
        y = v * r[..., None] * ww
        yb = (rel + 3 * U) * y.abs()
    out, ob = turned(rot, y, yb, pos)
    ob = ob + last * (out.abs() + ob) + 1e-30
    return {"out": (out, ob), "r": None if r is None else (r, rel * r + 1e-30)}


def rope_bwd_reference(rot, x, pos, w, r, dout):
    """{dx, dw: (value, bound)} of one side, at the given r."""
    D, last = x.shape[-1], ROUND[x.dtype]
    d = dout.double()
    dn, dnb = turned(rot, d, torch.zeros_like(d), pos, back=True)
    if r is None:
        return {"dx": (dn, dnb + last * (dn.abs() + dnb) + 1e-30), "dw": None}
    rr = r.double()[..., None]
    xh = x.double() * rr
    ww = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
    g = dn * ww
    gb = dnb * ww.abs() + 2 * U * g.abs()
    s = (g * xh).mean(-1, keepdim=True)
    sb = (gb * xh.abs()).mean(-1, keepdim=True) + (D + 8) * U * (g * xh).abs().mean(-1, keepdim=True)
    dx = rr * (g - xh * s)
    dxb = rr * (gb + xh.abs() * sb + 5 * U * (g.abs() + (xh * s).abs()))
    dxb = dxb + last * (dx.abs() + dxb) + 1e-30
    res = {"dx": (dx, dxb), "dw": None}
    if w is not None:
        n = x.shape[0] * x.shape[1]
        dw = (dn * xh).sum((0, 1))
        dwb = (dnb * xh.abs()).sum((0, 1)) + (n + 8) * U * (dn * xh).abs().sum((0, 1))
        res["dw"] = (dw, dwb + ROUND[w.dtype] * (dw.abs() + dwb) + 1e-30)
    return res


def visible(n, causal, window, sinks, device="cuda"):
    """[n, n]: row i sees key j."""
    i = torch.arange(n, device=device)
    apart = i[:, None] - i[None]
    vis = (apart.abs() < (window or n)) | (i[None] < sinks)
    return vis & (apart >= 0) if causal else vis


def shared_offset(k, n, begin, causal, window, sinks, windowed):
    """[n, D]: the four of a query row's keys whose mean the bf16 dQ pass takes for an offset that all its keys share, in
    the columns where they are no farther apart than half of it (a little more, for the mean's own rounding); zero in the
    others."""
    i = torch.arange(n, device=k.device)
    end = i + 1 if causal else torch.full_like(i, n)
    w = window or n
    lo, hi, s = (i - w + 1).clamp(min=0), torch.minimum(end, i + w), end.clamp(max=sinks)
    apart = s < lo                      # the sinks lie before the window, else the two are one interval
    lo, hi = torch.where(apart, lo, 0), torch.where(apart, hi, torch.maximum(hi, s))
    # the rows of 32 packed rows that are of one sequence take theirs from what all of them see, if that is anything
    if windowed:
        g = torch.div(begin + i, 32, rounding_mode="floor") * 32 - begin
        l, h = lo[(g + 31).clamp(max=n - 1)], hi[g.clamp(min=0)]
        lo, hi = torch.where(l < h, l, lo), torch.where(l < h, h, hi)
    m = hi - lo
    m = torch.where(m < 8, m, 2 ** torch.floor(torch.log2(m.double())).long())
    at = torch.stack([lo + (m * (2 * x + 1) >> 3) for x in range(4)])
    at[3] = torch.where(apart & (s > 0), s >> 1, at[3])
    four = k[at]
    c = four.mean(0)
    return torch.where(four.amax(0) - four.amin(0) <= 0.52 * c.abs(), c, 0.0)


def window_reference(seq_ptr, Q, K, V, scale, causal, window, sinks, dOut=None, out_used=None):
    """{name: (value, bound)} of out, lse and, with dOut, dQ, dK, dV: each sequence and head by itself.  The gradients'
    bound takes the forward's rounded out (out_used), from which the kernels form Delta."""
    dt, R = Q.dtype, LOW[Q.dtype]
    last = ROUND[dt]
    T, H, D = Q.shape
    g = H // K.shape[1]
    q, k, v = (t.double() for t in (Q, K, V))
    z = torch.zeros_like
    out, out_b, lse, lse_b = z(q), z(q), z(q[..., 0]), z(q[..., 0])
    res = {"out": (out, out_b), "lse": (lse, lse_b)}
    if dOut is not None:
        do, ou = dOut.double(), out_used.double()
        dQ, dQb, dK, dKb, dV, dVb = z(q), z(q), z(k), z(k), z(v), z(v)
        res |= {"dQ": (dQ, dQb), "dK": (dK, dKb), "dV": (dV, dVb)}
    ptr = [int(x) for x in seq_ptr]
    # (a window that holds every sequence is none)
    windowed = bool(window) and max(window, sinks) < max(e - b for b, e in zip(ptr[:-1], ptr[1:]))
    for b, e in zip(ptr[:-1], ptr[1:]):
        n = e - b
        if n == 0:
            continue
        vis = visible(n, causal, window, sinks, Q.device)
        for h in range(H):
            qi, ki, vi = q[b:e, h], k[b:e, h // g], v[b:e, h // g]
            s = torch.where(vis, scale * (qi @ ki.T), -torch.inf)
            ls = torch.logsumexp(s, 1)
            p = torch.exp(s - ls[:, None])
            ds = (D + 4) * U * scale * (qi.abs() @ ki.abs().T) + 8 * U * (1 + ls.abs()[:, None])
            ds = torch.where(vis, ds, 0.0)
            top = ds.amax(1)
            o = p @ vi
            out[b:e, h], lse[b:e, h] = o, ls
            lse_b[b:e, h] = top + (n + 8) * U * (1 + ls.abs())
            rel = R + 2 * top + 2 * (n + 8) * U
            out_b[b:e, h] = rel[:, None] * (p @ vi.abs()) + last * o.abs() + 1e-30
            if dOut is None:
                continue
            doi, oi = do[b:e, h], ou[b:e, h]
            dp = doi @ vi.T
            delta = (doi * o).sum(1)
            d_delta = (doi.abs() * (oi - o).abs()).sum(1) + (D + 4) * U * (doi.abs() * oi.abs()).sum(1)
            pe = p * (ds + lse_b[b:e, h][:, None] + 8 * U * (1 + ls.abs()[:, None]))
            dsv = p * (dp - delta[:, None])
            dse = (R + 4 * U) * dsv.abs() + pe * (dp - delta[:, None]).abs() + \
                p * ((D + 4) * U * (doi.abs() @ vi.abs().T) + d_delta[:, None])
            sums = (n * g + 8) * U
            dQ[b:e, h] = scale * (dsv @ ki)
            dQb[b:e, h] = scale * (dse @ ki.abs() + sums * (dsv.abs() @ ki.abs()))
            if R:
                # dQ is formed as sum_j (dS_j + e_j) k_j - (sum_j e_j) c with |e_j| <= R |dS_j|: off by sum_j e_j (k_j - c),
                # not sum_j e_j k_j; c is a mean in bf16 (three roundings of at most 2^-8)
                c = shared_offset(ki, n, b, causal, window, sinks, windowed)
                far = (dsv.abs()[:, :, None] * ((ki[None] - c[:, None]).abs() - ki.abs()[None]).clamp(min=0)).sum(1)
                dQb[b:e, h] += scale * R * (far + 2.0 ** -6 * c.abs() * dsv.abs().sum(1)[:, None])
            dK[b:e, h // g] += scale * (dsv.T @ qi)
            dKb[b:e, h // g] += scale * (dse.T @ qi.abs() + sums * (dsv.abs().T @ qi.abs()))
            dV[b:e, h // g] += p.T @ doi
            dVb[b:e, h // g] += (R * p + pe + sums * p).T @ doi.abs()
    if dOut is not None:
        for x, xb in ((dQ, dQb), (dK, dKb), (dV, dVb)):
            xb += last * (x.abs() + xb) + 1e-30
    return res


def _act(g, act):
    """act(g), its derivative, the size of the derivative's terms, and the kernels' relative error of an evaluation (fp32
    exponential or erfc: a few units, and as many more as their argument is large)."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s)), s + (g * s * (1 - s)).abs(), (16 + 4 * g.abs()) * U
    if act == "gelu":
        p, f = 0.5 * torch.special.erfc(-g * math.sqrt(0.5)), g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        return g * p, p + f, p + f.abs(), (16 + 4 * g.abs() + 2 * g * g) * U
    on = (g > 0).double()
    return torch.relu(g), on, on, torch.zeros_like(g)


def _product(a, ab, b, bb, dt, n):
    """a b and its bound from the operands'.  A sum of n products on the tensor cores: every addition drops at most 2 U of
    what has been summed (bf16: in runs of 16384; fp32: in runs of 256, of products of parts that leave out 2 U), and the
    runs' fp32 sums."""
    run = 256 if dt == torch.float32 else 16384
    k = 2 * (min(n, run) + 8) + n / run + 4
    mag = a.abs() @ b.abs()
    return a @ b, k * U * mag + ab @ b.abs() + a.abs() @ bb + ab @ bb


def ff_reference(X, Wg, Wu, act):
    """{out, G, U: (value, bound)}."""
    dt, last = X.dtype, ROUND[X.dtype]
    x, wg, wu = X.double().reshape(-1, X.shape[-1]), Wg.double(), Wu.double()
    z = torch.zeros_like
    g, gb = _product(x, z(x), wg, z(wg), dt, x.shape[1])
    u, ub = _product(x, z(x), wu, z(wu), dt, x.shape[1])
    a, _, _, rel = _act(g, act)
    ab = 1.2 * gb + rel * a.abs() + 1e-37     # (|act'| < 1.13; 1e-37: results below the normal range)
    out = a * u
    ob = ab * (u.abs() + ub) + a.abs() * ub + 2 * U * out.abs()
    fin = lambda v, b: (v.reshape(*X.shape[:-1], -1), (b + last * (v.abs() + b) + 1e-37).reshape(*X.shape[:-1], -1))
    return {"out": fin(out, ob), "G": fin(g, gb), "U": fin(u, ub)}


def ff_bwd_reference(X, Wg, Wu, G, Up, dOut, act):
    """{dX, dWg, dWu: (value, bound)} at the given G and U."""
    dt, last, R = X.dtype, ROUND[X.dtype], LOW[X.dtype]
    flat = lambda t: t.double().reshape(-1, t.shape[-1])
    x, wg, wu, g, u, do = flat(X), Wg.double(), Wu.double(), flat(G), flat(Up), flat(dOut)
    z = torch.zeros_like
    a, slope, terms, rel = _act(g, act)
    dg, du = do * u * slope, do * a
    dgb = (do * u).abs() * (rel + 4 * U) * terms + (3 * U + R) * dg.abs() + 1e-37
    dub = do.abs() * rel * a.abs() + (3 * U + R) * du.abs() + 1e-37
    M = wg.shape[1]
    dx, dxb = _product(torch.cat([dg, du], 1), torch.cat([dgb, dub], 1), torch.cat([wg, wu], 1).T, z(torch.cat([wg, wu], 1).T), dt, 2 * M)
    n = x.shape[0]
    dwg, dwgb = _product(x.T, z(x.T), dg, dgb, dt, n)
    dwu, dwub = _product(x.T, z(x.T), du, dub, dt, n)
    fin = lambda v, b, s: (v.reshape(s), (b + last * (v.abs() + b) + 1e-37).reshape(s))
    return {"dX": fin(dx, dxb, X.shape), "dWg": fin(dwg, dwgb, Wg.shape), "dWu": fin(dwu, dwub, Wu.shape)}
