"""Plain fp64 forms of the attention-layer operators for the tests, written from the formulas,
each with the sums that bound a kernel's error.

A kernel that rounds its probabilities (and score gradients) to a format with unit roundoff u and
otherwise computes in fp32 (eps = 2^-24) makes, for one output o = sum_j p_j v_j, an error of at
most  u |o| (its own rounding) + (u + c eps) sum_j p_j |v_j|:  every p_j is off by a rounding
and by c eps, where c counts the roundings of a score (its dot product's absolute sum), of the
exponential and of the sums.  The same holds for the gradients with the absolute sums of their
terms; a score gradient ds = p (dp - delta) is off by its own rounding, p's error, and delta's,
which takes the rounded output.  u = 2^-8 for bf16 (8 significant bits: 1 + 2^-8 rounds to 1) and
2^-24 for fp32."""
import math

import torch

EPS = 2.0 ** -24
D = torch.float64


def visible(pos, keys, window, sinks):
    """[rows, keys] truth values: a query at position pos sees a key."""
    dist = pos[:, None] - keys[None]
    see = dist >= 0
    if window:
        see &= (dist < window) | (keys < sinks)[None]
    return see


def attention(q, k, v, pos, window=0, sinks=0, scale=None, dout=None, u=0.0):
    """One sequence: q [Lq, Hq, d] at positions pos, k, v [Lk, Hkv, d].  Returns a dict of values
    and, under "tol", their elementwise error bounds for a kernel of unit roundoff u."""
    q, k, v = q.to(D), k.to(D), v.to(D)
    Lq, hq, d = q.shape
    Lk, hkv, _ = k.shape
    g = hq // hkv
    scale = scale or 1 / math.sqrt(d)
    qh = q.transpose(0, 1)
    kh, vh = (x.transpose(0, 1).repeat_interleave(g, 0) for x in (k, v))
    see = visible(pos, torch.arange(Lk), window, sinks)[None]
    s = qh @ kh.transpose(1, 2) * scale
    size = qh.abs() @ kh.abs().transpose(1, 2) * scale  # of a score's terms
    s = torch.where(see, s, -math.inf)
    lse = torch.logsumexp(s, -1) if Lk else torch.full((hq, Lq), -math.inf, dtype=D)
    any_ = lse > -math.inf
    p = torch.where(see, torch.exp(s - torch.where(any_, lse, 0.0)[..., None]), 0.0)
    o = p @ vh
    c = 16.0 + math.sqrt(d) + 2 * (float(torch.where(see, size, 0.0).max()) if Lk * Lq else 0.0)
    r = {"out": o.transpose(0, 1), "lse": lse.transpose(0, 1)}
    up = u + c * EPS
    tol = {"out": (u * o.abs() + up * (p @ vh.abs())).transpose(0, 1) + 1e-30,
           "lse": c * EPS * (1 + torch.where(any_, lse.abs(), 0.0)).transpose(0, 1)}
    if dout is not None:
        do = dout.to(D).transpose(0, 1)
        delta = (do * o).sum(-1, keepdim=True)
        dp = do @ vh.transpose(1, 2)
        ds = p * (dp - delta) * scale
        # terms whose rounding reaches ds: its own, p's, dp's sum, delta's sum and the output in it
        mag = do.abs() @ vh.abs().transpose(1, 2) + (do.abs() * o.abs()).sum(-1, keepdim=True)
        e_ds = (u + c * EPS) * ds.abs() + (u + c * EPS) * scale * p * (do.abs() * (o.abs() + p @ vh.abs())).sum(-1, keepdim=True)
        e_ds = e_ds + c * EPS * scale * p * mag

        def group(x):
            return x.view(hkv, g, Lk, d).sum(1).transpose(0, 1)

        r.update(dq=(ds @ kh).transpose(0, 1), dk=group(ds.transpose(1, 2) @ qh), dv=group(p.transpose(1, 2) @ do))
        n = 1 + math.log2(max(2, Lq * g))  # sums over rows and heads
        tol.update(dq=u * r["dq"].abs() + ((e_ds + c * EPS * ds.abs()) @ kh.abs()).transpose(0, 1) + 1e-30,
                   dk=u * r["dk"].abs() + group((e_ds + n * c * EPS * ds.abs()).transpose(1, 2) @ qh.abs()) + 1e-30,
                   dv=u * r["dv"].abs() + group(((u + n * c * EPS) * p).transpose(1, 2) @ do.abs()) + 1e-30)
    r["tol"] = tol
    return r


def packed(q, k, v, cu_q, cu_k, window=0, sinks=0, scale=None, dout=None, u=0.0):
    """attention() of every sequence, its outputs packed again."""
    parts = []
    for n in range(len(cu_q) - 1):
        a, b, c, e = cu_q[n], cu_q[n + 1], cu_k[n], cu_k[n + 1]
        pos = torch.arange(b - a) + (e - c) - (b - a)
        parts.append(attention(q[a:b], k[c:e], v[c:e], pos, window, sinks, scale,
                               None if dout is None else dout[a:b], u))
    names = [n for n in parts[0] if n != "tol"]
    r = {n: torch.cat([x[n] for x in parts]) for n in names}
    r["tol"] = {n: torch.cat([x["tol"][n] for x in parts]) for n in names}
    return r


def worst(got, ref, tol):
    """The largest error in units of its bound (0 where both are the same infinity)."""
    got = got.detach().cpu().to(D)
    same = torch.where(ref.isinf(), got == ref, got.isfinite())
    if not bool(same.all()):
        return math.inf
    err = torch.where(ref.isinf(), 0.0, (got - ref).abs())
    return float((err / tol).max()) if err.numel() else 0.0


def norm_rope(x, w, norm, eps, cos=None, sin=None, pos=None, layout="half", dy=None):
    """y, and with dy also dx and dw, in 64 bits, and the absolute sums of their terms."""
    x = x.to(D)
    T, H, d = x.shape
    ws = torch.ones(d, dtype=D) if w is None else w.to(D)
    cn = {"none": 0.0, "rms": 1.0 / d, "l2": 1.0}[norm]
    r = torch.ones(T, H, 1, dtype=D) if norm == "none" else \
        ((x * x).sum(-1, keepdim=True) * (1.0 / d if norm == "rms" else 1.0) + eps) ** -0.5
    # the rotation as one d x d matrix per token: y = M z
    M = torch.eye(d, dtype=D).repeat(T, 1, 1)
    if cos is not None:
        half = cos.shape[1]
        for i in range(half):
            a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
            c, s = cos.to(D)[pos.long(), i], sin.to(D)[pos.long(), i]
            M[:, a, a], M[:, a, b], M[:, b, a], M[:, b, b] = c, -s, s, c
    z = x * r * ws
    res = {"y": torch.einsum("tij,thj->thi", M, z), "y_abs": torch.einsum("tij,thj->thi", M.abs(), z.abs())}
    if dy is not None:
        dy = dy.to(D)
        g = torch.einsum("tji,thj->thi", M, dy)
        ga = torch.einsum("tji,thj->thi", M.abs(), dy.abs())
        gw = g * ws
        res["dx"] = r * gw - cn * r ** 3 * (x * gw).sum(-1, keepdim=True) * x
        res["dx_abs"] = r * ga * ws.abs() + cn * r ** 3 * (x.abs() * ga * ws.abs()).sum(-1, keepdim=True) * x.abs()
        res["dw"], res["dw_abs"] = (g * x * r).sum((0, 1)), (ga * x.abs() * r).sum((0, 1))
    return res
