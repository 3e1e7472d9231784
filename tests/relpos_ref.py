"""The relative-position-bias attention and the layer norm from their definitions in 64 bits, with
the elementwise error bounds that the kernels' roundings allow.

Bounds (u = 2^-8, half a step of bf16).  The kernels hold scores, exponentials and sums in fp32: an
exponent's argument below 64 in size with a few roundings of 2^-24 each, and the 2^-22 of the
hardware exp2, leave P within 2^-13 relatively (EXP).  P and dS are rounded to bf16 as operands (u
each), results to bf16 (u).  With A = sum_j P |v|, and B = sum_d |dO| (u |o| + (u + 2 EXP) A), the error of the
Delta read off the saved out:
  out:    u |out| + (u + 2 EXP) A
  dv:     u |dv| + sum (u + EXP) P |dO|
  dS:     E = EXP P (|dP| + |Delta|) + P B;   dq, dk: u |.| + scale sum (u |dS| + 2 E) |k or q|
  dtable: u |.| + sum (E + 2^-16 |dS|)  (fp32 sums of at most a few thousand terms in a row)
"""
import math

import torch

U, EXP = 2.0 ** -8, 2.0 ** -13


def log_buckets(n_buckets, max_distance):
    """The definition of the logarithmic buckets in whole numbers."""
    half = n_buckets // 2
    e = max(1, half // 2)
    m = half - e

    def near(n):
        if n < e:
            return n
        b = 0
        while b + 1 < m and n ** m >= e ** (m - b - 1) * max_distance ** (b + 1):
            b += 1
        return min(half - 1, e + b)

    return [near(-x) if x <= 0 else half + near(x) for x in range(-max_distance, max_distance + 1)]


def _with_slop(v, bound):
    return v, bound + 1e-30


def attention(off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v, dout=None, scale=None):
    """{name: (value, bound)} in 64 bits of out and lse, and with dout of the gradients."""
    D = (bucket_of.numel() - 1) // 2
    Hq, Hkv, dim = q.shape[1], k.shape[1], q.shape[2]
    G, NA, NB = Hq // Hkv, table.shape[0], table.shape[1]
    scale = scale or 1.0 / math.sqrt(dim)
    f = lambda x: x.double()  # noqa: E731
    q, k, v, table = f(q), f(k), f(v), f(table)
    do = None if dout is None else f(dout)
    z = torch.zeros_like
    out, out_b, dq, dq_b = z(q), z(q), z(q), z(q)
    dk, dk_b, dv, dv_b = z(k), z(k), z(v), z(v)
    dt, dt_b = z(table), z(table)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    oq, ok = off_q.tolist(), off_k.tolist()
    for a0, a1, b0, b1 in zip(oq[:-1], oq[1:], ok[:-1], ok[1:]):
        if a1 <= a0 or b1 <= b0:
            continue
        delta = (pos_k[None, b0:b1].long() - pos_q[a0:a1, None].long()).clamp(-D, D) + D
        bucket = bucket_of.long()[delta]
        for h in range(Hq):
            kk, vv, qq = k[b0:b1, h // G], v[b0:b1, h // G], q[a0:a1, h]
            t = qq @ kk.T * scale
            for a in range(NA):
                t = t + table[a, bucket[..., a], h]
            m = t.amax(1, keepdim=True)
            e = torch.exp(t - torch.where(m == -math.inf, 0.0, m))
            e = torch.where(t == -math.inf, 0.0, e)
            s = e.sum(1, keepdim=True)
            P = torch.where(s > 0, e / torch.where(s > 0, s, 1.0), 0.0)
            o = P @ vv
            A = P @ vv.abs()
            out[a0:a1, h], out_b[a0:a1, h] = o, U * o.abs() + (U + 2 * EXP) * A
            lse[a0:a1, h] = (m + torch.log(s))[:, 0]
            if do is None:
                continue
            d = do[a0:a1, h]
            dP = d @ vv.T
            Delta = (P * dP).sum(1, keepdim=True)
            B = (d.abs() * (U * o.abs() + (U + 2 * EXP) * A)).sum(1, keepdim=True)
            dS = P * (dP - Delta)
            E = EXP * P * (d.abs() @ vv.abs().T + Delta.abs()) + P * B
            dv[b0:b1, h // G] += P.T @ d
            dv_b[b0:b1, h // G] += (U + EXP) * (P.T @ d.abs())
            W = U * dS.abs() + 2 * E
            dq[a0:a1, h], dq_b[a0:a1, h] = dS @ kk * scale, W @ kk.abs() * scale
            dk[b0:b1, h // G] += dS.T @ qq * scale
            dk_b[b0:b1, h // G] += W.T @ qq.abs() * scale
            for a in range(NA):
                i = bucket[..., a].reshape(-1)
                dt[a, :, h] += torch.zeros(NB, dtype=torch.float64, device=q.device).index_add_(0, i, dS.reshape(-1))
                dt_b[a, :, h] += torch.zeros(NB, dtype=torch.float64, device=q.device).index_add_(
                    0, i, (E + 2.0 ** -16 * dS.abs()).reshape(-1))
    # lse: the fp32 sums and roundings, with 2^-13 for the exponentials
    r = {"out": (out, out_b), "lse": (lse, EXP + 2.0 ** -20 * torch.where(lse.isfinite(), lse.abs(), 0.0))}
    if do is not None:
        for n, x, b in (("dq", dq, dq_b), ("dk", dk, dk_b), ("dv", dv, dv_b), ("dtable", dt, dt_b)):
            r[n] = (x, b + U * x.abs())
    return r


def layer_norm(x, gamma, beta, eps, dy=None, saved=None):
    """{name: (value, bound)} in 64 bits; saved = the (mean, rstd) the backward is given.
    Bounds: u_t |y| for the type's rounding (u_t = 2^-8 or 2^-24), and 2^-20 of the terms' sizes for
    fp32 arithmetic (sums of at most 2^17 terms kept as partial sums, each 2^-24 of its size)."""
    u = U if x.dtype == torch.bfloat16 else 2.0 ** -24
    S = 2.0 ** -20
    C = x.shape[-1]
    X = x.double().reshape(-1, C)
    g = torch.ones(C, dtype=torch.float64, device=x.device) if gamma is None else gamma.double()
    b = torch.zeros(C, dtype=torch.float64, device=x.device) if beta is None else beta.double()
    if saved is None:
        mean = X.mean(1)
        rstd = 1.0 / torch.sqrt((X - mean[:, None]).pow(2).mean(1) + eps)
        # the mean's own fp32 error moves xh by S |x| rstd
        size = (X.abs() + X.abs().mean(1, keepdim=True)) * rstd[:, None]
        y = (X - mean[:, None]) * rstd[:, None] * g + b
        return {"y": (y, u * y.abs() + S * (size * g.abs() * (1 + size) + b.abs())),
                "mean": (mean, S * X.abs().mean(1) + 1e-30),
                "rstd": (rstd, S * rstd * (1 + size.square().mean(1)) + 1e-30)}
    mean, rstd = saved[0].double()[:, None], saved[1].double()[:, None]
    d = dy.double().reshape(-1, C)
    xh = (X - mean) * rstd
    xs = (X.abs() + mean.abs()) * rstd  # what xh is computed from
    up = d * g
    dx = rstd * (up - up.mean(1, keepdim=True) - xh * (up * xh).mean(1, keepdim=True))
    size = rstd * (up.abs() + up.abs().mean(1, keepdim=True) + (xs + 1) * (up.abs() * (xs + 1)).mean(1, keepdim=True))
    dg, db = (d * xh).sum(0), d.sum(0)
    return {"dx": (dx, u * dx.abs() + S * size), "dgamma": (dg, u * dg.abs() + S * (d.abs() * (xs + 1)).sum(0) + 1e-30),
            "dbeta": (db, u * db.abs() + S * d.abs().sum(0) + 1e-30)}


def check(name, got, want):
    """got against (value, bound): equal infinities, and every value within its bound."""
    value, bound = want
    got = got.double().reshape(value.shape)
    inf = value.isinf()
    assert torch.equal(got[inf], value[inf]), f"{name}: infinities differ"
    off = torch.where(inf, 0.0, (got - torch.where(inf, 0.0, value)).abs())
    ok = off <= bound
    if not bool(ok.all()):
        worst = int(torch.where(inf, 0.0, off / bound.clamp(min=1e-300)).nan_to_num(math.inf).argmax())
        raise AssertionError(f"{name}: {int((~ok).sum())} of {ok.numel()} values out of bounds, worst at {worst}: "
                             f"{got.reshape(-1)[worst].item()!r} for {value.reshape(-1)[worst].item()!r}, "
                             f"bound {bound.expand_as(value).reshape(-1)[worst].item():.3e}")
