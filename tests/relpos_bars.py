"""Bars on whole rows of the gradients of the relative-position-bias attention, from the 64-bit definition.

The elementwise bounds of relpos_ref add up what every pair may be off by, which on long segments is more
than the gradients themselves.  Roundings are independent, so here they add as a root of squares, row by row
(a token's head; an axis and head of the table), and the bars take what the kernels compute: Delta is the
exact row sum of P dP.  With u = 2^-8 (half a step of bf16) and D~ the Delta of the rounded out, off by at
most B = u sum_d |dO o|:

  P is off by at most  x = EXP P + P (1 - P) (e^(2 e) - 1),  e = 2^-24 (6 + axes) max_j |t|
      (EXP: exponentials and sums; e: the roundings of a row's scores, which a softmax that sums to 1 forgets
      where one key has all the weight)
  dS is off by  f = (x / P) |dS| + P sum_j (x / P) |dS| + P (EXP B + 2^-20 (|dO| |v| + |Delta|))
  dq: u |dq|, and over the keys    w = u |dS| + 2 u P B + f  times scale |k|
  dk: u |dk|, and over the queries w = u |dS| + f            times scale |q|
  dv: u |dv|, and over the queries w = u P + x               times |dO|
  dtable: u |dtable|, and over the pairs w = f + 2^-16 |dS|

The first part is a norm of its own; of the second, |w| <= its size has a deviation of at most size / sqrt(3),
so 4 times the root of the squares is seven deviations.
"""
import math

import torch

U, EXP = 2.0 ** -8, 2.0 ** -13


def pieces(off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v, dout, scale=None):
    """Per (segment, head) with pairs: the rows' ranges and the 64-bit t, P, dP, Delta, dS, buckets."""
    D = (bucket_of.numel() - 1) // 2
    Hq, Hkv, dim = q.shape[1], k.shape[1], q.shape[2]
    scale = scale or 1.0 / math.sqrt(dim)
    q, k, v, table, do = (x.double() for x in (q, k, v, table, dout))
    oq, ok = off_q.tolist(), off_k.tolist()
    for a0, a1, b0, b1 in zip(oq[:-1], oq[1:], ok[:-1], ok[1:]):
        if a1 <= a0 or b1 <= b0:
            continue
        gap = (pos_k[None, b0:b1].long() - pos_q[a0:a1, None].long()).clamp(-D, D) + D
        bucket = bucket_of.long()[gap]
        for h in range(Hq):
            g = h * Hkv // Hq
            t = q[a0:a1, h] @ k[b0:b1, g].T * scale
            for a in range(table.shape[0]):
                t = t + table[a, bucket[..., a], h]
            m = t.amax(1, keepdim=True)
            e = torch.exp(t - torch.where(m == -math.inf, 0.0, m))
            s = e.sum(1, keepdim=True)
            P = torch.where(s > 0, e / torch.where(s > 0, s, 1.0), 0.0)
            dP = do[a0:a1, h] @ v[b0:b1, g].T
            Delta = (P * dP).sum(1, keepdim=True)
            yield dict(rows=slice(a0, a1), keys=slice(b0, b1), h=h, g=g, t=t, P=P, dP=dP, Delta=Delta,
                       dS=P * (dP - Delta), bucket=bucket, q=q[a0:a1, h], k=k[b0:b1, g], v=v[b0:b1, g],
                       do=do[a0:a1, h], o=P @ v[b0:b1, g], scale=scale)


def table_sum(dS, bucket, n):
    return torch.zeros(n, dtype=dS.dtype, device=dS.device).index_add_(0, bucket.reshape(-1), dS.reshape(-1))


def gradients(off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v, dout, scale=None):
    """{name: (value, norm bar of each row)}: rows are the last axis, of the table the buckets."""
    val = {n: torch.zeros(x.shape, dtype=torch.float64, device=q.device)
           for n, x in (("dq", q), ("dk", k), ("dv", k))}
    val["dtable"] = torch.zeros(table.shape, dtype=torch.float64, device=q.device)
    var = {n: torch.zeros_like(x) for n, x in val.items()}
    NA, NB = table.shape[:2]
    for s in pieces(off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v, dout, scale):
        P, dS, at, to = s["P"], s["dS"], (s["rows"], s["h"]), (s["keys"], s["g"])
        size = torch.where(s["t"].isinf(), 0.0, s["t"].abs()).amax(1, keepdim=True)
        e = torch.expm1((2.0 ** -23 * (6 + NA) * size).clamp(max=1.0))
        x = EXP + (1 - P) * e  # of P
        B = U * (s["do"].abs() * s["o"].abs()).sum(1, keepdim=True)
        f = x * dS.abs() + P * (x * dS.abs()).sum(1, keepdim=True) + P * (
            EXP * B + 2.0 ** -20 * (s["do"].abs() @ s["v"].abs().T + s["Delta"].abs()))
        val["dq"][at] = dS @ s["k"] * s["scale"]
        var["dq"][at] = (U * dS.abs() + 2 * U * P * B + f).square() @ (s["k"] * s["scale"]).square()
        val["dk"][to] += dS.T @ s["q"] * s["scale"]
        var["dk"][to] += (U * dS.abs() + f).square().T @ (s["q"] * s["scale"]).square()
        val["dv"][to] += P.T @ s["do"]
        var["dv"][to] += ((U + x) * P).square().T @ s["do"].square()
        for a in range(NA):
            val["dtable"][a, :, s["h"]] += table_sum(dS, s["bucket"][..., a], NB)
            var["dtable"][a, :, s["h"]] += table_sum((f + 2.0 ** -16 * dS.abs()).square(), s["bucket"][..., a], NB)
    r = {}
    for n in val:
        y, w = (val[n], var[n]) if n != "dtable" else (val[n].transpose(1, 2), var[n].transpose(1, 2))
        r[n] = (y, U * y.norm(dim=-1) + 4 * w.sum(-1).sqrt() + 1e-30)
    return r


def worst(name, got, want):
    """The largest norm of a row's error over its bar."""
    value, bar = want
    got = got.double() if name != "dtable" else got.double().transpose(1, 2)
    return float(((got - value).norm(dim=-1) / bar).nan_to_num(math.inf).max()) if value.numel() else 0.0


def check(name, got, want):
    w = worst(name, got, want)
    assert w <= 1.0, f"{name}: a row is off by {w:.3g} of its bar"
