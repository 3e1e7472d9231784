"""The operators measured here: attention with a learned relative position bias by buckets
(forward, and a training step with the gradients of q, k, v and the bias table) and layer norm
(forward, and backward with the reduction of the weights' gradients).

`listed()` gives the cases, `draw()` more of the same ranges, `prepare()` the inputs, `run()` one
pass (the plain form in elementary torch operations, or the framework's own calls where `own`
is true), `work()` the bytes and operations a pass cannot do without, `exact()` the same outputs
from the definitions in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
LN_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # layer norm: the per-head query rows of the dense stage (20480 tokens x 32 heads of 32)
        dict(name="ln_fwd_head_rows", op="ln_fwd", rows=655360, width=32, dtype="bf16"),
        # the hidden rows (width 1024) of every token of the sparse stage
        dict(name="ln_fwd_hidden", op="ln_fwd", rows=121344, width=1024, dtype="bf16"),
        # one frame's tokens at an odd width in fp32: a small call, where latency counts
        dict(name="ln_fwd_frame_odd", op="ln_fwd", rows=1370, width=509, dtype="f32"),
        # the backward of the head rows: hundreds of thousands of rows reduced into 32 weights
        dict(name="ln_bwd_head_rows", op="ln_bwd", rows=655360, width=32, dtype="bf16"),
        # the backward of the sparse stage's hidden rows
        dict(name="ln_bwd_hidden", op="ln_bwd", rows=121344, width=1024, dtype="bf16"),
        # attention: the 1024-token scene, one segment, tokens placed by their order
        dict(name="attn_fwd_tiny", op="attn_fwd", segs=1, q_len=1024, k_len=1024, ragged=False, heads=32, kv_heads=2,
             dim=32, axes=1, buckets=32, max_distance=128, places="order"),
        # the dense stage's 4096 volume tokens in 64-token bricks, placed by their three voxel coordinates
        dict(name="attn_fwd_volume", op="attn_fwd", segs=1, q_len=4096, k_len=4096, ragged=False, heads=32, kv_heads=2,
             dim=32, axes=3, buckets=32, max_distance=16, places="bricks"),
        # every frame attends itself: eight frames of 37 x 37 patches and a camera token, 16 heads of 64
        dict(name="attn_fwd_frames", op="attn_fwd", segs=8, q_len=1370, k_len=1370, ragged=False, heads=16, kv_heads=16,
             dim=64, axes=2, buckets=32, max_distance=36, places="patches"),
        # one new token of 64 streams, each against its own long past of up to 8192 tokens
        dict(name="attn_fwd_one_token", op="attn_fwd", segs=64, q_len=1, k_len=8192, ragged=True, heads=32, kv_heads=2,
             dim=32, axes=1, buckets=32, max_distance=128, places="order"),
        # a training step on small ragged blocks of up to 64 tokens (bricks cut by a surface)
        dict(name="attn_train_blocks", op="attn_train", segs=256, q_len=64, k_len=64, ragged=True, heads=32, kv_heads=2,
             dim=32, axes=3, buckets=16, max_distance=16, places="bricks"),
        # a training step on the dense stage's 4096 volume tokens
        dict(name="attn_train_volume", op="attn_train", segs=1, q_len=4096, k_len=4096, ragged=False, heads=32,
             kv_heads=2, dim=32, axes=1, buckets=32, max_distance=128, places="order"),
        # a training step on six frames' own attention
        dict(name="attn_train_frames", op="attn_train", segs=6, q_len=1370, k_len=1370, ragged=False, heads=16,
             kv_heads=16, dim=64, axes=2, buckets=32, max_distance=36, places="patches"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "attn_fwd", "attn_fwd", "attn_train"])
    if op in ("ln_fwd", "ln_bwd"):
        # rows from one to all of the sparse stage's, widths from one head to wide hidden rows, odd ones among them
        width = _log(rng, 17, 4096)
        if rng.random() < 0.6:
            width = max(32, width // 32 * 32)
        rows = _log(rng, 1, max(1, 100_000_000 // width))
        return dict(op=op, rows=min(rows, 1_000_000), width=width, dtype=rng.choice(["bf16", "bf16", "f32"]))
    dim = rng.choice([32, 64])
    heads, kv_heads = rng.choice([(32, 2), (16, 16), (8, 2), (6, 2), (4, 1), (1, 1)])
    axes = rng.choice([1, 2, 3])
    shape = rng.choice(["one", "few", "square"]) if op == "attn_fwd" else "square"
    if shape == "one":
        segs, q_len, k_len = _log(rng, 1, 64), 1, _log(rng, 1, 8192)
    elif shape == "few":
        segs, q_len, k_len = _log(rng, 1, 16), _log(rng, 2, 40), _log(rng, 1, 4096)
    else:
        # one key alone has weight 1 whatever its score: all gradients of scores are 0, nothing to compare
        q_len = _log(rng, 2 if op == "attn_train" else 1, 2048)
        k_len = q_len if op == "attn_train" or rng.random() < 0.7 else _log(rng, 1, 2048)
        segs = _log(rng, 1, max(1, min(300, (3 << 20) // (q_len * k_len))))
    places = rng.choice(["order", "scattered"]) if axes == 1 else rng.choice(["scattered", "bricks"]) if axes == 3 else \
        rng.choice(["scattered", "patches"])
    return dict(op=op, segs=segs, q_len=q_len, k_len=k_len, ragged=rng.random() < 0.6, heads=heads, kv_heads=kv_heads,
                dim=dim, axes=axes, buckets=rng.choice([8, 16, 32, 64]), max_distance=_log(rng, 32, 500), places=places)


# ---- inputs --------------------------------------------------------------------------------------

def _lengths(case, which):
    """Segment lengths, which belong to the case: ragged ones spread over 0..len, the first whole."""
    segs, most = case["segs"], case[which]
    if not case["ragged"] or most == 1:
        return torch.full((segs,), most, dtype=torch.int64)
    lens = torch.randint(0, most + 1, (segs,), generator=torch.Generator().manual_seed(segs * 100003 + most))
    lens[0] = most
    return lens


def _both_lengths(case):
    lq = _lengths(case, "q_len")
    return lq, lq if case["q_len"] == case["k_len"] else _lengths(case, "k_len")


def _places(case, lens, gen):
    """Integer positions [tokens][axes] of the tokens, segment by segment."""
    n, axes, how = int(lens.sum()), case["axes"], case["places"]
    within = torch.arange(n) - torch.repeat_interleave(torch.cumsum(lens, 0) - lens, lens)
    if how == "order":  # the token's number in its segment
        return within[:, None].expand(n, axes).contiguous().int()
    if how == "bricks":  # 4 x 4 x 4 bricks of a 16-wide grid, repeated behind each other on the first axis
        brick, t = within // 64, within % 64
        x = [brick // 16 * 4 + t // 16, brick // 4 % 4 * 4 + t // 4 % 4, brick % 4 * 4 + t % 4]
        return torch.stack(x, 1).int()
    if how == "patches":  # a camera token, then the patches of a 37-wide frame by row and column
        p = (within - 1).clamp(min=0)
        return torch.stack([p // 37, p % 37], 1).int()
    return torch.randint(-300, 301, (n, axes), generator=gen).int()


def log_buckets(n_buckets, max_distance):
    """Bucket of every clamped distance -D..D: half the buckets a direction (keys behind the query
    first), the near half of these one distance each, the others spaced by the logarithm up to D.
    The comparison n^m >= e^(m-b) D^b is floor(m log(n/e) / log(D/e)) in whole numbers."""
    half = n_buckets // 2
    e = max(1, half // 2)
    m = half - e
    far, b = [], 0
    for n in range(max_distance + 1):
        if n < e:
            far.append(n)
            continue
        while b + 1 < m and n ** m >= e ** (m - b - 1) * max_distance ** (b + 1):
            b += 1
        far.append(min(e + b, half - 1))
    return [far[-x] if x <= 0 else half + far[x] for x in range(-max_distance, max_distance + 1)]


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEVICE).manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=gen, device=DEVICE) * std).to(dtype)

    state = dict(case)
    if case["op"] in ("ln_fwd", "ln_bwd"):
        t = LN_TYPES[case["dtype"]]
        rows, width = case["rows"], case["width"]
        # rows of a residual stream: their own mean and spread, weights around one
        state["x"] = normal(rows, width, dtype=t, std=1.5).add_(normal(rows, 1, dtype=t, std=0.5))
        state["gamma"] = (1.0 + normal(width, dtype=torch.float32, std=0.2)).to(t)
        state["beta"] = normal(width, dtype=t, std=0.2)
        if case["op"] == "ln_bwd":
            # what the forward pass kept
            x = state["x"].double()
            mean = x.mean(1)
            state["mean"] = mean.float()
            state["rstd"] = ((x - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
            state["dy"] = normal(rows, width, dtype=t)
        return state
    lq, lk = _both_lengths(case)
    same = case["q_len"] == case["k_len"]
    nq, nk, dim = int(lq.sum()), int(lk.sum()), case["dim"]
    pk = _places(case, lk, host)
    pq = pk if same else _places(case, lq, host)
    if case["places"] == "order" and not same:
        # the queries are the last tokens of their segments' past
        pq = pq + torch.repeat_interleave((lk - lq), lq)[:, None].int()

    def table_of(lens):
        return torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(lens, 0)]).int().to(DEVICE)

    state["off_k"] = table_of(lk)
    state["off_q"] = state["off_k"] if same else table_of(lq)
    state["pos_k"] = pk.to(DEVICE)
    state["pos_q"] = state["pos_k"] if same else pq.to(DEVICE)
    state["bucket_of"] = torch.tensor(log_buckets(case["buckets"], case["max_distance"]), dtype=torch.int32, device=DEVICE)
    state["table"] = normal(case["axes"], case["buckets"], case["heads"], std=0.5)
    state["q"] = normal(nq, case["heads"], dim)
    state["k"] = normal(nk, case["kv_heads"], dim)
    state["v"] = normal(nk, case["kv_heads"], dim)
    if case["op"] == "attn_train":
        state["dout"] = normal(nq, case["heads"], dim)
    return state


# ---- the plain forms -----------------------------------------------------------------------------

def _ln_forward(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    centred = x - mean
    rstd = torch.rsqrt((centred * centred).mean(1, keepdim=True) + EPS)
    y = centred * rstd * s["gamma"].float() + s["beta"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _ln_backward(s):
    t = s["x"].dtype
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["gamma"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    dgamma = (dy * xh).sum(0, dtype=torch.float64)
    dbeta = dy.sum(0, dtype=torch.float64)
    return {"dx": dx.to(t), "dgamma": dgamma.to(t), "dbeta": dbeta.to(t)}


def _padded(off, most):
    """Token numbers [segment][most] and which of them are there."""
    at = off[:-1, None].long() + torch.arange(most, device=off.device)
    there = at < off[1:, None]
    return torch.where(there, at, torch.zeros_like(at)), there


def _rows(x, at, there):
    """[segment][heads][most][dim] in 32 bits, zeros where there is no token."""
    return torch.where(there[..., None, None], x[at].float(), 0.0).transpose(1, 2)


def _attn(s, train):
    """All segments padded to the longest, as one batch."""
    dim, heads, kv_heads, top = s["dim"], s["heads"], s["kv_heads"], s["max_distance"]
    share, scale = heads // kv_heads, 1.0 / math.sqrt(dim)
    aq, tq = _padded(s["off_q"], s["q_len"])
    ak, tk = _padded(s["off_k"], s["k_len"])
    q, k, v = _rows(s["q"], aq, tq), _rows(s["k"], ak, tk), _rows(s["v"], ak, tk)
    k, v = k.repeat_interleave(share, 1), v.repeat_interleave(share, 1)
    delta = (s["pos_k"][ak][:, None, :, :] - s["pos_q"][aq][:, :, None, :]).clamp(-top, top) + top
    bucket = s["bucket_of"][delta.long()].long()  # [segment][q][k][axes]
    table = s["table"].float()
    bias = sum(table[a][bucket[..., a]] for a in range(s["axes"])).permute(0, 3, 1, 2)
    t = torch.matmul(q, k.transpose(2, 3)) * scale + bias
    t = torch.where(tk[:, None, None, :], t, -math.inf)
    top_t = t.amax(3, keepdim=True)
    e = torch.exp(t - torch.where(top_t == -math.inf, 0.0, top_t))
    total = e.sum(3, keepdim=True)
    p = torch.where(total > 0, e / total, 0.0)
    o = torch.matmul(p, v)
    lse = (top_t + torch.log(total))[..., 0]
    out = {"out": o.transpose(1, 2)[tq].to(torch.bfloat16), "lse": lse.transpose(1, 2)[tq]}
    if not train:
        return out
    do = _rows(s["dout"], aq, tq)
    dv = torch.matmul(p.transpose(2, 3), do)
    dp = torch.matmul(do, v.transpose(2, 3))
    ds = p * (dp - (p * dp).sum(3, keepdim=True))
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(2, 3), q) * scale

    def shared(x):  # the heads that share a key head, summed
        return x.view(x.shape[0], kv_heads, share, *x.shape[2:]).sum(2).transpose(1, 2)[tk].to(torch.bfloat16)

    ds = torch.where(tq[:, None, :, None], ds, 0.0)
    ids = torch.arange(s["buckets"], device=q.device)
    by_row = ds.permute(0, 2, 1, 3).reshape(-1, heads, ds.shape[3])  # [segment and q][heads][k]
    dtable = [torch.matmul(by_row, (bucket[..., a, None] == ids).float().reshape(-1, ds.shape[3], len(ids)))
              .sum(0, dtype=torch.float64).t() for a in range(s["axes"])]
    return {**out, "dq": dq.transpose(1, 2)[tq].to(torch.bfloat16), "dk": shared(dk), "dv": shared(dv),
            "dtable": torch.stack(dtable).to(torch.bfloat16)}


# ---- the framework's calls -----------------------------------------------------------------------

def _own_ln(s):
    from block_sparse_gqa_nsa_b200 import nsa

    x = s["x"]
    if s["op"] == "ln_fwd":
        y = torch.empty_like(x)
        mean, rstd = torch.empty(2, x.shape[0], dtype=torch.float32, device=x.device).unbind(0)
        nsa.lsrm_layer_norm_forward(x, s["gamma"], s["beta"], EPS, y, mean, rstd)
        return {"y": y, "mean": mean, "rstd": rstd}
    if "ws" not in s:
        s["ws"] = nsa.layer_norm_workspace(x.shape[0], x.shape[1], x.device)
    dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(s["gamma"]), torch.empty_like(s["gamma"])
    nsa.lsrm_layer_norm_backward(s["dy"], x, s["gamma"], s["mean"], s["rstd"], dx, dgamma, dbeta, s["ws"])
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def _own_attn(s):
    from block_sparse_gqa_nsa_b200 import nsa

    q, k, v = s["q"], s["k"], s["v"]
    if "desc" not in s:  # the descriptor and workspace that a program keeps
        s["desc"] = nsa.make_relpos_desc(q.shape[0], k.shape[0], s["segs"], s["heads"], s["kv_heads"], s["dim"],
                                         s["axes"], s["buckets"], s["max_distance"])
        s["ws"] = nsa.relpos_workspace(s["desc"], q.device)
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    where = (s["desc"], s["off_q"], s["off_k"], s["pos_q"], s["pos_k"], s["bucket_of"], s["table"])
    nsa.lsrm_relpos_forward(*where, q, k, v, out, lse, s["ws"])
    if s["op"] == "attn_fwd":
        return {"out": out, "lse": lse}
    dq, dk, dv, dtable = (torch.empty_like(x) for x in (q, k, v, s["table"]))
    nsa.lsrm_relpos_backward(*where, q, k, v, out, lse, s["dout"], dq, dk, dv, dtable, s["ws"])
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv, "dtable": dtable}


def run(state):
    if own:
        return _own_ln(state) if state["op"] in ("ln_fwd", "ln_bwd") else _own_attn(state)
    if state["op"] == "ln_fwd":
        return _ln_forward(state)
    if state["op"] == "ln_bwd":
        return _ln_backward(state)
    return _attn(state, state["op"] == "attn_train")


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    if case["op"] in ("ln_fwd", "ln_bwd"):
        rows, width = case["rows"], case["width"]
        size = 2 if case["dtype"] == "bf16" else 4
        back = case["op"] == "ln_bwd"
        return {"bytes": rows * width * size * (3 if back else 2) + rows * 8 + width * size * (3 if back else 2),
                "flops": rows * width * (13 if back else 8)}
    lens_q, lens_k = _both_lengths(case)
    nq, nk, pairs = int(lens_q.sum()), int(lens_k.sum()), int((lens_q * lens_k).sum())
    rows_q, rows_k = nq * case["heads"] * case["dim"] * 2, nk * case["kv_heads"] * case["dim"] * 2
    small = (nq + (nk if case["q_len"] != case["k_len"] else 0)) * case["axes"] * 4 + nq * case["heads"] * 4
    train = case["op"] == "attn_train"
    return {"bytes": (4 if train else 2) * rows_q + (4 if train else 2) * rows_k + small,
            "flops": pairs * case["heads"] * case["dim"] * (14 if train else 4)}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def _exact_ln(case, s):
    x = s["x"].double()
    n = x.shape[1]
    gamma, beta = s["gamma"].double(), s["beta"].double()
    if case["op"] == "ln_fwd":
        mean = x.sum(1) / n
        var = (x - mean[:, None]).pow(2).sum(1) / n
        rstd = 1.0 / torch.sqrt(var + EPS)
        return {"y": (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None] * gamma + beta, "mean": mean, "rstd": rstd}
    # the Jacobian of one row applied to dy * gamma
    mean, rstd, dy = s["mean"].double(), s["rstd"].double(), s["dy"].double()
    xh = (x - mean[:, None]) * rstd[:, None]
    up = dy * gamma
    inner = (up * xh).sum(1)
    dx = (up - up.sum(1)[:, None] / n - xh * (inner / n)[:, None]) * rstd[:, None]
    return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", dy, xh), "dbeta": torch.einsum("rc->c", dy)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("ln_fwd", "ln_bwd"):
        return _exact_ln(case, s)
    # segment by segment and key head by key head, with the bias looked up pair by pair
    train = case["op"] == "attn_train"
    share, top = case["heads"] // case["kv_heads"], case["max_distance"]
    f64 = torch.float64
    q, k, v, table = s["q"].double(), s["k"].double(), s["v"].double(), s["table"].double()
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=f64, device=q.device)
    dq, dk, dv, dtable = (torch.zeros_like(x) for x in (q, k, v, table))
    do = s["dout"].double() if train else None
    oq, ok = s["off_q"].tolist(), s["off_k"].tolist()
    for a0, a1, b0, b1 in zip(oq[:-1], oq[1:], ok[:-1], ok[1:]):
        if a1 == a0 or b1 == b0:
            continue
        gap = s["pos_k"][None, b0:b1].long() - s["pos_q"][a0:a1, None].long()
        bucket = s["bucket_of"].long()[torch.clamp(gap, min=-top, max=top) + top]
        for h in range(case["heads"]):
            g = h // share
            t = (q[a0:a1, h] @ k[b0:b1, g].T) / math.sqrt(case["dim"])
            for a in range(case["axes"]):
                t = t + table[a, :, h][bucket[..., a]]
            z = torch.logsumexp(t, 1)
            p = torch.exp(t - z[:, None])
            out[a0:a1, h], lse[a0:a1, h] = p @ v[b0:b1, g], z
            if not train:
                continue
            d = do[a0:a1, h]
            dv[b0:b1, g] += p.T @ d
            dp = d @ v[b0:b1, g].T
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            dq[a0:a1, h] = ds @ k[b0:b1, g] / math.sqrt(case["dim"])
            dk[b0:b1, g] += ds.T @ q[a0:a1, h] / math.sqrt(case["dim"])
            for a in range(case["axes"]):
                dtable[a, :, h] += torch.bincount(bucket[..., a].reshape(-1), ds.reshape(-1), case["buckets"])
    if not train:
        return {"out": out, "lse": lse}
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv, "dtable": dtable}
