"""The relative-position-bias attention on the GPU against its definition in 64 bits: forward, single
tokens against a long past, the gradients of q, k, v and the table, ragged and empty segments, masks
by the table, rows outside every segment, captured graphs and other streams."""
import math

import pytest
import torch

from block_sparse_gqa_nsa_b200 import nsa
import relpos_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Case:
    def __init__(self, lens_q, lens_k=None, heads=4, kv_heads=2, dim=32, axes=1, buckets=32, maxd=128, places="order",
                 scale=0.0, lead=0, seed=0, spread=1.0):
        """lead: tokens before the first and behind the last segment, which belong to none."""
        g = torch.Generator().manual_seed(seed)
        self.same = lens_k is None
        lens_k = lens_q if self.same else lens_k
        self.scale, self.lead = scale, lead
        self.lens = (lens_q, lens_k)

        def off(lens):
            o = [lead]
            for n in lens:
                o.append(o[-1] + n)
            return torch.tensor(o, dtype=torch.int32, device="cuda"), o[-1] + lead

        self.off_q, nq = off(lens_q)
        self.off_k, nk = off(lens_k)

        def pos(n):
            if places == "order":
                return torch.arange(n)[:, None].expand(n, axes).contiguous().int()
            if places == "far":  # the ends of the allowed range
                return (torch.randint(0, 3, (n, axes), generator=g) - 1).int() * 2 ** 29
            if places == "bricks":  # 4 x 4 x 4 tokens, the last axis the fastest
                i = torch.arange(n)
                return torch.stack([i // 16, i // 4 % 4 + i // 64, i % 4 + i // 64 % 3], 1)[:, 3 - axes:].int().contiguous()
            if places == "frames":  # long runs on one position
                return (torch.arange(n) // 40)[:, None].expand(n, axes).contiguous().int()
            return torch.randint(-2 * maxd, 2 * maxd + 1, (n, axes), generator=g).int()

        self.pos_k = pos(nk).cuda()
        self.pos_q = self.pos_k if self.same else pos(nq).cuda()
        self.bucket_of = (nsa.lsrm_relpos_log_buckets(buckets, maxd).cuda() if buckets % 2 == 0 else
                          torch.randint(0, buckets, (2 * maxd + 1,), generator=g).int().cuda())

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=g) * std).to(BF).cuda()

        self.table = normal(axes, buckets, heads)
        self.q, self.k, self.v = normal(nq, heads, dim, std=spread), normal(nk, kv_heads, dim), normal(nk, kv_heads, dim)
        self.dout = normal(nq, heads, dim)
        self.desc = nsa.make_relpos_desc(nq, nk, len(lens_q), heads, kv_heads, dim, axes, buckets, maxd, scale)
        self.ws = nsa.relpos_workspace(self.desc)

    @property
    def where(self):
        return (self.off_q, self.off_k, self.pos_q, self.pos_k, self.bucket_of, self.table)

    def forward(self, out=None, lse=None, ws=None):
        out = torch.full_like(self.q, float("nan")) if out is None else out
        lse = torch.full(self.q.shape[:2], float("nan"), device="cuda") if lse is None else lse
        nsa.lsrm_relpos_forward(self.desc, *self.where, self.q, self.k, self.v, out, lse, self.ws if ws is None else ws)
        return {"out": out, "lse": lse}

    def backward(self, f, into=None):
        r = into or {n: torch.full_like(x, float("nan")) for n, x in
                     (("dq", self.q), ("dk", self.k), ("dv", self.v), ("dtable", self.table))}
        nsa.lsrm_relpos_backward(self.desc, *self.where, self.q, self.k, self.v, f["out"], f["lse"], self.dout,
                                 r["dq"], r["dk"], r["dv"], r["dtable"], self.ws)
        return r

    def reference(self, train):
        return ref.attention(*self.where, self.q, self.k, self.v, self.dout if train else None, self.scale or None)

    def check(self, train=True, status=0):
        f = self.forward()
        got = {**f, **(self.backward(f) if train else {})}
        assert nsa.lsrm_nsa_last_device_status(self.ws) == status
        want = self.reference(train)
        for n, x in got.items():
            # rows outside the segments are not the call's
            rows = slice(self.lead, x.shape[0] - self.lead) if n != "dtable" else slice(None)
            ref.check(n, x[rows], (want[n][0][rows], want[n][1][rows]))
        return got, want


FORWARD = {
    "one": dict(lens_q=[1]),
    "two_keys": dict(lens_q=[2, 1, 2]),
    "tile_edges": dict(lens_q=[31, 32, 33, 63, 64, 65, 127, 128, 129]),
    "empty_first_last": dict(lens_q=[0, 5, 0, 0, 70, 0]),
    "gqa16": dict(lens_q=[200, 77], heads=32, kv_heads=2),
    "mha64": dict(lens_q=[130, 250], heads=4, kv_heads=4, dim=64),
    "odd_group": dict(lens_q=[90, 3, 41], heads=6, kv_heads=2, dim=64, axes=2, places="scattered"),
    "axes3": dict(lens_q=[300], axes=3, places="scattered", maxd=20, buckets=16),
    "axes3_d64": dict(lens_q=[150, 64], axes=3, places="scattered", maxd=7, buckets=7, dim=64),
    "frames": dict(lens_q=[400], places="frames", maxd=5, buckets=8),
    "far": dict(lens_q=[200], axes=2, places="far", maxd=1023, buckets=64),
    "near": dict(lens_q=[333], maxd=1, buckets=2),
    "widest_table": dict(lens_q=[140], axes=3, maxd=1023, buckets=64, dim=64, places="scattered"),
    "one_bucket": dict(lens_q=[100], buckets=1),
    "scale": dict(lens_q=[100], scale=0.7, spread=3.0),
    "long": dict(lens_q=[2500], heads=2, kv_heads=1),
    "cross": dict(lens_q=[50, 0, 7, 300], lens_k=[300, 20, 0, 9], places="scattered"),
    "no_keys_at_all": dict(lens_q=[40, 40], lens_k=[0, 0]),
    "no_queries_at_all": dict(lens_q=[0, 0], lens_k=[40, 40]),
    "outside": dict(lens_q=[70, 5], lead=9),
    # many short segments: several heads a CTA
    "short_ragged": dict(lens_q=[i * 7 % 65 for i in range(60)], heads=8, kv_heads=2, axes=3, places="scattered", maxd=9),
    "short_gqa16": dict(lens_q=[64, 1, 17, 0, 33] * 8, heads=32, kv_heads=2, buckets=16, maxd=20),
    "short_d64": dict(lens_q=[i * 5 % 61 for i in range(50)], heads=6, kv_heads=2, dim=64, axes=2, places="scattered"),
    "short_mha": dict(lens_q=[40, 16, 15, 3] * 20, heads=1, kv_heads=1),
    "short_wide_group": dict(lens_q=[30, 64, 5] * 15, heads=40, kv_heads=2, maxd=31, places="frames"),
    "short_with_long": dict(lens_q=[20, 0, 150, 9, 64] * 10, lens_k=[64, 7, 0, 200, 1] * 10, heads=8, kv_heads=2,
                            places="scattered"),
    "short_outside": dict(lens_q=[33, 12, 60] * 14, lead=5, heads=4, kv_heads=2, axes=3, places="scattered", maxd=7,
                          buckets=7),
    # long segments: 128-row tiles in the backward
    "long32": dict(lens_q=[300]),
    "long64": dict(lens_q=[300, 555], dim=64),
    "long_gqa16": dict(lens_q=[520, 300], heads=32, kv_heads=2),
    "long_ragged": dict(lens_q=[600, 0, 1, 700, 65, 640, 129], heads=2, kv_heads=2, places="scattered", axes=2),
    "long_cross": dict(lens_q=[400, 0, 300], lens_k=[300, 400, 500], dim=64, heads=6, kv_heads=2),
    "long_outside": dict(lens_q=[300, 400], lead=9, dim=64, axes=2, places="scattered", buckets=64, maxd=200),
    "long_axes3": dict(lens_q=[450], dim=64, axes=3, places="scattered", maxd=30, buckets=16),
    "long_frames": dict(lens_q=[640], dim=64, axes=2, places="frames", maxd=7, buckets=8),
    "long_widest": dict(lens_q=[330], axes=3, maxd=1023, buckets=64, dim=64, places="scattered"),
    "long_odd_buckets": dict(lens_q=[400, 300], axes=3, buckets=7, maxd=9, places="scattered"),
    "middle64": dict(lens_q=[200, 192, 130, 7], dim=64, axes=2, places="scattered", heads=6, kv_heads=2),
    "middle32": dict(lens_q=[300, 180, 150, 3], axes=3, places="scattered", maxd=60),
    "middle_rows": dict(lens_q=[330, 329], lens_k=[129, 140], axes=2, places="scattered"),
    # the key pass with two CTAs an SM and several heads, and where one CTA's sums fill the shared memory
    "long_turns": dict(lens_q=[520, 300], heads=8, kv_heads=2, axes=3, places="scattered", maxd=40),
    "long_turns64": dict(lens_q=[290, 310], heads=6, kv_heads=1, axes=2, places="frames", maxd=20, dim=64),
    "long_one_cta": dict(lens_q=[300, 411], axes=3, places="scattered", maxd=60, buckets=48),
    "long_one_cta64": dict(lens_q=[350], axes=3, places="scattered", dim=64),
    # columns whose positions repeat
    "bricks": dict(lens_q=[200, 64, 77], axes=3, places="bricks", maxd=6, buckets=12),
    "bricks_short": dict(lens_q=[64, 50, 64, 9] * 12, heads=8, kv_heads=2, axes=3, places="bricks", maxd=16, buckets=16),
    "bricks_short64": dict(lens_q=[64, 33, 0] * 20, dim=64, axes=2, places="bricks", maxd=3, buckets=6),
    "bricks_long": dict(lens_q=[333, 448], axes=3, places="bricks", maxd=16, buckets=16),
    "bricks_long64": dict(lens_q=[320, 290], axes=1, places="bricks", maxd=9, buckets=8, dim=64),
    "bricks_one_cta": dict(lens_q=[448], axes=3, places="bricks", maxd=20, buckets=48, dim=64),
    "bricks_cross": dict(lens_q=[3, 20, 1], lens_k=[600, 64, 128], axes=3, places="bricks", maxd=5, buckets=10),
    # 64 and 128 rows a CTA, and the most rows of the kernel for few
    "rows64": dict(lens_q=[61, 40], lens_k=[300, 33], axes=2, places="scattered"),
    "rows128": dict(lens_q=[90, 75, 101], lens_k=[400, 257, 70], axes=3, places="scattered"),
    "rows_few": dict(lens_q=[24, 19, 23], lens_k=[400, 257, 70], heads=32, axes=2, places="scattered"),
}


@pytest.mark.parametrize("name", FORWARD)
def test_forward_and_gradients(name):
    Case(**FORWARD[name]).check()


FEW = {
    "token": dict(lens_q=[1], lens_k=[1]),
    "tokens": dict(lens_q=[1] * 5, lens_k=[1, 31, 32, 33, 1000], heads=32, kv_heads=2, places="scattered"),
    "past": dict(lens_q=[1], lens_k=[5000], heads=32, kv_heads=2),
    "past_d64": dict(lens_q=[1, 1], lens_k=[3000, 0], heads=4, kv_heads=4, dim=64, axes=2, places="scattered"),
    "run": dict(lens_q=[7, 16, 1, 0, 5], lens_k=[700, 16, 2000, 5, 129], heads=6, kv_heads=2, axes=3, places="scattered"),
    "wide_group": dict(lens_q=[3, 2], lens_k=[400, 90], heads=40, kv_heads=2, dim=64),
    "split": dict(lens_q=[40], lens_k=[4000], heads=2, kv_heads=1),
    "split_ragged": dict(lens_q=[33, 60, 1], lens_k=[4100, 3, 0], heads=2, kv_heads=2, dim=64, places="scattered"),
    "outside": dict(lens_q=[2, 1], lens_k=[600, 40], lead=3),
}


@pytest.mark.parametrize("name", FEW)
def test_few_queries(name):
    Case(**FEW[name]).check()


def test_rows_outside_segments_stay():
    c = Case([70, 5], lens_k=[90, 0], lead=9)
    for x in (c.q, c.dout):
        x[:9] = float("nan")
        x[-9:] = float("nan")
    for x in (c.k, c.v):
        x[:9] = float("inf")
        x[-9:] = float("nan")
    got, _ = c.check()
    marked = {n: torch.full_like(x, 7.0) for n, x in got.items()}
    f = c.forward(marked["out"], marked["lse"])
    c.backward(f, marked)
    for n in ("out", "lse", "dq", "dk", "dv"):
        assert bool((marked[n][:9] == 7).all()) and bool((marked[n][-9:] == 7).all()), n
        assert torch.equal(marked[n][9:-9], got[n][9:-9]), n
    few = Case([1, 2], lens_k=[2000, 700], lead=4, heads=16, kv_heads=2)
    out = torch.full_like(few.q, 7.0)
    few.forward(out)
    assert bool((out[:4] == 7).all()) and bool((out[-4:] == 7).all())


# a neighbour segment's infinities and NaNs do not reach a row, whatever the tile
@pytest.mark.parametrize("lens", [[40, 23, 61], [1, 1, 1], [130, 5, 200], [300, 310, 333], [40, 23, 61] * 14])
def test_neighbours_do_not_leak(lens):
    c = Case(lens, dim=64)
    clean = {n: x.clone() for n, x in c.check()[0].items()}
    lo, hi = lens[0], lens[0] + lens[1]
    for x in (c.k, c.v, c.q, c.dout):
        x[lo:hi] = float("nan")
    f = c.forward()
    got = {**f, **c.backward(f)}
    for n in ("out", "lse", "dq", "dk", "dv"):
        for part in (slice(0, lo), slice(hi, None)):
            assert torch.equal(got[n][part], clean[n][part]), n


@pytest.mark.parametrize("lens_q,lens_k", [([130], None), ([3], [200]), ([290, 300], None), ([40, 23] * 20, None)])
@pytest.mark.parametrize("low", [-math.inf, torch.finfo(BF).min, -1e30])
def test_masks_by_the_table(lens_q, lens_k, low):
    """Entries at -inf or at the type's lowest value mask a bucket; a row whose every key is at -inf
    is empty, a row whose every key is at the lowest value is a mean over equals."""
    c = Case(lens_q, lens_k, buckets=4, maxd=3)
    c.table[0, 2:] = low  # keys after the query
    c.check()
    c.table[0, :, 1] = low  # every key of one head
    c.check()


def test_reproducible_and_no_lse():
    c = Case([300, 1, 129], axes=2, places="scattered", heads=8, kv_heads=2)
    a = c.forward()
    ga = {n: x.clone() for n, x in c.backward(a).items()}
    b = c.forward()
    gb = c.backward(b)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    for n in ga:
        assert torch.equal(ga[n], gb[n]), n
    out = torch.empty_like(c.q)
    nsa.lsrm_relpos_forward(c.desc, *c.where, c.q, c.k, c.v, out, None, c.ws)
    assert torch.equal(out, a["out"])


def test_differences():
    """The gradients agree with central differences of the 64-bit loss along random directions (the
    kernel's own outputs are too coarse for a difference)."""
    c = Case([50, 20], axes=2, places="scattered", maxd=9, buckets=8)
    got, _ = c.check()
    g = torch.Generator().manual_seed(3)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("table", "dtable")):
        base = getattr(c, name).double()
        way = torch.randn(base.shape, generator=g).cuda().double()
        loss = []
        for h in (1e-5, -1e-5):
            args = {"table": c.table, "q": c.q, "k": c.k, "v": c.v, name: base + h * way}
            o = ref.attention(c.off_q, c.off_k, c.pos_q, c.pos_k, c.bucket_of, args["table"], args["q"], args["k"],
                              args["v"])["out"][0]
            loss.append(float((o * c.dout.double()).sum()))
        want = (loss[0] - loss[1]) / 2e-5
        have = float((got[grad].double() * way).sum())
        # every entry of the gradient within its bound, met along the direction
        bound = float((c.reference(True)[grad][1] * way.abs()).sum())
        assert abs(have - want) <= bound + 1e-4 * abs(want), (name, have, want, bound)


@pytest.mark.parametrize("lens_q,lens_k", [([100, 260], None), ([300, 410], None), ([40, 23] * 50, None),
                                           ([1, 1, 2], [900, 40, 700]), ([1, 2], [7000, 5000]), ([600], None)])
def test_captured_and_other_stream(lens_q, lens_k):
    c = Case(lens_q, lens_k, heads=8, kv_heads=2, dim=64)
    want = {**c.forward()}
    want.update({n: x.clone() for n, x in c.backward(want).items()})
    f = {"out": torch.zeros_like(c.q), "lse": torch.zeros_like(want["lse"])}
    r = {n: torch.zeros_like(want[n]) for n in ("dq", "dk", "dv", "dtable")}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.forward(f["out"], f["lse"])
        c.backward(f, r)
    c.q.mul_(0.5)  # the replay works on what the tensors hold then
    graph.replay()
    torch.cuda.synchronize()
    new = c.reference(True)
    for n, x in {**f, **r}.items():
        ref.check(n, x, new[n])
    c.q.mul_(2.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f2 = c.forward()
        r2 = c.backward(f2)
    side.synchronize()
    for n, x in {**f2, **r2}.items():
        assert torch.equal(x, want[n]), n


def test_bad_tables_are_reported_not_followed():
    """Segment bounds, bucket ids and positions outside their ranges are clipped and reported."""
    c = Case([40, 40])
    c.off_k[1] = 1 << 20
    c.forward()
    assert nsa.lsrm_nsa_last_device_status(c.ws) == 5
    c = Case([40, 40])
    c.off_q[1] = -7
    f = c.forward()
    c.backward(f)
    assert nsa.lsrm_nsa_last_device_status(c.ws) == 5
    c = Case([40, 40])
    c.bucket_of[128] = 1000
    f = c.forward()
    c.backward(f)
    assert nsa.lsrm_nsa_last_device_status(c.ws) == 5
    c = Case([3], lens_k=[40])
    c.bucket_of[100:] = -1
    c.pos_k[7] = 2 ** 31 - 1
    c.forward()
    assert nsa.lsrm_nsa_last_device_status(c.ws) == 5
    assert nsa.lsrm_nsa_last_device_status(c.ws) == 0


@pytest.mark.parametrize("lens", [[40, 40], [300, 310, 290], [40, 24, 9] * 30])
@pytest.mark.parametrize("what", ["off_q", "off_k", "bucket_of", "pos_q", "pos_k"])
def test_bad_tables_in_every_kernel(lens, what):
    c = Case(lens, heads=8, kv_heads=2, axes=2, places="scattered")
    if what == "pos_q":
        c.pos_q = c.pos_q.clone()  # not the keys' any more
    x = getattr(c, what)
    keep = x.clone()
    if what.startswith("off"):
        x[1] = 2 ** 31 - 1
        x[2] = -5
    elif what == "bucket_of":
        x[:100] = 32
        x[150:] = -2 ** 31
    else:
        x[3], x[20] = 2 ** 31 - 1, -2 ** 31
    c.backward(c.forward())
    assert nsa.lsrm_nsa_last_device_status(c.ws) == 5
    x.copy_(keep)
    c.check()


def test_two_calls_at_once():
    cases = [Case([700, 300], heads=8, kv_heads=2), Case([40, 64, 1] * 40, heads=8, kv_heads=2, axes=3, places="bricks")]
    want = []
    for c in cases:
        f = c.forward()
        want.append({**f, **c.backward(f)})
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(3):
        for c, side, g in zip(cases, sides, got):
            with torch.cuda.stream(side):
                f = c.forward()
                g.append({**f, **c.backward(f)})
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for r in g:
            for n, x in r.items():
                assert torch.equal(x, w[n]), n


def test_norm_then_attend_then_back():
    """The run a training step makes: layer norm of the query and key rows per head, attention with
    the bias, and back through both, against the chain of the 64-bit definitions."""
    c = Case([96, 40], heads=8, kv_heads=2, dim=64, axes=3, places="scattered", maxd=12, buckets=16)
    g = torch.Generator().manual_seed(9)
    raw = {"q": (torch.randn(c.q.shape, generator=g) * 2 + 0.3).to(BF).cuda(),
           "k": (torch.randn(c.k.shape, generator=g) * 2 - 0.1).to(BF).cuda()}
    gamma = (1 + 0.1 * torch.randn(64, generator=g)).to(BF).cuda()
    beta = (0.1 * torch.randn(64, generator=g)).to(BF).cuda()
    stats = {}
    for n in ("q", "k"):
        rows = raw[n].numel() // 64
        stats[n] = torch.empty(2, rows, device="cuda").unbind(0)
        nsa.lsrm_layer_norm_forward(raw[n], gamma, beta, 1e-6, getattr(c, n), *stats[n])
    f = c.forward()
    r = c.backward(f)
    dq = {}
    for n in ("q", "k"):
        ws = nsa.layer_norm_workspace(raw[n].numel() // 64, 64)
        dq[n] = (torch.empty_like(raw[n]), torch.empty_like(gamma), torch.empty_like(beta))
        nsa.lsrm_layer_norm_backward(r["d" + n], raw[n], gamma, *stats[n], *dq[n], ws)
    # each step against its definition on the inputs that it was given
    for n in ("q", "k"):
        ref.check("y", getattr(c, n), {k: (v.reshape(getattr(c, n).shape), b.reshape(getattr(c, n).shape))
                                       for k, (v, b) in ref.layer_norm(raw[n], gamma, beta, 1e-6).items()
                                       if k == "y"}["y"])
        want = ref.layer_norm(raw[n], gamma, beta, 1e-6, r["d" + n], stats[n])
        for got, name in zip(dq[n], ("dx", "dgamma", "dbeta")):
            ref.check(name, got, want[name])
    want = c.reference(True)
    for n, x in {**f, **r}.items():
        ref.check(n, x, want[n])
