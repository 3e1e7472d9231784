"""The bars that the gradients of the relative-position-bias attention are held to, on the CPU: they let the
kernels' arithmetic pass and see a key tile, a warp's keys or the correction of Delta left out."""
import math

import pytest
import torch

import relpos_bars as bars
import relpos_ref as ref

BF = torch.bfloat16


def inputs(lens, heads=4, kv_heads=2, dim=32, axes=1, buckets=32, maxd=128, spread=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    off = torch.tensor([0] + lens).cumsum(0).int()
    n = int(off[-1])
    pos = torch.arange(n)[:, None].expand(n, axes).contiguous().int()
    normal = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF)  # noqa: E731
    return (off, off, pos, pos, torch.tensor(ref.log_buckets(buckets, maxd), dtype=torch.int32),
            normal(axes, buckets, heads), normal(n, heads, dim, std=spread), normal(n, kv_heads, dim),
            normal(n, kv_heads, dim), normal(n, heads, dim))


def computed(args, leave=None, coarse=False):
    """The kernels' arithmetic: fp32 with P and dS rounded to bf16 as operands, Delta from the rounded out
    plus its correction (not, where coarse); leave(i, j): pairs kept out of the table's gradient."""
    q, k, table = args[6], args[7], args[5]
    r = {"dq": torch.zeros(q.shape), "dk": torch.zeros(k.shape), "dv": torch.zeros(k.shape),
         "dtable": torch.zeros(table.shape, dtype=torch.float64)}
    round_ = lambda x: x.to(BF).float()  # noqa: E731
    for s in bars.pieces(*args):
        P, do, kk = s["P"].float(), s["do"].float(), s["k"].float()
        o = round_(round_(P) @ s["v"].float())
        d1 = (do * o).sum(1, keepdim=True)
        dP = s["dP"].float()
        ds = P * (dP - d1)
        more = torch.zeros_like(d1) if coarse else ds.sum(1, keepdim=True)
        r["dq"][s["rows"], s["h"]] = (round_(ds) @ kk - more * (round_(P) @ kk)) * s["scale"]
        ds = P * (dP - (d1 + more))
        r["dk"][s["keys"], s["g"]] += round_(ds).T @ s["q"].float() * s["scale"]
        r["dv"][s["keys"], s["g"]] += round_(P).T @ do
        if leave is not None:
            i, j = torch.meshgrid(torch.arange(ds.shape[0]), torch.arange(ds.shape[1]), indexing="ij")
            ds = torch.where(leave(i, j), 0.0, ds)
        for a in range(table.shape[0]):
            r["dtable"][a, :, s["h"]] += bars.table_sum(ds.double(), s["bucket"][..., a], table.shape[1])
    return {n: x.to(BF) for n, x in r.items()}


SHAPES = [dict(lens=[300]), dict(lens=[300, 555], dim=64), dict(lens=[2500], heads=2, kv_heads=1),
          dict(lens=[40, 64, 1, 7], axes=2), dict(lens=[512], dim=64, spread=8.0)]


@pytest.mark.parametrize("kw", SHAPES)
def test_the_kernels_arithmetic_passes(kw):
    args = inputs(**kw)
    want = bars.gradients(*args)
    for n, x in computed(args).items():
        bars.check(n, x, want[n])


@pytest.mark.parametrize("kw,leave", [
    (SHAPES[2], lambda i, j: j // 64 == 5),  # a tile of 64 keys
    (SHAPES[1], lambda i, j: j // 16 == 3),  # a warp's 16 keys
    (SHAPES[0], lambda i, j: j == 299),      # the last key
    (SHAPES[2], lambda i, j: i // 64 == 20), # a chunk of 64 queries
])
def test_left_out_pairs_are_seen(kw, leave):
    args = inputs(**kw)
    want = bars.gradients(*args)
    assert bars.worst("dtable", computed(args, leave)["dtable"], want["dtable"]) > 1.5


@pytest.mark.parametrize("spread", [4.0, 8.0])
def test_a_coarse_delta_is_seen(spread):
    """Peaked rows, whose dq nearly cancels: without the correction rows are off by several times their size."""
    args = inputs([512], dim=64, spread=spread)
    want = bars.gradients(*args)
    got = computed(args, coarse=True)
    for n in ("dq", "dk"):
        assert bars.worst(n, got[n], want[n]) > 1.0, n


def test_a_factor_on_a_row_is_seen():
    """P that sums to 1.02 instead of 1 shows in dv."""
    args = inputs([200], spread=1e5)
    want = bars.gradients(*args)
    got = computed(args)["dv"].float() * 1.02
    assert bars.worst("dv", got, want["dv"]) > 1.0
    assert bars.worst("dv", got / 1.02, want["dv"]) <= 1.0
    assert math.isfinite(float(want["dv"][1].max()))
