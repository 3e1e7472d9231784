"""The gradients of the relative-position-bias attention on the GPU row by row against their definition in
64 bits: the shapes of every kernel, peaked rows, scores and biases of any size."""
import math

import pytest
import torch

import relpos_bars as bars
import relpos_ref as ref
from test_gpu_relpos import FEW, FORWARD, Case

from block_sparse_gqa_nsa_b200 import nsa

pytestmark = pytest.mark.gpu


def rows(c, status=0):
    f = c.forward()
    got = c.backward(f)
    assert nsa.lsrm_nsa_last_device_status(c.ws) == status
    want = bars.gradients(*c.where, c.q, c.k, c.v, c.dout, c.scale or None)
    for n, x in got.items():
        # rows outside the segments are not the call's
        at = slice(c.lead, x.shape[0] - c.lead) if n != "dtable" else slice(None)
        bars.check(n, x[at], (want[n][0][at], want[n][1][at]))
    return f, got


@pytest.mark.parametrize("name", FORWARD)
def test_rows(name):
    rows(Case(**FORWARD[name]))


@pytest.mark.parametrize("name", FEW)
def test_rows_of_few_queries(name):
    rows(Case(**FEW[name]))


# the backward's kernels: many short segments, 64-row tiles, and 128-row tiles at both head dims
SHAPES = {
    "many_short": dict(lens_q=[64, 33, 1, 50] * 25, heads=8, kv_heads=2),
    "many_short64": dict(lens_q=[i * 7 % 65 for i in range(70)], heads=12, kv_heads=3, dim=64, axes=2,
                         places="scattered", maxd=40),
    "many_short_bricks": dict(lens_q=[64, 20, 64] * 23, heads=12, kv_heads=3, axes=3, places="bricks", maxd=16,
                              buckets=16),
    "short": dict(lens_q=[64, 33, 1, 50] * 15, heads=8, kv_heads=2),
    "middle32": dict(lens_q=[300, 200, 77]),
    "middle64": dict(lens_q=[120, 100, 31], dim=64),
    "past128": dict(lens_q=[140, 160], lens_k=[200, 130]),
    "long32": dict(lens_q=[600, 511]),
    "long64": dict(lens_q=[512, 300], dim=64),
    "long_axes": dict(lens_q=[450], dim=64, axes=3, places="scattered", maxd=30, buckets=16),
    "long_turns": dict(lens_q=[520, 400], axes=2, places="scattered", maxd=40),
    "cross": dict(lens_q=[400, 330], lens_k=[300, 500], heads=6, dim=64),
    "few": dict(lens_q=[1, 9, 3], lens_k=[700, 64, 2000], heads=16),
    "past64": dict(lens_q=[340, 400], lens_k=[70, 128]),
    "past64_dim64": dict(lens_q=[200, 140, 150], lens_k=[65, 128, 66], dim=64, heads=6),
    "group4": dict(lens_q=[40, 64, 1, 0] * 15, heads=8, kv_heads=2, axes=2, places="scattered"),
}


# what the kernels of many short segments can meet
MANY = {
    "wide_group": dict(lens_q=[40, 30] * 51, heads=40, kv_heads=2, axes=1, buckets=8),
    "long_beside": dict(lens_q=[20, 0, 150, 9, 64] * 40, lens_k=[64, 7, 0, 200, 1] * 40, heads=4, kv_heads=1,
                        places="scattered"),
    "outside": dict(lens_q=[33, 12, 60] * 34, lead=5, heads=8, kv_heads=2, axes=3, places="scattered", maxd=7, buckets=7),
    "few_keys64": dict(lens_q=[50, 41] * 100, lens_k=[1, 2] * 100, heads=4, kv_heads=1, dim=64),
    "frames": dict(lens_q=[64, 31] * 50, heads=8, kv_heads=2, axes=2, places="frames", maxd=5, buckets=6),
}


@pytest.mark.parametrize("name", MANY)
def test_many_short_segments(name):
    c = Case(**MANY[name])
    c.check()
    rows(c)


@pytest.mark.parametrize("low", [-math.inf, torch.finfo(torch.bfloat16).min, -1e30])
def test_many_short_segments_under_masks(low):
    c = Case(lens_q=[40, 23, 64] * 35, heads=8, kv_heads=2, buckets=4, maxd=3)
    c.table[0, 2:] = low  # keys after the query
    c.check()
    rows(c)
    c.table[0, :, 1] = low  # every key of one head
    c.check()
    rows(c)


@pytest.mark.parametrize("what", ["off_q", "off_k", "bucket_of", "pos_q", "pos_k"])
def test_bad_tables_of_many_short_segments(what):
    c = Case(lens_q=[40, 24, 9] * 35, heads=8, kv_heads=2, axes=2, places="scattered")
    c.pos_q = c.pos_q.clone()  # not the keys'
    x = getattr(c, what)
    keep = x.clone()
    if what.startswith("off"):
        x[1], x[2] = 2 ** 31 - 1, -5
    elif what == "bucket_of":
        x[:100], x[150:] = 32, -2 ** 31
    else:
        x[3], x[20] = 2 ** 31 - 1, -2 ** 31
    c.backward(c.forward())
    assert nsa.lsrm_nsa_last_device_status(c.ws) == 5
    x.copy_(keep)
    c.check()


def test_neighbours_of_many_short_segments_do_not_leak():
    c = Case([40, 23, 61] * 40, dim=64, heads=4, kv_heads=2 // 2)
    clean = {n: x.clone() for n, x in c.check()[0].items()}
    for x in (c.k, c.v, c.q, c.dout):
        x[40:63] = float("nan")
    f = c.forward()
    got = {**f, **c.backward(f)}
    for n in ("out", "lse", "dq", "dk", "dv"):
        for part in (slice(0, 40), slice(63, None)):
            assert torch.equal(got[n][part], clean[n][part]), n


@pytest.mark.parametrize("spread", [4.0, 8.0])
@pytest.mark.parametrize("name", SHAPES)
def test_peaked_rows(name, spread):
    """Rows with nearly all weight on one key: dS nearly cancels, so the Delta of the rounded out would show."""
    rows(Case(**SHAPES[name], spread=spread))


@pytest.mark.parametrize("spread", [2e3, 3e4, 3e5, 2e6])
@pytest.mark.parametrize("name", SHAPES)
def test_huge_scores_beside_a_small_table(name, spread):
    """LSE so large that fp32 loses the sum: every row's weights still sum to 1."""
    f, got = rows(Case(**SHAPES[name], spread=spread))
    assert all(bool(x.isfinite().all()) for x in got.values())


@pytest.mark.parametrize("spread", [3e5, 2e6])
@pytest.mark.parametrize("name", SHAPES)
def test_huge_scores_beside_one_heads_large_table(name, spread):
    """A head whose table is large is scored in other units than its neighbours, in both passes alike."""
    c = Case(**SHAPES[name], spread=spread)
    c.table[0, :, 1] = 100.0
    rows(c)


@pytest.mark.parametrize("name", ["middle32", "long32", "long64"])
def test_some_huge_rows(name):
    """A few rows of huge scores among ordinary ones."""
    c = Case(**SHAPES[name])
    c.q[::37] = (c.q[::37].float() * 3e5).to(c.q.dtype)
    c.q[50:60, 1] = (c.q[50:60, 1].float() * 1e4).to(c.q.dtype)
    rows(c)


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("low", [-1e5, -1e7, -1e9, -1e30])
def test_rows_under_a_mask_on_one_axis_and_biases_on_another(name, low):
    """Every key of a row at a finite mask on one axis: the order in which the axes are added decides how a
    score rounds, so every pass has to take the same one.  The other axis makes one key stand out (distance
    0) by far more than the mask's spacing, where a mask still has one."""
    kw = {**SHAPES[name], "axes": 2, "places": "order"}
    kw.pop("maxd", None)
    c = Case(**kw)
    c.table[0, :, 0] = low
    c.table[1, :, 0] = -100.5
    c.table[1, c.bucket_of[128].item(), 0] = 100.5
    if low < -1e8:  # the mask swallows the other axis: equal weights
        c.table[1, :, 0] = 0
        c.q[:, 0] = 0
    rows(c)


def test_one_key_has_all_the_weight():
    """Whatever its bias: dv is the sum of dO over the queries and heads."""
    for lens_q, lens_k in (([1] * 50, [1] * 50), ([64, 30] * 30, [1] * 60), ([300], [1]), ([700, 700], [400, 1])):
        c = Case(lens_q, lens_k, axes=2, places="scattered", heads=4, kv_heads=2)
        c.table[0] = -1e7
        c.table[1] = (c.table[1].float() * 40).to(c.table.dtype)
        f, got = rows(c)
        lo = 0
        for n, m, at in zip(lens_q, lens_k, c.off_k.tolist()):
            if m == 1:
                want = c.dout[lo:lo + n].double().view(n, 2, 2, 32).sum((0, 2))
                size = c.dout[lo:lo + n].double().abs().view(n, 2, 2, 32).sum((0, 2))
                assert bool(((got["dv"][at].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size).all())
            lo += n


def test_a_masked_head_over_a_long_past():
    """A head whose every bias is the type's lowest value: the mean over many keys."""
    c = Case([400, 3], [20000, 17], heads=2, kv_heads=1, dim=64)
    c.table[0, :, 1] = torch.finfo(torch.bfloat16).min
    f, got = rows(c)
    want = c.reference(False)
    ref.check("out", f["out"], want["out"])
    ref.check("lse", f["lse"], want["lse"])


def test_gradients_are_the_same_bits_again():
    for name in ("long32", "long64", "middle32"):
        c = Case(**SHAPES[name], spread=1e5)
        f = c.forward()
        a = {n: x.clone() for n, x in c.backward(f).items()}
        b = c.backward(f)
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_scores_past_the_documented_size_are_reported():
    """Scores past 2^27 lose LSE itself: finite and reported, or right."""
    c = Case([300], spread=1e12)
    f = c.forward()
    c.backward(f)
    assert nsa.lsrm_nsa_last_device_status(c.ws) in (0, 5)
    assert math.isfinite(float(f["out"].float().abs().max()))
