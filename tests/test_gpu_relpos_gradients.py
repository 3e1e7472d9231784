"""The gradients of the relative-position-bias attention on the GPU row by row against their definition in
64 bits: the shapes of every kernel, and peaked rows."""
import pytest

import relpos_bars as bars
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


# the backward's kernels: short segments, 64-row tiles, and 128-row tiles at both head dims
SHAPES = {
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
}


@pytest.mark.parametrize("spread", [4.0, 8.0])
@pytest.mark.parametrize("name", SHAPES)
def test_peaked_rows(name, spread):
    """Rows with nearly all weight on one key: dS nearly cancels, so the Delta of the rounded out would show."""
    rows(Case(**SHAPES[name], spread=spread))
