"""Calls of the relative-position-bias attention from two host threads at once, whose bias tables need
different amounts of shared memory of the same kernels."""
import threading

import pytest
import torch

from test_gpu_relpos import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens_q,lens_k,maxd", [
    ([70, 60, 75], [90, 300, 40], 600),   # forward of 128 rows a CTA, dq and key pass of 64
    ([40, 64, 33] * 20, None, 60),        # short segments
    ([300, 290], None, 1000),             # tensor-memory forward, key pass of 64 rows
    ([500, 450], None, 300),              # tensor-memory kernels
    ([3, 1], [900, 600], 1000),           # few queries
])
def test_two_threads_with_tables_of_different_sizes(lens_q, lens_k, maxd):
    kw = dict(axes=3, places="scattered", buckets=16)
    cases = [Case(lens_q, lens_k, maxd=maxd, **kw), Case(lens_q, lens_k, maxd=1, **kw)]
    want = []
    for c in cases:
        f = c.forward()
        want.append({**f, **c.backward(f)})
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(cases))

    def work(c, want):
        try:
            stream = torch.cuda.Stream()
            f = {n: torch.empty_like(want[n]) for n in ("out", "lse")}
            g = {n: torch.empty_like(want[n]) for n in ("dq", "dk", "dv", "dtable")}
            torch.cuda.synchronize()
            start.wait()
            with torch.cuda.stream(stream):
                for _ in range(400):
                    c.forward(f["out"], f["lse"])
                    c.backward(f, g)
            stream.synchronize()
            wrong.extend(n for n, x in {**f, **g}.items() if not torch.equal(x, want[n]))
        except Exception as e:  # reported by the test's own thread
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
