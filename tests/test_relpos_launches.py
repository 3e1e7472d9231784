"""What the relative-position attention asks of the CUDA runtime, on the CPU: a stand-in for the few runtime
calls that it makes records them and launches nothing."""
import json
import os
import subprocess
import sys

import pytest

from block_sparse_gqa_nsa_b200.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = r"""
#include <stdio.h>
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3_;
typedef struct { dim3_ grid, block; size_t smem; void* stream; void* attrs; unsigned n; } config_;
int cudaFuncSetAttribute(const void* f, int attr, int value) { printf("[\"set\", %zu, %d, %d]\n", (size_t)f, attr, value); return 0; }
int cudaLaunchKernel(const void* f, dim3_ g, dim3_ b, void** args, size_t smem, void* s) {
  printf("[\"launch\", %zu, %u, %zu, %u]\n", (size_t)f, g.x, smem, b.x); return 0; }
int cudaLaunchKernelExC(const config_* c, const void* f, void** args) {
  printf("[\"launch\", %zu, %u, %zu, %u]\n", (size_t)f, c->grid.x, c->smem, c->block.x); return 0; }
int cudaGetLastError(void) { return 0; }
static int encode() { return 0; }
int cudaGetDriverEntryPoint(const char* name, void** p, unsigned long long flags, int* q) { *p = (void*)encode; *q = 0; return 0; }
"""

CALLS = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from block_sparse_gqa_nsa_b200 import nsa
lib = nsa.load_library()
for maxd, nb in ((1, 2), (1023, 64), (100, 16), (1, 64)):
    for S, q, k in ((2, 1, 900), (2, 9, 900), (2, 50, 900), (2, 90, 900), (60, 50, 50), (2, 200, 200), (2, 700, 700),
                    (1, 30, 30)):
        for dim in (32, 64):
            for axes in (1, 2, 3):
                for heads, kv in ((4, 2), (32, 2)):
                    d = nsa.make_relpos_desc(S * q, S * k, S, heads, kv, dim, axes, nb, maxd)
                    n = nsa.lsrm_relpos_workspace_size(d)
                    for r in (lib.lsrm_relpos_forward(ctypes.byref(d), *[4096] * 11, 4096, n, None),
                              lib.lsrm_relpos_backward(ctypes.byref(d), *[4096] * 16, 4096, n, None)):
                        if r:
                            sys.exit(f"status {r}")
"""


SHAPES = r"""
import ctypes, json, sys
sys.path.insert(0, sys.argv[1])
from block_sparse_gqa_nsa_b200 import nsa
lib = nsa.load_library()
for name, c in json.loads(sys.argv[2]).items():
    lq, lk = c["lens_q"], c.get("lens_k") or c["lens_q"]
    d = nsa.make_relpos_desc(sum(lq), sum(lk), len(lq), c.get("heads", 4), c.get("kv_heads", 2), c.get("dim", 32),
                             c.get("axes", 1), c.get("buckets", 32), c.get("maxd", 128))
    n = nsa.lsrm_relpos_workspace_size(d)
    print(json.dumps(["case", name]), flush=True)
    lib.lsrm_relpos_forward(ctypes.byref(d), *[4096] * 11, 4096, n, None)
    lib.lsrm_relpos_backward(ctypes.byref(d), *[4096] * 16, 4096, n, None)
    ctypes.CDLL(None).fflush(None)
"""


@pytest.fixture(scope="module")
def recorded(tmp_path_factory):
    build()
    d = tmp_path_factory.mktemp("fake")
    (d / "fake.c").write_text(FAKE)
    subprocess.check_call(["gcc", "-shared", "-fPIC", "-w", "-o", str(d / "fake.so"), str(d / "fake.c")])

    def run(calls, *args):
        (d / "calls.py").write_text(calls)
        out = subprocess.run([sys.executable, str(d / "calls.py"), ROOT, *args],
                             env={**os.environ, "LD_PRELOAD": str(d / "fake.so")}, capture_output=True, text=True)
        assert out.returncode == 0, out.stderr[-500:]
        return [json.loads(x) for x in out.stdout.splitlines() if x.startswith("[")]

    return run


@pytest.fixture(scope="module")
def records(recorded):
    return recorded(CALLS)


def test_a_kernels_shared_memory_limit_is_the_same_for_every_call(records):
    """The limit belongs to the kernel, not to the call: one that followed a call's table could be lowered by a
    second thread between the first one's setting and its launch."""
    limits = {}
    for what, f, *x in records:
        if what == "set":
            limits.setdefault((f, x[0]), set()).add(x[1])
    assert len(limits) > 20
    assert all(len(v) == 1 for v in limits.values()), sorted(limits.values(), key=len)[-1]


def test_launches_are_within_their_limits(records):
    limit, seen = {}, set()
    for what, f, *x in records:
        if what == "set":
            limit[f] = x[1]
        else:
            assert 0 < x[0] < 2 ** 31 and x[1] <= max(limit.get(f, 0), 48 * 1024), (x, limit.get(f))
            seen.add(f)
    assert len(seen) > 30


def test_the_gradient_tests_shapes_take_every_kernel(recorded):
    """By the threads of their CTAs: 256 with shared memory for many short segments, 320 on tensor memory."""
    import test_gpu_relpos_gradients as g

    many = {f"MANY {n}": c for n, c in g.MANY.items()}
    threads, name = {}, None
    for what, *x in recorded(SHAPES, json.dumps({**g.SHAPES, **many})):
        if what == "case":
            name = x[0]
        elif what == "launch":
            threads.setdefault(name, []).append(x[3] if x[2] else 0)
    for name, t in threads.items():
        assert (t.count(256) == 2) == name.startswith(("many", "MANY")), (name, t)
        assert (t.count(320) == 3) == name.startswith(("long", "cross", "past64")), (name, t)


@pytest.mark.timeout(60)
def test_too_many_heads_are_refused_at_once():
    """The plans try every split of a group's heads: not of 2^31 of them (ten seconds a call)."""
    import time

    from block_sparse_gqa_nsa_b200 import nsa

    build()
    nsa.load_library()
    for q in (100, 1000):
        start = time.time()
        assert nsa.lsrm_relpos_workspace_size(nsa.make_relpos_desc(q, q, 1, 2 ** 31 - 1, 1, 32, 1, 32, 128)) == 0
        assert time.time() - start < 1
    assert nsa.lsrm_relpos_workspace_size(nsa.make_relpos_desc(10, 10, 1, 65535, 1, 32, 1, 32, 128)) > 0
    assert nsa.lsrm_relpos_workspace_size(nsa.make_relpos_desc(10, 10, 1, 65536, 1, 32, 1, 32, 128)) == 0
