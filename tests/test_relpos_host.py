"""Host side of the relative-position-bias attention and the layer norm: the logarithmic buckets, the
workspace sizes and the refusals, none of which touches a GPU."""
import ctypes
import math

import pytest
import torch

from block_sparse_gqa_nsa_b200 import nsa
from block_sparse_gqa_nsa_b200.build import build
import relpos_ref as ref


@pytest.fixture(scope="module")
def lib():
    build()
    return nsa.load_library()


def desc(**kw):
    base = dict(n_q_tokens=100, n_k_tokens=100, n_segs=2, n_q_heads=4, n_kv_heads=2, head_dim=32, n_axes=1,
                n_buckets=32, max_distance=128)
    return nsa.make_relpos_desc(**{**base, **kw})


@pytest.mark.parametrize("n,d", [(2, 1), (4, 1), (8, 16), (32, 128), (32, 8), (6, 1000), (64, 1023), (64, 5), (32, 4096 // 8)])
def test_log_buckets(lib, n, d):
    got = nsa.lsrm_relpos_log_buckets(n, d).tolist()
    assert got == ref.log_buckets(n, d)
    half = n // 2
    assert got[d] == 0 and max(got) < n and min(got) >= 0
    assert all(b >= half for b in got[d + 1:]) and all(b < half for b in got[:d + 1])


def test_log_buckets_borders():
    """A border that is a power: with 8 exact distances, 8 spaced ones up to 128 meet 16, 32, 64, 128
    exactly (8 * 2^(b/2)); floating-point logarithms would have to get these right by luck."""
    got = nsa.lsrm_relpos_log_buckets(32, 128).tolist()
    for b, n in ((10, 16), (12, 32), (14, 64)):
        assert got[128 - n] == b and got[128 - n + 1] == b - 1


def test_log_buckets_refusals(lib):
    for n, d in ((0, 8), (3, 8), (66, 8), (8, 0), (8, 1024), (8, -1)):
        with pytest.raises(nsa.NsaError):
            nsa.lsrm_relpos_log_buckets(n, d)
    assert lib.lsrm_relpos_log_buckets(8, 8, None) == 1


def test_workspace_size(lib):
    assert nsa.lsrm_relpos_workspace_size(desc()) % 256 == 0 and nsa.lsrm_relpos_workspace_size(desc()) > 0
    assert nsa.lsrm_relpos_workspace_size(desc(n_q_tokens=0, n_k_tokens=0)) > 0
    for bad in (dict(n_q_tokens=-1), dict(n_k_tokens=-1), dict(n_segs=0), dict(n_q_heads=3), dict(n_kv_heads=0),
                dict(head_dim=48), dict(head_dim=128), dict(n_axes=0), dict(n_axes=4), dict(n_buckets=0),
                dict(n_buckets=65), dict(max_distance=0), dict(max_distance=1024), dict(scale=-1.0),
                dict(scale=math.inf), dict(scale=math.nan), dict(n_q_tokens=2 ** 31), dict(n_k_tokens=2 ** 31),
                dict(n_q_tokens=2 ** 31 - 1, n_q_heads=128, n_kv_heads=128)):
        assert nsa.lsrm_relpos_workspace_size(desc(**bad)) == 0, bad
        with pytest.raises(nsa.NsaError):
            nsa.relpos_workspace(desc(**bad), "cpu")
    assert lib.lsrm_relpos_workspace_size(None) == 0
    assert nsa.lsrm_layer_norm_workspace_size(0, 8) > 0
    assert nsa.lsrm_layer_norm_workspace_size(-1, 8) == 0 and nsa.lsrm_layer_norm_workspace_size(8, 0) == 0


def test_relpos_refusals_before_any_launch(lib):
    d = desc()
    n = nsa.lsrm_relpos_workspace_size(d)
    fwd = lambda dd, p, ws=256, size=n: lib.lsrm_relpos_forward(ctypes.byref(dd), *p, ws, size, None)  # noqa: E731
    good = [16] * 11
    assert fwd(desc(head_dim=48), good) == 2
    assert fwd(desc(n_axes=4), good) == 1
    assert fwd(d, good, None) == 6 and fwd(d, good, 128) == 6 and fwd(d, good, 256, n - 1) == 6
    for i in range(10):  # lse may be missing
        assert fwd(d, good[:i] + [None] + good[i + 1:]) == 1, i
    for i in (6, 7, 8, 9):
        assert fwd(d, good[:i] + [24] + good[i + 1:]) == 1, i
    for i in (0, 1, 2, 3, 4, 10):
        assert fwd(d, good[:i] + [18] + good[i + 1:]) == 1, i
    assert fwd(d, good[:5] + [17] + good[6:]) == 1
    assert lib.lsrm_relpos_forward(None, *good, 256, n, None) == 1
    bwd = lambda dd, p, ws=256, size=n: lib.lsrm_relpos_backward(ctypes.byref(dd), *p, ws, size, None)  # noqa: E731
    good = [16] * 16
    assert bwd(d, good, None) == 6 and bwd(d, good, 256, 0) == 6
    for i in range(16):
        assert bwd(d, good[:i] + [None] + good[i + 1:]) == 1, i
    for i in (6, 7, 8, 9, 11, 12, 13, 14):
        assert bwd(d, good[:i] + [24] + good[i + 1:]) == 1, i
    for i in (0, 1, 2, 3, 4, 10):
        assert bwd(d, good[:i] + [18] + good[i + 1:]) == 1, i
    for i in (5, 15):
        assert bwd(d, good[:i] + [17] + good[i + 1:]) == 1, i
    assert lib.lsrm_relpos_workspace_init(ctypes.byref(d), 256, n - 1, None) == 6


def test_layer_norm_refusals_before_any_launch(lib):
    fwd = lib.lsrm_layer_norm_forward
    assert fwd(4, 8, 0, None, None, None, 1e-6, 16, None, None, None) == 1
    assert fwd(4, 8, 0, 16, None, None, 1e-6, None, None, None, None) == 1
    assert fwd(-1, 8, 0, 16, None, None, 1e-6, 16, None, None, None) == 1
    assert fwd(4, 0, 0, 16, None, None, 1e-6, 16, None, None, None) == 1
    assert fwd(4, 8, 2, 16, None, None, 1e-6, 16, None, None, None) == 1
    for eps in (-1.0, math.inf, math.nan):
        assert fwd(4, 8, 0, 16, None, None, eps, 16, None, None, None) == 1
    assert fwd(4, 8, 1, 18, None, None, 1e-6, 16, None, None, None) == 1  # fp32 off its 4 bytes
    assert fwd(0, 8, 0, None, None, None, 1e-6, None, None, None, None) == 0
    bwd = lib.lsrm_layer_norm_backward
    n = nsa.lsrm_layer_norm_workspace_size(4, 8)
    good = [16, 16, None, 16, 16, 16, None, None]
    for i in (0, 1, 3, 4, 5):
        assert bwd(4, 8, 0, *(good[:i] + [None] + good[i + 1:]), 256, n, None) == 1, i
    for i in (3, 4):
        assert bwd(4, 8, 0, *(good[:i] + [18] + good[i + 1:]), 256, n, None) == 1, i
    assert fwd(4, 8, 0, 16, None, None, 1e-6, 16, 18, None, None) == 1
    assert bwd(4, 8, 0, *good, None, n, None) == 6 and bwd(4, 8, 0, *good, 256, n - 1, None) == 6
    assert bwd(4, 8, 0, *good, 128, n, None) == 6


def test_binding_refuses_wrong_tensors():
    d = desc()
    bf, i32 = torch.bfloat16, torch.int32
    t = dict(off_q=torch.zeros(3, dtype=i32), off_k=torch.zeros(3, dtype=i32), pos_q=torch.zeros(100, 1, dtype=i32),
             pos_k=torch.zeros(100, 1, dtype=i32), bucket_of=torch.zeros(257, dtype=i32),
             table=torch.zeros(1, 32, 4, dtype=bf), q=torch.zeros(100, 4, 32, dtype=bf),
             k=torch.zeros(100, 2, 32, dtype=bf), v=torch.zeros(100, 2, 32, dtype=bf),
             out=torch.zeros(100, 4, 32, dtype=bf), lse=torch.zeros(100, 4))
    ws = torch.zeros(256, dtype=torch.uint8)
    call = lambda **kw: nsa.lsrm_relpos_forward(d, **{**t, **kw}, ws=ws)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        call()
    for name, x in t.items():
        with pytest.raises(TypeError, match=name):
            call(**{name: x.double()})
        with pytest.raises(ValueError, match=name):
            call(**{name: x[:-1]})
        if x.dim() > 1 and min(x.shape[:2]) > 1:
            with pytest.raises(ValueError, match=name):
                call(**{name: x.transpose(0, 1).contiguous().transpose(0, 1)})
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        nsa.lsrm_layer_norm_forward(x.double(), None, None, 1e-6, x)
    with pytest.raises(ValueError, match="y"):
        nsa.lsrm_layer_norm_forward(x, None, None, 1e-6, x[:2])
    with pytest.raises(ValueError, match="gamma"):
        nsa.lsrm_layer_norm_forward(x, x[0, :4], None, 1e-6, x)
    with pytest.raises(ValueError, match="CUDA"):
        nsa.lsrm_layer_norm_forward(x, None, None, 1e-6, x)
