"""Layer norm on the GPU against its definition in 64 bits: both directions, both types, widths that
take every kernel variant, unaligned rows, in place, no rows, captured graphs."""
import pytest
import torch

from block_sparse_gqa_nsa_b200 import nsa
import relpos_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(rows, width, dtype, seed=0, shift=0.5):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g) * std + mean).to(dtype).cuda()

    return (normal(rows, width, std=1.5, mean=shift), normal(width, std=0.2, mean=1.0), normal(width, std=0.2),
            normal(rows, width))


def both(x, gamma, beta, dy, eps=EPS):
    rows, width = x.numel() // x.shape[-1], x.shape[-1]
    y = torch.full_like(x, float("nan"))
    mean, rstd = torch.full((2, rows), float("nan"), device="cuda").unbind(0)
    nsa.lsrm_layer_norm_forward(x, gamma, beta, eps, y, mean, rstd)
    dx = torch.full_like(x, float("nan"))
    dgamma, dbeta = (torch.full((width,), float("nan"), dtype=x.dtype, device="cuda") for _ in range(2))
    nsa.lsrm_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, nsa.layer_norm_workspace(rows, width))
    got = {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    want = {**ref.layer_norm(x, gamma, beta, eps), **ref.layer_norm(x, gamma, beta, eps, dy, (mean, rstd))}
    for n in got:
        ref.check(n, got[n], want[n])
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width", [
    (1, 1), (1, 8), (3, 2), (5, 4), (9, 8), (7, 16), (1, 32), (1000, 32), (513, 64), (33, 96), (20, 128), (70, 256),
    (9, 257), (31, 509), (5, 512), (65, 1000), (40, 1024), (3, 1025), (12, 1536), (4, 2048), (3, 2047), (2, 4096),
    (3, 4104), (2, 5001), (1, 8192), (2, 8200), (3, 8193), (1, 20000), (200, 12000), (5000, 40)])
def test_both_directions(rows, width, dtype):
    both(*make(rows, width, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_rows(dtype):
    x, gamma, beta, dy = make(37, 64, dtype)

    def moved(t):  # the same values one element past a 16-byte border
        s = torch.empty(t.numel() + 1, dtype=dtype, device="cuda")[1:].view(t.shape)
        return s.copy_(t)

    both(moved(x), gamma, beta, dy)
    both(x, moved(gamma), beta, moved(dy))


def test_without_weights_and_statistics():
    x, gamma, beta, dy = make(50, 96, torch.bfloat16)
    both(x, None, None, dy)
    both(x, gamma, None, dy)
    a = torch.empty_like(x)
    b = torch.empty_like(x)
    mean, rstd = torch.empty(2, 50, device="cuda").unbind(0)
    nsa.lsrm_layer_norm_forward(x, gamma, beta, EPS, a)
    nsa.lsrm_layer_norm_forward(x, gamma, beta, EPS, b, mean, rstd)
    assert torch.equal(a, b)
    dx, dx2 = torch.empty_like(x), torch.empty_like(x)
    dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(beta)
    ws = nsa.layer_norm_workspace(50, 96)
    nsa.lsrm_layer_norm_backward(dy, x, gamma, mean, rstd, dx, None, None, ws)
    nsa.lsrm_layer_norm_backward(dy, x, gamma, mean, rstd, dx2, dgamma, None, ws)
    assert torch.equal(dx, dx2)
    want = ref.layer_norm(x, gamma, beta, EPS, dy, (mean, rstd))
    ref.check("dgamma", dgamma, want["dgamma"])
    nsa.lsrm_layer_norm_backward(dy, x, gamma, mean, rstd, dx2, None, dbeta, ws)
    ref.check("dbeta", dbeta, want["dbeta"])


@pytest.mark.parametrize("width", [32, 1024, 1031, 4096, 9000])
def test_in_place(width):
    x, gamma, beta, dy = make(300, width, torch.bfloat16)
    got = both(x, gamma, beta, dy)
    y = x.clone()
    nsa.lsrm_layer_norm_forward(y, gamma, beta, EPS, y)
    assert torch.equal(y, got["y"])
    ws = nsa.layer_norm_workspace(300, width)
    for over in (x.clone(), dy.clone()):
        xx, dd = (over, dy) if torch.equal(over, x) else (x, over)
        dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(beta)
        nsa.lsrm_layer_norm_backward(dd, xx, gamma, got["mean"], got["rstd"], over, dgamma, dbeta, ws)
        assert torch.equal(over, got["dx"]) and torch.equal(dgamma, got["dgamma"]) and torch.equal(dbeta, got["dbeta"])


def test_constant_and_large_rows():
    """A constant row has xh = 0 exactly; an offset much larger than the spread keeps the two-pass variance."""
    x = torch.full((4, 512), 3.0, device="cuda")
    y, beta = torch.empty_like(x), torch.randn(512, device="cuda")
    nsa.lsrm_layer_norm_forward(x, None, beta, EPS, y)
    assert torch.equal(y, beta.expand_as(y))
    x, gamma, beta, dy = make(64, 512, torch.float32, shift=100.0)
    both(x, gamma, beta, dy)


def test_no_rows_and_many_rows():
    x, gamma, beta, dy = make(0, 64, torch.bfloat16)
    dgamma, dbeta = torch.ones_like(gamma), torch.ones_like(beta)
    none = torch.empty(0, device="cuda")
    nsa.lsrm_layer_norm_forward(x, gamma, beta, EPS, torch.empty_like(x), none, none)
    nsa.lsrm_layer_norm_backward(dy, x, gamma, none, none, torch.empty_like(x), dgamma, dbeta,
                                 nsa.layer_norm_workspace(0, 64))
    assert not dgamma.any() and not dbeta.any()
    both(*make(300001, 32, torch.bfloat16))


def test_reproducible_captured_and_shaped():
    x, gamma, beta, dy = make(6000, 64, torch.bfloat16)
    a, b = both(x, gamma, beta, dy), both(x, gamma, beta, dy)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    heads, dheads = x.view(1000, 6, 64), dy.view(1000, 6, 64)
    y, dx, dgamma, dbeta = torch.empty_like(heads), torch.empty_like(heads), torch.empty_like(gamma), torch.empty_like(beta)
    mean, rstd = torch.empty(2, 6000, device="cuda").unbind(0)
    ws = nsa.layer_norm_workspace(6000, 64)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        nsa.lsrm_layer_norm_forward(heads, gamma, beta, EPS, y, mean, rstd)
        nsa.lsrm_layer_norm_backward(dheads, heads, gamma, mean, rstd, dx, dgamma, dbeta, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y.view(6000, 64), a["y"]) and torch.equal(dx.view(6000, 64), a["dx"])
    assert torch.equal(dgamma, a["dgamma"]) and torch.equal(dbeta, a["dbeta"])
