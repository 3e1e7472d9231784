"""Host side of the layer norm: rows of more elements than the kernels' 32-bit column counters reach, and more rows
than a grid has CTAs, are refused (no call here launches anything)."""
import pytest
import torch

from block_sparse_gqa_nsa_b200 import nsa
from block_sparse_gqa_nsa_b200.build import build

MOST = 2 ** 30


@pytest.fixture(scope="module")
def lib():
    build()
    return nsa.load_library()


@pytest.mark.timeout(60)
@pytest.mark.parametrize("width", [MOST + 1, 2 ** 31 - 9, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype", [0, 1])
def test_widest_rows(lib, width, dtype):
    assert lib.lsrm_layer_norm_forward(1, width, dtype, 16, None, None, 1e-6, 16, None, None, None) == 2
    assert lib.lsrm_layer_norm_backward(1, width, dtype, 16, 16, None, 16, 16, 16, None, None, 256, 2 ** 60, None) == 2
    assert nsa.lsrm_layer_norm_workspace_size(1, width) == 0
    with pytest.raises(nsa.NsaError):
        nsa.layer_norm_workspace(1, width, "meta")
    assert nsa.lsrm_layer_norm_workspace_size(1, MOST) > 0


@pytest.mark.parametrize("rows", [2 ** 40 + 1, 2 ** 62, 2 ** 63 - 1])
def test_most_rows(lib, rows):
    assert lib.lsrm_layer_norm_forward(rows, 8, 0, 16, None, None, 1e-6, 16, None, None, None) == 2
    assert lib.lsrm_layer_norm_backward(rows, 8, 0, 16, 16, None, 16, 16, 16, None, None, 256, 2 ** 60, None) == 2
    assert nsa.lsrm_layer_norm_workspace_size(rows, 8) == 0


def test_no_rows_of_any_width(lib):
    assert lib.lsrm_layer_norm_forward(0, MOST, 0, None, None, None, 1e-6, None, None, None, None) == 0


@pytest.mark.parametrize("make", [lambda device: nsa.layer_norm_workspace(4, 8, device),
                                  lambda device: nsa.relpos_workspace(nsa.make_relpos_desc(4, 4, 1, 2, 2, 32, 1, 8, 8),
                                                                      device)])
def test_workspaces_are_made_on_the_device_that_was_named(lib, make, monkeypatch):
    """Device 0 by its number is that device, not the current one."""
    asked = []

    def empty(n, dtype, device):
        asked.append(device)
        return torch.zeros(n, dtype=dtype)

    monkeypatch.setattr(nsa.torch, "empty", empty)
    monkeypatch.setattr(nsa, "lsrm_relpos_workspace_init", lambda *a: None)
    for given, want in ((0, 0), (1, 1), (None, "cuda"), ("cuda:1", "cuda:1")):
        make(given)
        assert asked[-1] == want, given
