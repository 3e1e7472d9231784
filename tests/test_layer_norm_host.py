"""Host side of the layer norm: rows of more elements than the kernels' 32-bit column counters reach, and more rows
than a grid has CTAs, are refused (no call here launches anything)."""
import pytest

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
