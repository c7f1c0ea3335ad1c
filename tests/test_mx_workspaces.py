"""What the products ask for as workspace, on the host."""

import ctypes

import pytest

from scaled_fp8_casting_amd import _lib
from scaled_fp8_casting_amd._lib import NcMxMatrix

A = 0x10000


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


@pytest.mark.parametrize("fmt", [_lib.NC_E4M3, _lib.NC_E5M2, _lib.NC_E2M1])
@pytest.mark.parametrize("n,k", [(4096, 4096), (11008, 4096), (130, 20000), (1, 1 << 20), (70, 100)])
def test_rows_that_the_product_quantises_need_none(lib, n, k, fmt):
    """Up to 8 rows of a linear layer are quantised by the product itself, which cuts no sum along the columns."""
    w = NcMxMatrix(A, n, k, _lib.NC_E2M1, 0)
    for rows in range(9):
        assert lib.nc_mx_workspace_bytes(ctypes.byref(w), rows, fmt) == 0
    assert lib.nc_mx_workspace_bytes(ctypes.byref(w), 9, fmt) >= lib.nc_mx_bytes(9, k, fmt)
