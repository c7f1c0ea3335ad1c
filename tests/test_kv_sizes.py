"""Sizes that nc_kv_attention takes and refuses, on the host.  Without a GPU a call
that passes its checks ends at its launch (NC_E_HIP); with one these would launch
on addresses that are not there, so they are skipped."""

import ctypes

import pytest
import torch

from scaled_fp8_casting_amd import _lib
from scaled_fp8_casting_amd._lib import NcKvAttn, NcKvCache

A = 0x10000          # an aligned address that no call reaches
W = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("calls that pass their checks would launch")
    return _lib.load()


def call(lib, heads=8, dim=128, pages=20000, page=16, dtype=1, ws=W, **kw):
    cache = NcKvCache(A, pages, page, heads, dim, _lib.NC_E2M1)
    f = dict(q=A, q_token_stride=4096, q_head_stride=dim, out=A, out_token_stride=4096, out_head_stride=dim, lse=A,
             lse_token_stride=32, q_start=A, kv_len=A, table=A, table_pages=2, batch=1, total_q=3, q_heads=4 * heads, max_q=3,
             max_kv=32, causal=1, window=0, scale=0.125)
    f.update(kw)
    need = lib.nc_kv_workspace_bytes(ctypes.byref(cache), dtype, f["q_heads"], f["batch"], f["max_q"], f["max_kv"])
    size = need if ws is None else ws
    return lib.nc_kv_attention(ctypes.byref(cache), ctypes.byref(NcKvAttn(**f)), dtype, A if size else None, size, None)


# one prompt among single tokens; single tokens of many sequences that may be long, of more that are short; a
# few queries of so many that a thread block for each row would pass a launch's threads
SERVED = [dict(batch=128, max_q=32768, max_kv=32768), dict(batch=4096, max_q=1, max_kv=1 << 20),
          dict(batch=64, max_q=1, max_kv=2 ** 31 - 1, table_pages=1 << 16), dict(batch=1 << 19, max_q=1, max_kv=100),
          dict(batch=1 << 16, max_q=16, max_kv=4096), dict(batch=1 << 16, max_q=15, max_kv=8192)]


@pytest.mark.parametrize("kw", SERVED)
@pytest.mark.parametrize("window", [0, 1000, 5000])
def test_served(lib, kw, window):
    """With the workspace that is asked for."""
    assert call(lib, ws=None, window=window, **kw) == _lib.NC_E_HIP


def test_launches_that_are_too_large(lib):
    assert call(lib, batch=1 << 21, max_q=1, max_kv=100) == _lib.NC_E_ARG
    assert call(lib, batch=1 << 20, max_q=16, max_kv=100) == _lib.NC_E_ARG


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.5e38])
def test_scales_that_32_bits_do_not_hold(lib, scale):
    """Scores are counted in powers of two: scale * log2(e) has to be finite."""
    assert call(lib, scale=scale) == _lib.NC_E_ARG
    assert call(lib, scale=2.3e38) == _lib.NC_E_HIP
