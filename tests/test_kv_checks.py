"""The key/value cache's refusals, at the C-ABI and in the binding, sizes, and
pins of its oracle.  Nothing here launches a kernel: every call fails its checks
(or is empty) first, so these run without a GPU."""

import ctypes

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc
from oracle import E4M3, bulk, kv
from scaled_fp8_casting_amd import _lib
from scaled_fp8_casting_amd._lib import NcKvAttn, NcKvCache, NcKvRows

A = 0x10000          # an aligned address that no call reaches
W = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def cache(**kw):
    f = dict(data=A, pages=4, page=16, heads=2, dim=64, fmt=_lib.NC_E2M1)
    f.update(kw)
    return ctypes.byref(NcKvCache(**f))


def rows(p=A, ts=128, hs=64):
    return ctypes.byref(NcKvRows(p, ts, hs))


BAD_CACHES = [
    (dict(fmt=_lib.NC_E5M2), _lib.NC_E_UNSUPPORTED), (dict(fmt=3), _lib.NC_E_UNSUPPORTED),
    (dict(dim=32), _lib.NC_E_UNSUPPORTED), (dict(dim=80), _lib.NC_E_UNSUPPORTED), (dict(dim=0), _lib.NC_E_UNSUPPORTED),
    (dict(page=0), _lib.NC_E_SHAPE), (dict(page=8), _lib.NC_E_SHAPE), (dict(page=-16), _lib.NC_E_SHAPE),
    (dict(pages=-1), _lib.NC_E_ARG), (dict(heads=0), _lib.NC_E_ARG), (dict(data=None), _lib.NC_E_ARG),
    (dict(pages=1 << 28, heads=1), _lib.NC_E_ARG), (dict(pages=1 << 40), _lib.NC_E_ARG),
    (dict(pages=1 << 26, heads=64), _lib.NC_E_ARG), (dict(data=A + 8), _lib.NC_E_ALIGN),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_caches(lib, kw, status):
    one = cache(**kw)
    assert lib.nc_kv_write(one, rows(), rows(), 5, 1, A, 2, None) == status
    assert lib.nc_kv_read(one, rows(), rows(), 5, 1, A, None) == status
    assert lib.nc_kv_attention(one, ctypes.byref(attn()), 1, A, W, None) == status
    if "data" not in kw:
        f = dict(pages=4, page=16, heads=2, dim=64, fmt=_lib.NC_E2M1)
        f.update(kw)
        assert lib.nc_kv_cache_bytes(f["pages"], f["page"], f["heads"], f["dim"], f["fmt"]) == 0


def test_write_and_read(lib):
    ok, none = cache(), None
    for call in (lambda c, k, v, n, dt, s: lib.nc_kv_write(c, k, v, n, dt, s, 2, None),
                 lambda c, k, v, n, dt, s: lib.nc_kv_read(c, k, v, n, dt, s, None)):
        assert call(none, rows(), rows(), 1, 1, A) == _lib.NC_E_ARG
        assert call(ok, none, rows(), 1, 1, A) == _lib.NC_E_ARG
        assert call(ok, rows(), none, 1, 1, A) == _lib.NC_E_ARG
        assert call(ok, rows(), rows(), 1, 1, None) == _lib.NC_E_ARG
        assert call(ok, rows(None), rows(), 1, 1, A) == _lib.NC_E_ARG
        assert call(ok, rows(), rows(), -1, 1, A) == _lib.NC_E_ARG
        assert call(ok, rows(), rows(), 1 << 32, 1, A) == _lib.NC_E_ARG
        assert call(ok, rows(), rows(ts=-128), 1, 1, A) == _lib.NC_E_ARG
        assert call(ok, rows(), rows(), 1, 2, A) == _lib.NC_E_UNSUPPORTED
        assert call(ok, rows(A + 8), rows(), 1, 1, A) == _lib.NC_E_ALIGN
        assert call(ok, rows(), rows(ts=100), 1, 1, A) == _lib.NC_E_ALIGN
        assert call(ok, rows(), rows(hs=68), 1, 1, A) == _lib.NC_E_ALIGN
        assert call(ok, rows(), rows(hs=66), 1, 0, A) == _lib.NC_E_ALIGN
        assert call(ok, rows(), rows(), 1, 1, A + 4) == _lib.NC_E_ALIGN
        assert call(ok, none, none, 0, 1, None) == _lib.NC_OK
    assert lib.nc_kv_write(ok, rows(), rows(), 1, 1, A, 3, None) == _lib.NC_E_UNSUPPORTED
    # slots of an empty cache can be given; there is nothing to reach
    assert lib.nc_kv_write(cache(pages=0, data=None), none, none, 0, 1, None, 2, None) == _lib.NC_OK


def attn(**kw):
    f = dict(q=A, q_token_stride=256, q_head_stride=64, out=A, out_token_stride=256, out_head_stride=64, lse=A,
             lse_token_stride=4, q_start=A, kv_len=A, table=A, table_pages=2, batch=1, total_q=3, q_heads=4, max_q=3,
             max_kv=32, causal=1, window=0, scale=0.125)
    f.update(kw)
    return NcKvAttn(**f)


BAD_CALLS = [
    (dict(q=None), _lib.NC_E_ARG), (dict(out=None), _lib.NC_E_ARG), (dict(q_start=None), _lib.NC_E_ARG),
    (dict(kv_len=None), _lib.NC_E_ARG), (dict(table=None), _lib.NC_E_ARG), (dict(batch=-1), _lib.NC_E_ARG),
    (dict(total_q=-1), _lib.NC_E_ARG), (dict(max_q=-1), _lib.NC_E_ARG), (dict(max_kv=-1), _lib.NC_E_ARG),
    (dict(window=-1), _lib.NC_E_ARG), (dict(table_pages=-1), _lib.NC_E_ARG), (dict(q_heads=0), _lib.NC_E_ARG),
    (dict(scale=float("nan")), _lib.NC_E_ARG), (dict(scale=float("inf")), _lib.NC_E_ARG),
    (dict(q_token_stride=-256), _lib.NC_E_ARG), (dict(lse_token_stride=-1), _lib.NC_E_ARG),
    (dict(q_heads=3), _lib.NC_E_SHAPE), (dict(q=A + 4), _lib.NC_E_ALIGN), (dict(out_head_stride=65), _lib.NC_E_ALIGN),
    (dict(lse=A + 2), _lib.NC_E_ALIGN), (dict(kv_len=A + 1), _lib.NC_E_ALIGN),
    (dict(max_q=1 << 30), _lib.NC_E_ARG), (dict(batch=1 << 30), _lib.NC_E_ARG),
]


@pytest.mark.parametrize("kw,status", BAD_CALLS)
def test_attention(lib, kw, status):
    assert lib.nc_kv_attention(cache(), ctypes.byref(attn(**kw)), 1, A, W, None) == status


def test_attention_rest(lib):
    assert lib.nc_kv_attention(None, ctypes.byref(attn()), 1, A, W, None) == _lib.NC_E_ARG
    assert lib.nc_kv_attention(cache(), None, 1, A, W, None) == _lib.NC_E_ARG
    assert lib.nc_kv_attention(cache(), ctypes.byref(attn()), 2, A, W, None) == _lib.NC_E_UNSUPPORTED
    for kw in (dict(batch=0), dict(max_q=0), dict(total_q=0)):
        assert lib.nc_kv_attention(cache(), ctypes.byref(attn(**kw)), 1, None, 0, None) == _lib.NC_OK


@pytest.mark.parametrize("batch,max_q,max_kv,heads", [(1, 1, 262144, 8), (1, 1, 9000, 1), (3, 7, 40000, 2)])
def test_workspace(lib, batch, max_q, max_kv, heads):
    """A call that splits its keys needs the workspace, whatever its window; smaller ones fit in it."""
    c = cache(pages=20000, heads=heads)
    need = lib.nc_kv_workspace_bytes(c, 1, 4 * heads, batch, max_q, max_kv)
    assert need > 0
    kw = dict(batch=batch, max_q=max_q, max_kv=max_kv, q_heads=4 * heads)
    for ws, size in ((None, W), (A, 0), (A + 8, W)):
        assert lib.nc_kv_attention(c, ctypes.byref(attn(**kw)), 1, ws, size, None) == _lib.NC_E_WORKSPACE
    for m in (max_kv // 2, max_kv // 7, 100, 0):
        assert lib.nc_kv_workspace_bytes(c, 1, 4 * heads, batch, max_q, m) <= need
    assert lib.nc_kv_workspace_bytes(c, 1, 4 * heads, 0, max_q, max_kv) == 0
    assert lib.nc_kv_workspace_bytes(c, 1, 0, batch, max_q, max_kv) == 0
    assert lib.nc_kv_workspace_bytes(cache(), 1, 3, batch, max_q, max_kv) == 0      # not a multiple of two heads
    assert lib.nc_kv_workspace_bytes(c, 5, 4 * heads, batch, max_q, max_kv) == 0


def test_struct_sizes():
    assert ctypes.sizeof(NcKvCache) == 32
    assert ctypes.sizeof(NcKvRows) == 24
    assert ctypes.sizeof(NcKvAttn) == 128


@pytest.mark.parametrize("fmt,bits", [("e2m1", 4), ("e4m3", 8)])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_bytes(lib, fmt, bits, dim):
    """A token and head: its codes and one byte for 32 of them, for the key and the value."""
    assert nc.kv_page_bytes(48, 3, dim, fmt) == 48 * 3 * 2 * (dim * bits // 8 + dim // 32)
    assert lib.nc_kv_cache_bytes(7, 48, 3, dim, nc.KV_FMT[fmt]) == 7 * nc.kv_page_bytes(48, 3, dim, fmt)


# -- the binding --------------------------------------------------------------

def host(fmt="e2m1", heads=2, dim=64, pages=4, page=16):
    return nc.new_kv_cache(pages, page, heads, dim, fmt, device="cpu")


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("args", [(4, 16, 2, 64, "e5m2"), (4, 8, 2, 64, "e2m1"), (4, 16, 0, 64, "e2m1"),
                                  (4, 16, 2, 80, "e2m1"), (4, 0, 2, 64, "e2m1"), (4, 16, 2, 64, "E2M1")])
def test_new_cache_refuses(args):
    with pytest.raises(ValueError):
        nc.new_kv_cache(*args, device="cpu")


def test_cache_over_given_memory():
    each = nc.kv_page_bytes(16, 2, 64, "e2m1")
    nc.KvCache(torch.zeros((3, each), dtype=torch.uint8), 16, 2, 64, "e2m1")
    for data in (torch.zeros((3, each + 1), dtype=torch.uint8), torch.zeros(3 * each, dtype=torch.uint8),
                 torch.zeros((3, each), dtype=torch.int8), torch.zeros((each, 3), dtype=torch.uint8).T):
        with pytest.raises(ValueError, match="data: shape"):
            nc.KvCache(data, 16, 2, 64, "e2m1")


def test_binding_write_and_read():
    c, s = host(), torch.arange(5)
    for call in (nc.nc_kv_write, lambda c, k, v, s: nc.nc_kv_read(c, s, k, v)):
        with pytest.raises(ValueError, match="k: shape"):
            call(c, bf16(4, 2, 64), bf16(5, 2, 64), s)
        with pytest.raises(ValueError, match="v: shape"):
            call(c, bf16(5, 2, 64), bf16(5, 3, 64), s)
        with pytest.raises(ValueError, match="v: .*float32"):
            call(c, bf16(5, 2, 64), bf16(5, 2, 64).float(), s)
        with pytest.raises(TypeError):
            call(c, bf16(5, 2, 64).half(), bf16(5, 2, 64).half(), s)
        with pytest.raises(ValueError, match="slots: .*int32"):
            call(c, bf16(5, 2, 64), bf16(5, 2, 64), s.int())
        with pytest.raises(ValueError, match="slots: shape"):
            call(c, bf16(5, 2, 64), bf16(5, 2, 64), s[:, None])
        with pytest.raises(ValueError, match="k: strides"):
            call(c, bf16(5, 2, 65)[..., 1:], bf16(5, 2, 64), s)
        with pytest.raises(ValueError, match="k: strides"):
            call(c, bf16(5, 2, 128)[..., ::2], bf16(5, 2, 64), s)
        with pytest.raises(ValueError, match="device tensor expected"):
            call(c, bf16(5, 2, 64), bf16(5, 2, 64), s)
    with pytest.raises(ValueError, match="k: strides.*overlap"):
        nc.nc_kv_read(c, s, bf16(1, 2, 64).expand(5, 2, 64), bf16(5, 2, 64))
    with pytest.raises(KeyError):
        nc.nc_kv_write(c, bf16(5, 2, 64), bf16(5, 2, 64), s, "floor")


def test_binding_attention():
    c = host()
    good = dict(q=bf16(3, 4, 64), out=bf16(3, 4, 64), q_start=i32(0, 1, 3), kv_len=i32(9, 9),
                table=torch.zeros((2, 2), dtype=torch.int32), max_q=2, max_kv=9)
    call = lambda **kw: nc.nc_kv_attention(c, **{**good, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="device tensor expected"):
        call()
    for kw, match in ((dict(q=bf16(3, 3, 64)), "q: 3 heads"), (dict(q=bf16(3, 4, 96)), "q: shape"),
                      (dict(q=bf16(12, 64)), "q: shape"), (dict(out=bf16(2, 4, 64)), "out: shape"),
                      (dict(out=bf16(3, 4, 64).float()), "out: .*float32"), (dict(out=bf16(3, 1, 64).expand(3, 4, 64)), "overlap"),
                      (dict(q_start=i32(0, 3)), "q_start"), (dict(q_start=torch.tensor([0, 1, 3])), "q_start: .*int64"),
                      (dict(kv_len=torch.tensor([9, 9])), "kv_len: .*int64"), (dict(table=torch.zeros((2, 2))), "table: shape"),
                      (dict(table=torch.zeros((3, 2), dtype=torch.int32)), "table: shape"),
                      (dict(max_q=-1), "negative"), (dict(window=-1), "negative"), (dict(scale=float("nan")), "scale"),
                      (dict(lse=torch.zeros(3, 3)), "lse: shape"), (dict(lse=torch.zeros(4, 3).T), "lse: shape"),
                      (dict(ws=torch.zeros(4)), "ws: dtype")):
        with pytest.raises(ValueError, match=match):
            call(**kw)
    with pytest.raises(TypeError):
        call(q=bf16(3, 4, 64).half())


# -- the oracle -----------------------------------------------------------------

@pytest.mark.parametrize("rule", ["ocp", "plus1", "ceil"])
def test_held_e4m3_is_the_mx_cast(rule):
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((64, 96)) * 2.0 ** rng.integers(-40, 40, (64, 1))).astype(np.float32).astype(np.float64)
    codes, scales, _ = bulk.cast_mx_f64(E4M3, x.ravel(), 96, rule)
    want = bulk.represented_f64(E4M3, codes, np.repeat(127 - scales.astype(np.int64), 32)).reshape(x.shape)
    assert np.array_equal(want, kv.held(x, "e4m3", rule))


def test_held_e2m1_by_hand():
    row = np.zeros((1, 32))
    row[0, :12] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.2, 0.3, -5, -0.25]
    held = [6, 4, 4, 2, 2, 1, 1, 0, 0, 0.5, -4, -0.0]        # ties to the even code
    got = kv.held(row, "e2m1", "ocp")                         # a = 6 = 1.5 2^2: X = 0
    assert got[0, :12].tolist() == held and np.signbit(got[0, 11])
    row[0, 0] = 7                                             # 7 = 1.75 2^2: ocp saturates, ceil takes X = 1
    assert kv.held(row, "e2m1", "ocp")[0, 0] == 6
    assert kv.held(row, "e2m1", "ceil")[0, :4].tolist() == [8, 4, 4, 2]
    assert kv.held(row, "e2m1", "plus1")[0, :4].tolist() == [8, 4, 4, 2]
    row[0, 3] = np.nan
    assert np.isnan(kv.held(row, "e2m1", "ocp")).all()


def test_seen_and_attend():
    assert kv.seen(3, 2, True, 0).tolist() == [[True, True, False], [True, True, True]]
    assert kv.seen(3, 2, True, 2).tolist() == [[True, True, False], [False, True, True]]
    assert kv.seen(2, 3, True, 0).tolist() == [[False, False], [True, False], [True, True]]
    assert kv.seen(2, 1, False, 0).tolist() == [[True, True]]
    q, k, v = np.array([[1.0, 0]]), np.array([[np.log(3), 5], [0, 7]]), np.array([[1.0], [5]])
    out, lse, spread, reach = kv.attend(q, k, v, np.array([[True, True]]), 1.0)
    assert np.allclose(out, 2) and np.allclose(lse, np.log(4)) and np.allclose(spread, 2) and np.allclose(reach, np.log(3))
    out, lse, _, _ = kv.attend(q, k, v, np.array([[False, False]]), 1.0)
    assert out[0, 0] == 0 and np.isneginf(lse[0])


@pytest.mark.parametrize("dim", (64, 192, 256))
@pytest.mark.parametrize("dtype", (0, 1))
def test_workspace_serves_smaller_calls(lib, dtype, dim):
    """One workspace for the largest sizes is enough whichever of them shrink, also where the largest call itself
    does not split its keys."""
    c = cache(pages=40000, heads=4, dim=dim)
    grid = [(b, q, n) for b in (1, 3, 16, 32, 200) for q in (1, 3, 9, 100, 4096) for n in (0, 40, 2048, 2100, 4100, 65536)]
    need = {at: lib.nc_kv_workspace_bytes(c, dtype, 16, *at) for at in grid}
    for large in grid:
        for small in grid:
            if all(x <= y for x, y in zip(small, large)):
                assert need[small] <= need[large], (small, large)
    assert need[200, 4096, 40] == 0 and need[1, 1, 65536] > 0
