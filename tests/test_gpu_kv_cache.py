"""nc_kv_write and nc_kv_read against the definition, value for value."""

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc
from oracle import kv
from tests._kv import DT, f64, rounded, stale

pytestmark = pytest.mark.gpu


def values(rng, tokens, heads, dim, dtype):
    """Rows with wide block scales, grid midpoints, zeros of both signs and zero blocks."""
    x = rng.standard_normal((tokens, heads, dim)) * 2.0 ** rng.integers(-30, 30, (tokens, heads, dim // 32, 1)) \
        .repeat(32, -1).reshape(tokens, heads, dim)
    pick = rng.random(x.shape)
    x = np.where(pick < 0.1, np.round(x * 4) / 4, x)
    x = np.where((pick > 0.1) & (pick < 0.15), -0.0, x)
    if tokens:
        x[0, 0, :32] = 0
    return rounded(x, dtype)


def same(got, want):
    got, want = f64(got) if isinstance(got, torch.Tensor) else got, np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = np.isnan(want) | ((got == want) & (np.signbit(got) == np.signbit(want)))
    assert ok.all(), (np.argwhere(~ok)[:4], got[~ok][:4], want[~ok][:4])


def as_dtype(v, dtype):
    """Binary64 held values in an output type, rounded to nearest even."""
    with np.errstate(over="ignore"):
        return f64(torch.from_numpy(np.asarray(v)).to(DT[dtype]))


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype,rule", [("bf16", "ceil"), ("bf16", "ocp"), ("fp32", "plus1"), ("fp32", "ceil")])
def test_round_trip(fmt, dtype, rule, dim):
    rng = np.random.default_rng(dim + len(rule))
    page, heads, tokens, pages = 48, 3, 133, 5
    cache = nc.new_kv_cache(pages, page, heads, dim, fmt)
    slots = rng.permutation(pages * page)[:tokens]
    k, v = values(rng, tokens, heads, dim, dtype), values(rng, tokens, heads, dim, dtype)
    s = torch.from_numpy(slots).cuda()
    nc.nc_kv_write(cache, k.cuda(), v.cuda(), s, rule)
    for out in ("fp32", "bf16"):
        ko = torch.full(k.shape, 3.0, dtype=DT[out], device="cuda")
        vo = torch.full_like(ko, 3.0)
        nc.nc_kv_read(cache, s, ko, vo)
        same(ko, as_dtype(kv.held(f64(k), fmt, rule), out))
        same(vo, as_dtype(kv.held(f64(v), fmt, rule), out))
    # every slot that was not written reads as zero
    rest = np.setdiff1d(np.arange(pages * page), slots)
    ko = torch.full((len(rest), heads, dim), 3.0, device="cuda")
    vo = torch.full_like(ko, 3.0)
    nc.nc_kv_read(cache, torch.from_numpy(rest).cuda(), ko, vo)
    assert not ko.any() and not vo.any()


@pytest.mark.parametrize("fmt,dim", [("e2m1", 96), ("e2m1", 192), ("e4m3", 96), ("e4m3", 128)])
def test_a_token_is_written_alone(fmt, dim):
    """Rewriting single tokens leaves their neighbours, and slots outside the cache are skipped."""
    rng = np.random.default_rng(3)
    page, heads, pages = 16, 2, 3
    cache = nc.new_kv_cache(pages, page, heads, dim, fmt)
    every = torch.arange(pages * page, device="cuda")
    k, v = values(rng, pages * page, heads, dim, "bf16"), values(rng, pages * page, heads, dim, "bf16")
    nc.nc_kv_write(cache, k.cuda(), v.cuda(), every)
    for at in (0, 17, 47):
        k[at], v[at] = values(rng, 1, heads, dim, "bf16")[0], values(rng, 1, heads, dim, "bf16")[0]
        nc.nc_kv_write(cache, k[at:at + 1].cuda(), v[at:at + 1].cuda(), every[at:at + 1])
    off = torch.tensor([-1, pages * page, 2 ** 40, -2 ** 62], device="cuda")
    junk = torch.full((4, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    nc.nc_kv_write(cache, junk, junk, off)
    ko, vo = torch.empty_like(k, device="cuda"), torch.empty_like(v, device="cuda")
    nc.nc_kv_read(cache, every, ko, vo)
    same(ko, as_dtype(kv.held(f64(k), fmt, "ceil"), "bf16"))
    same(vo, as_dtype(kv.held(f64(v), fmt, "ceil"), "bf16"))
    ko, vo = junk.clone(), junk.clone()
    nc.nc_kv_read(cache, off, ko, vo)
    assert not ko.any() and not vo.any()


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("tokens,heads,page", [(1, 1, 16), (7, 8, 64), (1025, 1, 128), (259, 5, 16)])
def test_strides(fmt, tokens, heads, page):
    """Keys and values as slices of a fused projection; outputs with the heads outermost."""
    rng = np.random.default_rng(tokens)
    dim = 128
    pages = -(-tokens // page) + 1
    cache = nc.new_kv_cache(pages, page, heads, dim, fmt)
    rows = values(rng, tokens, 3 * heads, dim, "bf16").cuda()
    slots = torch.arange(pages * page - tokens, pages * page, device="cuda")
    nc.nc_kv_write(cache, rows[:, heads:2 * heads], rows[:, 2 * heads:], slots, "ocp")
    ko = torch.empty((heads, tokens, dim), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    vo = torch.empty((tokens, 2, heads, dim), dtype=torch.bfloat16, device="cuda")
    nc.nc_kv_read(cache, slots, ko, vo[:, 1])
    same(ko, as_dtype(kv.held(f64(rows[:, heads:2 * heads]), fmt, "ocp"), "bf16"))
    same(vo[:, 1], as_dtype(kv.held(f64(rows[:, 2 * heads:]), fmt, "ocp"), "bf16"))


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("rule", ["ocp", "plus1", "ceil"])
def test_extremes(fmt, rule):
    """Every scale byte, fp32's subnormals and largest numbers, infinities, NaN."""
    rng = np.random.default_rng(11)
    dim, heads = 64, 1
    with np.errstate(over="ignore"):
        x = np.concatenate([rng.uniform(-2, 2, (1, 64)) * 2.0 ** e for e in range(-149, 128)]).astype(np.float32)
    x = np.clip(x, -np.finfo(np.float32).max, np.finfo(np.float32).max)
    special = np.tile(rng.standard_normal((6, 64)).astype(np.float32), (1, 1))
    special[0, 3], special[1, 40], special[2, 5] = np.inf, -np.inf, np.nan
    special[3, 32:] = np.inf
    special[4, :32] = -0.0
    special[5, 1], special[5, 2] = np.nan, np.inf
    x = np.concatenate([x, special])[:, None, :]
    t = torch.from_numpy(x).cuda()
    cache = nc.new_kv_cache(20, 16, heads, dim, fmt)
    slots = torch.arange(len(x), device="cuda")
    nc.nc_kv_write(cache, t, t.flip(-1).contiguous(), slots, rule)
    ko, vo = torch.empty_like(t), torch.empty_like(t)
    nc.nc_kv_read(cache, slots, ko, vo)
    want = kv.held(x.astype(np.float64), fmt, rule)
    flip = kv.held(x[..., ::-1].astype(np.float64), fmt, rule)
    same(ko, as_dtype(want, "fp32"))
    same(vo, as_dtype(flip, "fp32"))


def test_pages_are_rows():
    """A page copied as a row of the data holds the same tokens."""
    rng = np.random.default_rng(5)
    cache = nc.new_kv_cache(4, 32, 2, 96, "e2m1")
    stale(cache, rng)
    k, v = values(rng, 32, 2, 96, "bf16").cuda(), values(rng, 32, 2, 96, "bf16").cuda()
    nc.nc_kv_write(cache, k, v, torch.arange(64, 96, device="cuda"))
    cache.data[0].copy_(cache.data[2])
    a, b, c, d = (torch.empty_like(k) for _ in range(4))
    nc.nc_kv_read(cache, torch.arange(32, device="cuda"), a, b)
    nc.nc_kv_read(cache, torch.arange(64, 96, device="cuda"), c, d)
    assert torch.equal(a, c) and torch.equal(b, d)


def test_empty_and_stream():
    cache = nc.new_kv_cache(2, 16, 1, 64, "e2m1")
    none = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    nc.nc_kv_write(cache, none, none, torch.empty(0, dtype=torch.int64, device="cuda"))
    nc.nc_kv_read(cache, torch.empty(0, dtype=torch.int64, device="cuda"), none, none)
    s = torch.cuda.Stream()
    x = torch.ones((32, 1, 64), dtype=torch.bfloat16, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    slots = torch.arange(32, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    nc.nc_kv_write(cache, x, x, slots, stream=s)
    nc.nc_kv_read(cache, slots, y, z, stream=s)
    s.synchronize()
    assert torch.equal(x, y) and torch.equal(x, z)
