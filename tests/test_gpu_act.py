"""Activations that keep their inputs as MX blocks, and their gradients, against the
oracle in binary64 and against differences."""

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc
from oracle import mx
from tests._mx import DT, FMTS, close, data, f64, rounded, stale

pytestmark = pytest.mark.gpu

ACTS = ("silu", "gelu", "gelu_tanh", "relu2")


def bound(want, size, dtype, steps=6):
    """size: what relative errors of 2^-20 of the activation's fp32 steps move the result by (oracle.mx.act); then
    `steps` roundings of products, and the result's own."""
    half = torch.finfo(DT[dtype]).eps / 2
    t = 2.0 ** -20 * size + steps * 2.0 ** -24 * np.abs(want) + 1e-36 * (1 + size)
    return t * (1 + half) + half * np.abs(want)


def like(x):
    return torch.full(x.shape, 3.0, dtype=x.dtype, device="cuda")


def values(rng, rows, cols, dtype):
    x = data(rng, rows, cols, dtype, tail=0.8)
    x[0, 0], x[-1, -1] = 0.0, -0.0
    x[rows // 2, 0], x[rows // 2, cols - 1] = 35.0, -35.0
    return x


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("act", ACTS)
def test_forward_and_backward(act, gated, dtype):
    rng = np.random.default_rng(1)
    for (rows, cols), fmt in zip([(1, 1), (1, 300), (33, 257), (70, 1000), (40, 64)], ("e4m3", "e5m2", "e4m3", "e2m1", "e5m2")):
        g, u = values(rng, rows, cols, dtype), values(rng, rows, cols, dtype) if gated else None
        gq, uq = (stale(nc.new_mx_matrix(rows, cols, fmt), rng) for _ in range(2))
        uq = uq if gated else None
        y = like(g)
        nc.nc_act_forward(g.cuda(), u.cuda() if gated else None, y, gq, uq, act=act, rule="plus1")
        f, _, sf, _ = mx.act(f64(g), act)
        w = f64(u) if gated else 1.0
        close(y, f * w, bound(f * w, sf * np.abs(w), dtype))
        want = {"g": mx.held(f64(g), fmt, "plus1"), "u": mx.held(f64(u), fmt, "plus1") if gated else 1.0}
        for q, name in ((gq, "g"), (uq, "u")):
            if q is not None:
                kept = torch.empty(rows, cols, device="cuda")
                nc.nc_mx_read(q, kept)
                assert np.array_equal(f64(kept), want[name])
        bare = like(g)
        nc.nc_act_forward(g.cuda(), u.cuda() if gated else None, bare, act=act)
        assert torch.equal(bare, y)
        # gradients, from what was kept
        dy = data(rng, rows, cols, dtype)
        f, df, sf, sdf = mx.act(want["g"], act)
        d, w = f64(dy), want["u"]
        dg, du, again = like(g), like(g) if gated else None, like(g)
        nc.nc_act_backward(dy.cuda(), gq, uq, dg, du, act=act, y=again)
        close(dg, d * w * df, bound(d * w * df, sdf * np.abs(d * w), dtype))
        close(again, f * w, bound(f * w, sf * np.abs(w), dtype))
        if gated:
            close(du, d * f, bound(d * f, sf * np.abs(d), dtype))
        dg2, du2 = like(g), like(g) if gated else None
        nc.nc_act_backward(dy.cuda(), gq, uq, dg2, du2, act=act)
        assert torch.equal(dg2, dg) and (not gated or torch.equal(du2, du))


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(act):
    """d y / d gate at the kept values by central differences of the oracle's f: off by h^2 / 6 times the third
    derivative (below 3 for all four near 0; 0 for relu2 off its kink) and 1e-16 / h of the difference."""
    rng = np.random.default_rng(2)
    g = rounded(rng.uniform(-3, 3, (40, 96)), "fp32")
    gq = nc.new_mx_matrix(40, 96, "e4m3")
    y, dg = like(g), like(g)
    nc.nc_act_forward(g.cuda(), None, y, gq, act=act)
    nc.nc_act_backward(torch.ones(40, 96, device="cuda"), gq, None, dg, act=act)
    z, h = mx.held(f64(g), "e4m3", "ceil"), 1e-4
    diff = (mx.act(z + h, act)[0] - mx.act(z - h, act)[0]) / (2 * h)
    off = np.abs(f64(dg) - diff)
    away = np.abs(z) > h if act == "relu2" else np.ones(z.shape, bool)
    assert (off[away] <= 3 * h * h + 1e-10 + 2.0 ** -18 * (1 + np.abs(diff[away]))).all()
    assert (off <= 2 * h).all() or act != "relu2"


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act", ACTS)
def test_large_and_not_finite(act, dtype):
    """Far arguments: the limits, no NaN; infinities are kept as the largest value; a NaN stays one."""
    z = rounded(np.array([[1e30, -1e30, 3e38, -3e38, 100.0, -100.0, 20.0, -20.0, 1e-30, -1e-30, 0.0, 5e18, -5e18]]), dtype)
    y = like(z)
    nc.nc_act_forward(z.cuda(), None, y, act=act)
    with np.errstate(over="ignore"):
        want = mx.act(f64(z), act)[0]
        want = f64(torch.from_numpy(want).to(DT[dtype])) if act == "relu2" else want
    got = f64(y)
    assert not np.isnan(got).any()
    assert (np.abs(got - want)[np.isfinite(want)] <= 1e-3 * np.abs(want)[np.isfinite(want)] + 1e-36).all()
    assert np.array_equal(np.isinf(got), np.isinf(want))
    # one block each, so that every value is kept as it is
    wide = torch.zeros(1, 32 * z.shape[1], dtype=DT[dtype])
    wide[0, ::32] = z[0]
    q, dg, yy = nc.new_mx_matrix(1, wide.shape[1], "e5m2"), like(wide), like(wide)
    nc.nc_mx_write(wide.cuda(), q)
    nc.nc_act_backward(torch.ones_like(wide).cuda(), q, None, dg, act=act, y=yy)
    kept = mx.held(f64(wide), "e5m2", "ceil")
    df = mx.act(kept, act)[1]
    got = f64(dg)
    assert not np.isnan(got).any()
    fin = np.abs(df) < 3e38
    assert (np.abs(got - df)[fin] <= 1e-2 * np.abs(df)[fin] + 1e-30).all()
    x = rounded(np.array([[np.inf, np.nan, 1.0, 2.0] + [0.5] * 60]), dtype)
    y, q = like(x), nc.new_mx_matrix(1, 64, "e4m3")
    nc.nc_act_forward(x.cuda(), None, y, q, act=act)
    got = f64(y)
    assert np.isposinf(got[0, 0]) and np.isnan(got[0, 1]) and not np.isnan(got[0, 2:]).any()
    nc.nc_act_backward(torch.ones_like(x).cuda(), q, None, dg := like(x), act=act)
    assert np.array_equal(np.isnan(f64(dg)[0]), np.arange(64) == 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides_and_places(dtype):
    """Halves of one projection, gradients into halves of another, in place; the columns between are left alone."""
    rng = np.random.default_rng(3)
    rows, cols = 50, 301
    both = data(rng, rows, 2 * cols + 5, dtype).cuda()
    g, u = both[:, :cols], both[:, cols + 5:]
    plain = [like(g), nc.new_mx_matrix(rows, cols, "e4m3"), nc.new_mx_matrix(rows, cols, "e4m3")]
    nc.nc_act_forward(g.contiguous(), u.contiguous(), *plain)
    y, gq, uq = like(both), nc.new_mx_matrix(rows, cols, "e4m3"), nc.new_mx_matrix(rows, cols, "e4m3")
    nc.nc_act_forward(g, u, y[:, 3:3 + cols], gq, uq)
    assert torch.equal(y[:, 3:3 + cols], plain[0]) and torch.equal(gq.data, plain[1].data)
    assert torch.equal(uq.data, plain[2].data)
    assert bool((y[:, :3] == 3).all()) and bool((y[:, 3 + cols:] == 3).all())
    dy = data(rng, rows, cols, dtype).cuda()
    want = [like(dy), like(dy)]
    nc.nc_act_backward(dy, gq, uq, *want)
    d = like(both)
    nc.nc_act_backward(dy, gq, uq, d[:, :cols], d[:, cols + 5:])
    assert torch.equal(d[:, :cols], want[0]) and torch.equal(d[:, cols + 5:], want[1])
    assert bool((d[:, cols:cols + 5] == 3).all())
    nc.nc_act_backward(dy, gq, uq, dy, d[:, :cols])       # over dy itself
    assert torch.equal(dy, want[0]) and torch.equal(d[:, :cols], want[1])
    over = g.contiguous()
    nc.nc_act_forward(over, u, over)                      # over gate itself
    assert torch.equal(over, plain[0])


def test_empty():
    for rows, cols in ((0, 7), (7, 0)):
        x, q = torch.empty(rows, cols, device="cuda"), nc.new_mx_matrix(rows, cols, "e4m3")
        nc.nc_act_forward(x, None, torch.empty_like(x), q)
        nc.nc_act_backward(x, q, None, torch.empty_like(x))
