"""The largest and lowest values of the types, as masks hold them, through what a matrix
keeps: such a value rounds up to 2^128 in its block (a finite number by the definition),
which no fp32 number is."""

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc
from oracle import mx
from tests._mx import DT, FMTS, close, f64, product, rounded, written
from tests.test_gpu_act import ACTS, bound, like

pytestmark = pytest.mark.gpu


def gradients(gate, up, step, act, fmt, dtype):
    """The gradients for gates, ups and steps' gradients each in a block of its own, against the formula at what is kept.
    The kept 2^128 counts as fp32's largest value: one rounding more.  f and f' are fp32 numbers, so what they have
    below the smallest normal one, 2^-126, may be lost (gelu of -16 is 1e-56): that times the other factors, which
    reach 2^128 here."""
    top = float(torch.finfo(DT[dtype]).max)
    n = 32 * len(gate)
    g, u, dy = (np.zeros((1, n)) for _ in range(3))
    g[0, ::32], u[0, ::32], dy[0, ::32] = gate, up, step
    g, u, dy = (rounded(x, dtype) for x in (g, u, dy))
    gq, uq = written(g, fmt), written(u, fmt)
    z, w, d = mx.held(f64(g), fmt, "ceil"), mx.held(f64(u), fmt, "ceil"), f64(dy)
    f, df, sf, sdf = mx.act(z, act)
    for up_q, v in ((uq, w), (None, 1.0)):
        dg, du, y = like(g), like(g) if up_q is not None else None, like(g)
        nc.nc_act_backward(dy.cuda(), gq, up_q, dg, du, act=act, y=y)
        for got, want, size, factor in ((dg, d * v * df, sdf, d * v), (du, d * f, sf, d), (y, f * v, sf, v)):
            if got is None:
                continue
            got = f64(got)
            assert not np.isnan(got).any()
            # past fp32 the result is infinite, or a step of it is (relu2 of the largest gate)
            fits = np.abs(want) < 2.0 ** 127.9
            if act == "relu2":
                fits &= z < 2.0 ** 60
            tol = bound(want, size * np.abs(factor), dtype, steps=9) + 2.0 ** -126 * np.abs(factor)
            bad = fits & ~(np.abs(got - want) <= tol)
            assert not bad.any(), (got[bad], want[bad], tol[bad])
            over = np.abs(want) > 2.0 ** 128
            assert (np.abs(got[over]) >= top * (1 - 2.0 ** -7)).all() and (np.sign(got[over]) == np.sign(want[over])).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", ACTS)
def test_gradients_of_lowest_values(act, fmt, dtype):
    """Gates and ups at either end of the type's range."""
    t = float(torch.finfo(DT[dtype]).max)
    gate = [-t, t, -t, t, -20.0, -200.0, 0.5, 0.0]
    up = [0.5, -0.5, -t, 2.0 ** -100, t, -t, 2.0 ** -20, -t]
    step = [0.5, 0.25, 0.5, 0.25, 0.5, -0.25, 1.0, 2.0 ** -10]
    gradients(gate, up, step, act, fmt, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", ACTS)
def test_steps_whose_product_with_up_passes_fp32(act, fmt, dtype):
    """dy u is past fp32, dy u f'(g) is not."""
    t = float(torch.finfo(DT[dtype]).max)
    gradients([-20.0, -20.0, -200.0, -200.0, -20.0], [t, -t, t, -t, 1e30], [4.0, 4.0, 4.0, -8.0, 1e12], act, fmt, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", FMTS)
def test_read_at_every_scale(fmt, dtype):
    """Every value of the grid at every exponent that fp32 has, read as fp32 and as bf16: rounded once below the
    normal range, infinite where a block's largest value rounds up past it."""
    g = mx.grid(fmt)
    rows = []
    for e in range(-149, 128):
        for i in range(0, len(g), 30):                   # the block's largest value fixes its scale
            part = np.concatenate([[g[-1], -g[-1]], g[i:i + 30], np.zeros(30)])[:32]
            rows.append(part / 2.0 ** mx.EMAX[fmt] * 2.0 ** e)
    x = np.array(rows)
    top = float(torch.finfo(torch.float32).max)
    x = np.clip(x, -top, top)                            # the highest blocks: fp32's largest value
    x = rounded(x, "fp32")
    m = written(x, fmt)
    want = mx.held(f64(x), fmt, "ceil")
    out = torch.empty(x.shape, dtype=DT[dtype], device="cuda")
    nc.nc_mx_read(m, out)
    # at most four bits: fp32 holds them down to 2^-149, so the step through fp32 rounds only what fp32 rounds
    with np.errstate(over="ignore"):
        ref = torch.from_numpy(want.astype(np.float32)).to(DT[dtype])
    assert torch.equal(out.cpu(), ref)


@pytest.mark.parametrize("m", [3, 700])
@pytest.mark.parametrize("fa,fb", [("e2m1", "e2m1"), ("e4m3", "e2m1"), ("e5m2", "e4m3")])
def test_products_of_lowest_values(fa, fb, m):
    """A column at the type's lowest value against small and zero weights.  The scaled instruction has 2^128 as it is;
    fp32 results of 8-bit operands have what a matrix reads back as in fp32, an infinity."""
    rng = np.random.default_rng(1)
    n, k = 40, 96
    x, w = rng.standard_normal((m, k)), rng.standard_normal((n, k))
    x[:, 32:64] = 0                                      # a block of its own
    x[:, 40] = float(torch.finfo(torch.bfloat16).min)
    w[:, 32:64] = 0
    w[::2, 40] = 2.0 ** -100
    x, w = rounded(x, "bf16"), rounded(w, "bf16")
    a, b = written(x, fa), written(w, fb)
    exact = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    nc.nc_mx_matmul(a, b, exact)
    close(exact, *product(x, w, fa, fb, "bf16"))
    out = torch.empty(m, n, device="cuda")
    nc.nc_mx_matmul(a, b, out)
    if fa == fb == "e2m1":
        close(out, *product(x, w, fa, fb, "fp32"))
    else:
        assert bool((out[:, ::2] == -float("inf")).all()) and bool(out[:, 1::2].isnan().all())
