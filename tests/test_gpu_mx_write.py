"""Matrices of MX blocks written and read back on the GPU, against the oracle: equal."""

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc
from oracle import mx
from tests._mx import DT, FMTS, data, f64, rounded, stale, written

pytestmark = pytest.mark.gpu


def read(m, dtype):
    out = torch.full((m.rows, m.cols), 7.0, dtype=DT[dtype], device="cuda")
    nc.nc_mx_read(m, out)
    return out


def equal(got, want):
    """Equal values, signs of zeros and NaN alike."""
    g = f64(got)
    assert g.shape == want.shape
    assert np.array_equal(np.isnan(g), np.isnan(want))
    n = ~np.isnan(want)
    assert np.array_equal(g[n], want[n]) and np.array_equal(np.signbit(g[n]), np.signbit(want[n]))


@pytest.mark.parametrize("rule", ["ocp", "plus1", "ceil"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", FMTS)
def test_rows_and_columns(fmt, dtype, rule):
    rng = np.random.default_rng(1)
    for rows, cols in [(1, 1), (1, 256), (5, 31), (32, 64), (33, 257), (97, 300), (256, 33), (300, 513), (64, 1000)]:
        x = data(rng, rows, cols, dtype, tail=1.5)
        want, want_t = mx.held(f64(x), fmt, rule), mx.held(f64(x).T, fmt, rule)
        xd = x.cuda()
        alone, alone_t, m, t = (stale(nc.new_mx_matrix(*s, fmt), rng)
                                for s in ((rows, cols), (cols, rows), (rows, cols), (cols, rows)))
        nc.nc_mx_write(xd, alone, rule=rule)
        nc.nc_mx_write(xd, t=alone_t, rule=rule)
        nc.nc_mx_write(xd, m, t, rule=rule)
        equal(read(m, "fp32"), want)
        equal(read(t, "fp32"), want_t)
        assert torch.equal(m.data, alone.data) and torch.equal(t.data, alone_t.data)   # every byte, filling too
        if dtype == "bf16":                              # a value of at most four bits within bf16's range: exact
            equal(read(m, "bf16"), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_every_bf16_pattern(fmt):
    """Every bf16 value against blocks of large, middle and small company, non-finite ones included."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    for company in (None, 1.0, 3.0e38, 1e-30):
        rows = x.view(-1, 32).clone() if company is None else torch.cat(
            [x.view(-1, 8), torch.full((8192, 24), company, dtype=torch.bfloat16)], 1)
        for rule in ("ocp", "ceil"):
            want = mx.held(f64(rows), fmt, rule)
            for y in (rows, rows.float()):
                m = written(y, fmt, rule)
                with np.errstate(over="ignore"):
                    equal(read(m, "fp32"), want.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("fmt", FMTS)
def test_not_finite(fmt):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((70, 130)).astype(np.float32)
    for v in (np.inf, -np.inf, np.nan):
        x[rng.random(x.shape) < 0.004] = v
    x[3, :32] = np.inf
    x[4, 32:64] = 0.0
    x[5, 64:96] = -0.0
    x[6, :32] = 1e-42                                    # below fp32's normal range
    x[7, 128:] = np.nan
    for dtype in ("fp32", "bf16"):
        xt = rounded(x, dtype)
        m, t = nc.new_mx_matrix(70, 130, fmt), nc.new_mx_matrix(130, 70, fmt)
        nc.nc_mx_write(xt.cuda(), m, t)
        equal(read(m, "fp32"), mx.held(f64(xt), fmt, "ceil").astype(np.float32).astype(np.float64))
        equal(read(t, "fp32"), mx.held(f64(xt).T, fmt, "ceil").astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", FMTS)
def test_strides(fmt, dtype):
    """Rows on any element, of any stride; what lies between them is left alone."""
    rng = np.random.default_rng(3)
    wide = data(rng, 45, 333, dtype).cuda()
    for at, cols in ((0, 300), (1, 256), (3, 77), (8, 264)):
        x = wide[:, at:at + cols]
        m, t = nc.new_mx_matrix(45, cols, fmt), nc.new_mx_matrix(cols, 45, fmt)
        nc.nc_mx_write(x, m, t)
        want = mx.held(f64(x), fmt, "ceil")
        hold = torch.full((45, 333), 5.0, dtype=DT[dtype], device="cuda")
        nc.nc_mx_read(m, hold[:, at:at + cols])
        equal(hold[:, at:at + cols], want)
        assert bool((hold[:, :at] == 5).all()) and bool((hold[:, at + cols:] == 5).all())
        equal(read(t, "fp32"), mx.held(f64(x).T, fmt, "ceil"))
    row = wide[:1].expand(40, 333)                       # one row for all: stride 0
    m = nc.new_mx_matrix(40, 333, fmt)
    nc.nc_mx_write(row, m)
    equal(read(m, "fp32"), np.repeat(mx.held(f64(wide[:1]), fmt, "ceil"), 40, 0))


def test_larger_buffer_and_empty():
    rng = np.random.default_rng(4)
    buf = torch.full((nc.mx_bytes(100, 700, "e4m3") + 512,), 9, dtype=torch.uint8, device="cuda")
    m = nc.MxMatrix(buf, 50, 300, "e4m3")                # a smaller matrix in a larger buffer
    x = data(rng, 50, 300, "bf16")
    nc.nc_mx_write(x.cuda(), m)
    equal(read(m, "fp32"), mx.held(f64(x), "e4m3", "ceil"))
    assert bool((buf[nc.mx_bytes(50, 300, "e4m3"):] == 9).all())
    for rows, cols in ((0, 5), (5, 0), (0, 0)):
        m, t = nc.new_mx_matrix(rows, cols), nc.new_mx_matrix(cols, rows)
        nc.nc_mx_write(torch.empty(rows, cols, device="cuda"), m, t)
        nc.nc_mx_read(m, torch.empty(rows, cols, device="cuda"))


def test_against_the_cast():
    """8-bit matrices hold what nc_cast_mx and nc_dequant make of the same rows."""
    rng = np.random.default_rng(5)
    x = data(rng, 64, 512, "bf16", tail=1.0).cuda()
    for fmt in ("e4m3", "e5m2"):
        codes = torch.empty(x.numel(), dtype=torch.uint8, device="cuda")
        scales = torch.empty(x.numel() // 32, dtype=torch.uint8, device="cuda")
        y = torch.empty(x.numel(), dtype=torch.bfloat16, device="cuda")
        nc.nc_cast_mx([x.view(-1)], [codes], [scales], [512], fmt, "ocp", nc.new_counts(1))
        nc.nc_dequant([codes], [y], fmt, scales=[scales], cols=[512])
        assert torch.equal(read(written(x, fmt, "ocp"), "bf16").view(-1), y)
