"""Products of MX matrices on the GPU against the oracle's values in binary64."""

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc
from oracle import mx
from tests._mx import DT, FMTS, close, data, f64, product, rounded, stale, written

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 1), (1, 40, 300), (3, 33, 64), (32, 32, 256), (33, 65, 31), (100, 130, 1000), (257, 140, 520)]


def blank(rows, cols, dtype):
    return torch.full((rows, cols), 3.0, dtype=DT[dtype], device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fb", FMTS)
@pytest.mark.parametrize("fa", FMTS)
def test_formats(fa, fb, dtype):
    rng = np.random.default_rng(1)
    for m, n, k in SIZES:
        xa, xb = data(rng, m, k, "fp32", tail=0.7), data(rng, n, k, "bf16", tail=0.7)
        out = blank(m, n, dtype)
        nc.nc_mx_matmul(written(xa, fa), written(xb, fb), out)
        close(out, *product(xa, xb, fa, fb, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fa,fb", [("e2m1", "e2m1"), ("e4m3", "e2m1"), ("e5m2", "e4m3")])
def test_larger(fa, fb, dtype):
    """Sizes of many workgroups, whole and ragged, and long sums."""
    rng = np.random.default_rng(2)
    for m, n, k in [(512, 512, 512), (300, 777, 1100), (600, 280, 257), (64, 96, 9000), (40, 1030, 256), (1025, 257, 64)]:
        xa, xb = data(rng, m, k, "bf16"), data(rng, n, k, "bf16")
        out = blank(m, n, dtype)
        nc.nc_mx_matmul(written(xa, fa), written(xb, fb), out)
        close(out, *product(xa, xb, fa, fb, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fa,fb", [("e2m1", "e2m1"), ("e4m3", "e4m3")])
def test_bias_accumulate_and_strides(fa, fb, dtype):
    """Bias of each column, addition to what is there, any row stride; what lies between the rows is left alone."""
    rng = np.random.default_rng(3)
    for m, n, k in [(1, 70, 300), (45, 33, 700), (300, 531, 512), (260, 260, 2048)]:
        xa, xb = data(rng, m, k, "bf16"), data(rng, n, k, "bf16")
        a, b = written(xa, fa), written(xb, fb)
        bias, there = data(rng, 1, n, dtype)[0], data(rng, m, n, dtype)
        hold = torch.full((m, n + 9), 3.0, dtype=DT[dtype], device="cuda")
        out = hold[:, 5:5 + n]
        nc.nc_mx_matmul(a, b, out, bias=bias.cuda())
        close(out, *product(xa, xb, fa, fb, dtype, add=f64(bias)[None, :]))
        out.copy_(there)
        nc.nc_mx_matmul(a, b, out, bias=bias.cuda(), accumulate=True)
        close(out, *product(xa, xb, fa, fb, dtype, add=f64(bias)[None, :] + f64(there)))
        assert bool((hold[:, :5] == 3).all()) and bool((hold[:, 5 + n:] == 3).all())


@pytest.mark.parametrize("x_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fb", ["e2m1", "e4m3"])
@pytest.mark.parametrize("fa", FMTS)
def test_linear(fa, fb, x_dtype):
    """Rows quantised on the way, from one to several strips of 32."""
    rng = np.random.default_rng(4)
    for m, n, k in [(1, 70, 1), (1, 300, 4096), (2, 33, 300), (17, 100, 700), (32, 64, 2048), (33, 64, 511), (200, 130, 640)]:
        x, w = data(rng, m, k + 3, x_dtype, tail=0.7)[:, 3:], data(rng, n, k, "bf16")
        wq = written(w, fb)
        for rule in ("ceil", "ocp"):
            for dtype in ("bf16", "fp32"):
                out = blank(m, n, dtype)
                wide = torch.zeros(m, k + 3, dtype=DT[x_dtype], device="cuda")
                wide[:, 3:] = x.cuda()
                nc.nc_mx_linear(wide[:, 3:], wq, out, fmt=fa, rule=rule)
                close(out, *product(x, w, fa, fb, dtype, rule_a=rule))
        ws = nc.new_mx_workspace(300, wq, fa)             # one for more rows serves fewer
        again = blank(m, n, "fp32")
        nc.nc_mx_linear(wide[:, 3:], wq, again, fmt=fa, rule="ocp", ws=ws)
        assert torch.equal(again, out)


@pytest.mark.parametrize("fa,fb", [("e2m1", "e2m1"), ("e4m3", "e2m1"), ("e5m2", "e4m3")])
@pytest.mark.parametrize("m,n", [(3, 40), (300, 300)])
def test_not_finite(fa, fb, m, n):
    """A NaN reaches its row or column and no other; infinities are held as the largest value; the rows past the end
    of a stale buffer reach nothing."""
    rng = np.random.default_rng(5)
    k = 600
    xa, xb = data(rng, m, k, "bf16"), data(rng, n, k, "bf16")
    xa[m - 1, k - 1] = float("nan")
    xa[0, 5] = float("inf")
    xb[n // 2, 100] = float("nan")
    xb[1, 7] = -float("inf")
    a, b = stale(nc.new_mx_matrix(m, k, fa), rng), stale(nc.new_mx_matrix(n, k, fb), rng)
    nc.nc_mx_write(xa.cuda(), a)
    nc.nc_mx_write(xb.cuda(), b)
    for dtype in ("bf16", "fp32"):
        out = blank(m, n, dtype)
        nc.nc_mx_matmul(a, b, out)
        want, tol = product(xa, xb, fa, fb, dtype)
        assert np.isnan(want[m - 1]).all() and np.isnan(want[:, n // 2]).all() and not np.isnan(want[0, 0])
        close(out, want, np.nan_to_num(tol))
        out = blank(m, n, dtype)
        nc.nc_mx_linear(xa.cuda(), b, out, fmt=fa)
        close(out, want, np.nan_to_num(tol))


@pytest.mark.parametrize("fa,fb", [("e2m1", "e2m1"), ("e4m3", "e5m2")])
def test_far_scales(fa, fb):
    """Blocks at both ends of the scales' range."""
    rng = np.random.default_rng(6)
    k = 256
    xa = rounded(rng.standard_normal((40, k)) * np.ldexp(1.0, np.repeat(rng.integers(-60, 60, (40, k // 32)), 32, 1)), "fp32")
    xb = rounded(rng.standard_normal((70, k)) * np.ldexp(1.0, np.repeat(rng.integers(-60, 60, (70, k // 32)), 32, 1)), "fp32")
    for dtype in ("bf16", "fp32"):
        out = blank(40, 70, dtype)
        nc.nc_mx_matmul(written(xa, fa), written(xb, fb), out)
        close(out, *product(xa, xb, fa, fb, dtype))


def test_no_columns_rows_or_results():
    for fa, fb in (("e2m1", "e2m1"), ("e4m3", "e2m1")):
        a, b = nc.new_mx_matrix(5, 0, fa), nc.new_mx_matrix(70, 0, fb)
        for dtype in ("bf16", "fp32"):
            bias = torch.arange(70, dtype=DT[dtype], device="cuda")
            out = blank(5, 70, dtype)
            nc.nc_mx_matmul(a, b, out)
            assert bool((out == 0).all())
            nc.nc_mx_matmul(a, b, out, bias=bias, accumulate=True)
            nc.nc_mx_linear(torch.empty(5, 0, device="cuda"), b, out, bias=bias, accumulate=True)
            assert torch.equal(out, (2 * bias).expand(5, 70))
            big = blank(100, 70, dtype)
            nc.nc_mx_linear(torch.empty(100, 0, device="cuda"), b, big, bias=bias)
            assert torch.equal(big, bias.expand(100, 70))
        nc.nc_mx_matmul(nc.new_mx_matrix(0, 9, fa), nc.new_mx_matrix(4, 9, fb), torch.empty(0, 4, device="cuda"))
        nc.nc_mx_matmul(nc.new_mx_matrix(4, 9, fa), nc.new_mx_matrix(0, 9, fb), torch.empty(4, 0, device="cuda"))
        nc.nc_mx_linear(torch.empty(0, 9, device="cuda"), nc.new_mx_matrix(4, 9, fb), torch.empty(0, 4, device="cuda"))


def test_same_bits_every_time():
    rng = np.random.default_rng(7)
    a, b = written(data(rng, 90, 8000, "bf16"), "e4m3"), written(data(rng, 200, 8000, "bf16"), "e4m3")
    for dtype in ("bf16", "fp32"):
        outs = []
        for _ in range(3):
            out = blank(90, 200, dtype)
            nc.nc_mx_matmul(a, b, out)
            outs.append(out)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_a_matrix_with_itself():
    """Both operands one matrix."""
    rng = np.random.default_rng(8)
    x = data(rng, 130, 320, "bf16")
    a = written(x, "e4m3")
    out = blank(130, 130, "fp32")
    nc.nc_mx_matmul(a, a, out)
    close(out, *product(x, x, "e4m3", "e4m3", "fp32"))
    assert torch.equal(out, out.T)


@pytest.mark.parametrize("rows", [5, 6, 7, 8, 9])
@pytest.mark.parametrize("fa,fb", [("e2m1", "e2m1"), ("e4m3", "e2m1"), ("e4m3", "e4m3"), ("e5m2", "e4m3")])
def test_linear_where_rows_are_written_first(fa, fb, rows):
    """Either side of the number of rows that a product quantises itself, over eight chunks of columns and more (sixteen
    waves), with rows past the last that a stale place in LDS could reach, and a workspace for other rows."""
    rng = np.random.default_rng(6)
    for n, k in [(40, 2048), (300, 2500), (33, 4100)]:
        x, w = data(rng, rows, k, "bf16", tail=0.7), data(rng, n, k, "bf16")
        wq, xg = written(w, fb), x.cuda()
        for dtype in ("bf16", "fp32"):
            out, again = blank(rows, n, dtype), blank(rows, n, dtype)
            nc.nc_mx_linear(xg, wq, out, fmt=fa)
            close(out, *product(x, w, fa, fb, dtype))
            nc.nc_mx_linear(xg, wq, again, fmt=fa, ws=nc.new_mx_workspace(200, wq, fa))
            assert torch.equal(again, out)
