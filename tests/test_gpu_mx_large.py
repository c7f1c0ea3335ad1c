"""Matrices whose codes, rows and results pass 32 bits: offsets in the writes, reads and
products.  One row stands for all (stride 0), so that the inputs stay small."""

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc
from oracle import mx
from tests._mx import close, data, f64, product

pytestmark = pytest.mark.gpu


def test_codes_past_32_bits():
    rows, cols = 70000, 65536                            # 4.6e9 codes
    rng = np.random.default_rng(1)
    row = data(rng, 1, cols, "bf16")
    want = mx.held(f64(row), "e4m3", "ceil")
    m = nc.new_mx_matrix(rows, cols, "e4m3")
    assert m.data.numel() > 2 ** 32
    x = row.cuda().expand(rows, cols)
    nc.nc_mx_write(x, m)
    back = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    nc.nc_mx_read(m, back)
    first = back[0].clone()
    assert np.array_equal(f64(first)[None], want)
    for at in range(0, rows, 10000):
        assert bool((back[at:at + 10000] == first).all())
    del back
    xb = data(rng, 40, cols, "bf16")
    b = nc.new_mx_matrix(40, cols, "e2m1")
    nc.nc_mx_write(xb.cuda(), b)
    out, turned = torch.empty(rows, 40, device="cuda"), torch.empty(40, rows, device="cuda")
    nc.nc_mx_matmul(m, b, out)
    nc.nc_mx_matmul(b, m, turned)
    ref, tol = product(row, xb, "e4m3", "e2m1", "fp32")
    close(out[:1], ref, tol)
    assert bool((out == out[0]).all())                   # the same sums in the same order
    close(turned[:, -1:], ref.T, tol.T)
    assert bool((turned == turned[:, :1]).all())
    del m, out, turned
    t = nc.new_mx_matrix(cols, rows, "e4m3")             # blocks of equal values down the columns
    nc.nc_mx_write(x, t=t)
    back = torch.empty(cols, rows, dtype=torch.bfloat16, device="cuda")
    nc.nc_mx_read(t, back)
    want = mx.held(np.repeat(f64(row).T, 32, 1), "e4m3", "ceil")[:, 0]
    assert np.array_equal(f64(back[:, 0]), want) and bool((back == back[:, :1]).all())


def test_results_past_32_bits():
    m, n, k = 70000, 65000, 64                           # 4.5e9 results
    rng = np.random.default_rng(2)
    xa, xb = data(rng, 1, k, "bf16"), data(rng, 40, k, "bf16")
    a, b = nc.new_mx_matrix(m, k), nc.new_mx_matrix(n, k)
    nc.nc_mx_write(xa.cuda().expand(m, k), a)
    nc.nc_mx_write(xb.cuda().repeat(n // 40, 1), b)
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    nc.nc_mx_matmul(a, b, out)
    ref, tol = product(xa, xb, "e2m1", "e2m1", "bf16")
    close(out[:1, :40], ref, tol)
    for at in range(0, m, 10000):
        assert bool((out[at:at + 10000].view(-1, n // 40, 40) == out[0, :40]).all())


def test_activation_rows_past_32_bits():
    """Rows far apart: strides whose products with the row pass 32 bits."""
    stride, rows, cols = 1 << 27, 40, 70                 # 5.4e9 elements between the first and the last row
    rng = np.random.default_rng(3)
    hold = torch.empty(stride * (rows - 1) + cols, dtype=torch.bfloat16, device="cuda")
    x = hold.as_strided((rows, cols), (stride, 1))
    g = data(rng, rows, cols, "bf16").cuda()
    x.copy_(g)
    want, y = torch.empty_like(g), torch.empty_like(g)
    a, b = nc.new_mx_matrix(rows, cols, "e4m3"), nc.new_mx_matrix(rows, cols, "e4m3")
    nc.nc_act_forward(g, None, want, a)
    nc.nc_act_forward(x, None, y, b)
    assert torch.equal(y, want) and torch.equal(a.data, b.data)
    nc.nc_act_forward(g, None, x, b)
    assert torch.equal(x, want)
    nc.nc_act_backward(g, a, None, want)
    nc.nc_act_backward(g, a, None, x)
    assert torch.equal(x, want)
