"""Products by the kernel that they take (tests/_mx_plans.py): every kernel, with every
pair of formats that it serves, over one chunk of columns and many, whole and ragged."""

import os
import sys

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc
from oracle import mx
from tests._mx import DT, f64
from tests._mx_plans import ANY, CALLS, name

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import mx_mlp  # noqa: E402

pytestmark = pytest.mark.gpu


def whole(g, rows, cols):
    """Numbers that every format holds, with scales of their own in every block: 0, +-1, 2, 3, 4, 6 times 1 or 2."""
    grid = torch.tensor([0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6], dtype=torch.float32, device="cuda")
    x = grid[torch.randint(11, (rows, cols), generator=g, device="cuda")]
    double = torch.randint(2, (rows, -(-cols // 32)), generator=g, device="cuda").repeat_interleave(32, 1)[:, :cols]
    return (x * (1 + double)).bfloat16()


def written(x, fmt):
    m = nc.new_mx_matrix(x.shape[0], x.shape[1], fmt)
    nc.nc_mx_write(x, m)
    return m


def full(m, n, dtype):
    return torch.full((m, n), 3.0, dtype=DT[dtype], device="cuda")


@pytest.mark.parametrize("call", CALLS, ids=name)
def test_whole_numbers(call):
    """Products and sums of whole numbers below 2^24 are exact in fp32 in any order (at most 12 * 12 * 70000 < 2^24), and
    no product's bits lie 2^-13 below another product (144 and 1: 2^-7): results are the exact sums, rounded once."""
    m, n, k, _, fa, fb, dtype = call
    g = torch.Generator(device="cuda").manual_seed(m + 7 * n + k)
    xa, xb = whole(g, m, k), whole(g, n, k)
    a, b = written(xa, fa), written(xb, fb)
    want = xa.double() @ xb.double().T
    assert float(want.abs().max()) < 2 ** 24
    out = full(m, n, dtype)
    ws = nc.new_mx_workspace(m, b)
    ws.fill_(255)                                        # what is not written reads as NaN
    nc.nc_mx_matmul(a, b, out, ws=ws)
    assert torch.equal(out, want.to(DT[dtype]))
    again = full(m, n, dtype)
    nc.nc_mx_matmul(a, b, again)                         # workspace from torch
    assert torch.equal(again, out)


SOME = [c for c in CALLS if (c[4], c[5]) in (("e2m1", "e2m1"), ("e4m3", "e2m1"), ("e5m2", "e4m3"), ("e4m3", "e4m3"))
        and c[:3] in ((4000, 4000, 1300), (4096, 4096, 1280), (4522, 7059, 523), (850, 2729, 1), (2000, 2000, 1300), (2048, 2048, 768), (100, 130, 20000),
                      (100, 131, 70000), (500, 1000, 16000), (1, 1, 19265), (900, 1000, 1300), (202, 3540, 1398), (321, 2227, 2842), (168, 5431, 4434), (300, 777, 1100))]


@pytest.mark.parametrize("call", SOME, ids=name)
def test_bias_accumulate_and_strides(call):
    """Whole numbers again, with a bias and what is there; rows apart, on any element (and, whole, past the caches)."""
    m, n, k, _, fa, fb, dtype = call
    g = torch.Generator(device="cuda").manual_seed(m + n + 5 * k)
    xa, xb = whole(g, m, k), whole(g, n, k)
    a, b = written(xa, fa), written(xb, fb)
    want = xa.double() @ xb.double().T
    bias = torch.randint(-200, 201, (n,), generator=g, device="cuda").to(DT[dtype])
    there = torch.randint(-200, 201, (m, n), generator=g, device="cuda").to(DT[dtype])
    ws = nc.new_mx_workspace(m, b)
    for at, more in ((5, 9), (0, 0)):
        hold = full(m, n + more, dtype)
        out = hold[:, at:at + n]
        nc.nc_mx_matmul(a, b, out, bias=bias, ws=ws)
        assert torch.equal(out, (want + bias.double()).to(DT[dtype]))
        out.copy_(there)
        nc.nc_mx_matmul(a, b, out, accumulate=True, ws=ws)
        assert torch.equal(out, (want + there.double()).to(DT[dtype]))
        out.copy_(there)
        nc.nc_mx_matmul(a, b, out, bias=bias, accumulate=True, ws=ws)
        assert torch.equal(out, (want + there.double() + bias.double()).to(DT[dtype]))
        assert bool((hold[:, :at] == 3).all()) and bool((hold[:, at + n:] == 3).all())


def groups(v, x, fmt):
    """Largest factor of each group of eight columns; an element counts as its scale's smallest normal one at least."""
    least = torch.from_numpy(np.ldexp(1.0, mx.exponents(f64(x), fmt, "ceil") + mx.EMIN[fmt])).cuda()
    w = torch.maximum(v.abs().nan_to_num(), least)
    return torch.nn.functional.pad(w, (0, -x.shape[1] % 8)).unflatten(1, (-1, 8)).amax(2)


@pytest.mark.parametrize("call", SOME, ids=name)
def test_heavy_tails_and_not_finite(call):
    """Values of all sizes against a product of what the matrices hold in 64 bits.  fp32 sums of k products, in any order
    and cut instead of rounded, are off by at most k + 42 times 2^-23 of the sum of magnitudes; bf16 results of 8-bit
    operands by 8 * 2^-13 of the sum over groups of eight columns of the largest factors' products; then the result's own
    rounding.  A NaN reaches its row or column and no other."""
    m, n, k, _, fa, fb, dtype = call
    g = torch.Generator(device="cuda").manual_seed(m + 3 * n + k)

    def values(rows):
        x = torch.randn(rows, k, generator=g, device="cuda") * torch.exp(0.8 * torch.randn(rows, k, generator=g, device="cuda"))
        return (x * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g, device="cuda"))).bfloat16()
    xa, xb = values(m), values(n)
    if min(m, n) > 1:
        xa[m - 1, k - 1] = xb[n // 2, 0] = float("nan")
        xa[0, 0], xb[1, k - 1] = float("inf"), -float("inf")
    a, b = written(xa, fa), written(xb, fb)
    va, vb = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda")
    nc.nc_mx_read(a, va)
    nc.nc_mx_read(b, vb)
    va, vb = va.double(), vb.double()
    want, mag = va @ vb.T, va.abs() @ vb.abs().T
    half = torch.finfo(DT[dtype]).eps / 2
    tol = (k + 42) * 2.0 ** -23 * mag + 1e-37
    if dtype == "bf16" and (fa, fb) != ("e2m1", "e2m1"):
        tol = tol + 8 * 2.0 ** -13 * (groups(va, xa, fa) @ groups(vb, xb, fb).T)
    tol = tol * (1 + half) + half * want.abs()
    outs = []
    for _ in range(3):
        out = full(m, n, dtype)
        nc.nc_mx_matmul(a, b, out)
        outs.append(out)
    nan = want.isnan()
    assert torch.equal(outs[0].isnan(), nan)
    if min(m, n) > 1:
        assert bool(nan[m - 1].all()) and bool(nan[:, n // 2].all()) and int(nan.sum()) == m + n - 1
    assert bool(((outs[0].double() - want).abs() <= tol)[~nan].all())
    for out in outs[1:]:                                 # the same bits every time
        assert torch.equal(out.view(torch.uint8), outs[0].view(torch.uint8))


@pytest.mark.parametrize("x_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", [(4000, 4000, 1300), (2000, 2000, 1300), (100, 130, 20000), (900, 1000, 1300)])
@pytest.mark.parametrize("fa,fb", [("e2m1", "e2m1"), ("e4m3", "e2m1"), ("e5m2", "e4m3")])
def test_linear_of_many_rows(fa, fb, m, n, k, x_dtype):
    """Rows quantised first, into the same workspace as the splits' parts."""
    g = torch.Generator(device="cuda").manual_seed(m + n)
    x, w = whole(g, m, k), whole(g, n, k)
    want = x.double() @ w.double().T
    wq = written(w, fb)
    ws = nc.new_mx_workspace(m, wq, fa)
    ws.fill_(255)
    for dtype in ANY:
        out = full(m, n, dtype)
        nc.nc_mx_linear(x.to(DT[x_dtype]), wq, out, fmt=fa, ws=ws)
        assert torch.equal(out, want.to(DT[dtype]))


@pytest.mark.parametrize("rows", [8, 9, 12])
def test_serving_either_side_of_the_rows_that_a_product_quantises(rows):
    r = mx_mlp.serve(rows=rows, width=288, hidden=600)
    for got, want in zip(r["got"], r["want"]):
        assert torch.equal(got, want) and bool(torch.isfinite(got).all()) and bool(got.any())
    assert not torch.equal(r["got"][0], r["got"][1])


def test_graphs_of_split_products_share_a_workspace():
    """Two captured products whose sums are cut along the columns, replayed in turn with one workspace and with eager
    work between the replays, against the exact sums."""
    g = torch.Generator(device="cuda").manual_seed(1)
    w = whole(g, 130, 20000)
    wq = written(w, "e4m3")
    ws = nc.new_mx_workspace(100, wq)
    xs = [whole(g, m, 20000) for m in (40, 100)]
    ms = [written(x, "e4m3") for x in xs]
    outs = [full(x.shape[0], 130, "fp32") for x in xs]
    graphs = []
    for q, o in zip(ms, outs):
        nc.nc_mx_matmul(q, wq, o, ws=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            nc.nc_mx_matmul(q, wq, o, ws=ws)
    for seed in range(3):
        xs = [whole(g, x.shape[0], 20000) for x in xs]
        for q, x, o in zip(ms, xs, outs):
            nc.nc_mx_write(x, q)
            o.zero_()
        ws.fill_(255)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for x, o in zip(xs, outs):
            assert torch.equal(o, (x.double() @ w.double().T).float())


def test_columns_up_to_31_bits():
    """The longest rows: 2^31 - 1 columns, in splits and quantised on the way."""
    k, m, n = 2 ** 31 - 1, 12, 5
    at = torch.tensor([0, 255, 256, 2 ** 30 + 7, 2 ** 31 - 300, 2 ** 31 - 2], device="cuda")
    x, y = (torch.zeros(k, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[at] = torch.tensor([1, 2, -3, 4, 6, 3.0], device="cuda").bfloat16()
    y[at] = torch.tensor([4, -1, 2, 3, 1, -6.0], device="cuda").bfloat16()
    want = float((x[at].float() * y[at].float()).sum())
    b = nc.new_mx_matrix(n, k)
    nc.nc_mx_write(y[None].expand(n, k), b)
    del y
    out = full(3, n, "bf16")
    nc.nc_mx_linear(x[None].expand(3, k), b, out, fmt="e2m1")
    assert bool((out == want).all())
    a = nc.new_mx_matrix(m, k)
    nc.nc_mx_write(x[None].expand(m, k), a)
    for dtype in ANY:
        out = full(m, n, dtype)
        nc.nc_mx_matmul(a, b, out)
        assert bool((out == want).all())


def test_workspace_from_torch_on_any_stream():
    """ws=None where splits need one: streams given as objects and by number, the default one's 0, under capture too."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w = whole(g, 100, 20000), whole(g, 130, 20000)
    a, b = written(x, "e4m3"), written(w, "e4m3")
    want = (x.double() @ w.double().T).float()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for stream in (None, 0, side, side.cuda_stream):
        out = full(100, 130, "fp32")
        torch.cuda.synchronize()
        nc.nc_mx_matmul(a, b, out, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    out = full(100, 130, "fp32")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nc.nc_mx_matmul(a, b, out)
    for _ in range(3):
        out.zero_()
        junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(8)]     # eager work between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del junk
