"""MX matrices, products and activations used together: a feed-forward block trained
and served, graphs, streams, workspaces."""

import os
import sys

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc
from oracle import mx
from tests._mx import close, data, f64, product, written

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import mx_mlp  # noqa: E402

pytestmark = pytest.mark.gpu


def test_training_step():
    """Every product of the step against the oracle over the very inputs that it had, and the gradients against the
    unquantised block's formula.

    Far apart the latter lie by the casts: an element is off by half a step at most, 2^-4 of itself (E4M3) or 2^-3
    (E5M2), spread evenly 2^-4 / sqrt(3) and 2^-3 / sqrt(3) in the mean square.  Errors of different elements are
    independent, so a result's relative error (2-norm) is the root of the sum of its operands' squares: four E4M3
    operands for out, four more of E4M3 and two of E5M2 at most for a gradient.  Twice that is allowed."""
    r = mx_mlp.train(tokens=300, width=256, hidden=640)
    half8, half5 = 2.0 ** -4 / 3 ** 0.5, 2.0 ** -3 / 3 ** 0.5
    h = 640
    dw_in = dw_out = 0
    tol_in = tol_out = 0
    for s in r["steps"]:
        both, y = s["forward"]["both"], s["forward"]["y"]
        close(both, *product(s["x"], r["w_in"], "e4m3", "e4m3", "bf16"))
        close(s["out"], *product(y, r["w_out"], "e4m3", "e4m3", "bf16"))
        dy, again, dboth = (s["backward"][k] for k in ("dy", "y", "dboth"))
        close(dy, *product(s["dout"], r["w_out"].T.contiguous(), "e5m2", "e4m3", "bf16"))
        close(s["dx"], *product(dboth, r["w_in"].T.contiguous(), "e5m2", "e4m3", "bf16"))
        g, u, d = mx.held(f64(both[:, :h]), "e4m3", "ceil"), mx.held(f64(both[:, h:]), "e4m3", "ceil"), f64(dy)
        f, df, sf, sdf = mx.act(g, "silu")
        for got, want, size in ((again, f * u, sf * np.abs(u)), (dboth[:, :h], d * u * df, sdf * np.abs(d * u)), (dboth[:, h:], d * f, sf * np.abs(d))):
            close(got, want, 2.0 ** -20 * size + 1e-36 + 2.0 ** -7.99 * np.abs(want))
        # weights' gradients: the two micro-batches' sums
        want, tol = product(s["dout"].T.contiguous(), again.T.contiguous(), "e5m2", "e4m3", "fp32")
        dw_out, tol_out = dw_out + want, tol_out + tol
        want, tol = product(dboth.T.contiguous(), s["x"].T.contiguous(), "e5m2", "e4m3", "fp32")
        dw_in, tol_in = dw_in + want, tol_in + tol
        out, dx, _, _ = mx_mlp.formula(r["w_in"], r["w_out"], s["x"], s["dout"])
        assert (s["out"].double() - out).norm() <= 2 * (4 * half8 ** 2) ** 0.5 * out.norm()
        assert (s["dx"].double() - dx).norm() <= 2 * (8 * half8 ** 2 + 2 * half5 ** 2) ** 0.5 * dx.norm()
    close(r["dw_out"], dw_out, tol_out)
    close(r["dw_in"], dw_in, tol_in)
    grads = [mx_mlp.formula(r["w_in"], r["w_out"], s["x"], s["dout"])[2:] for s in r["steps"]]
    for got, want in ((r["dw_in"], grads[0][0] + grads[1][0]), (r["dw_out"], grads[0][1] + grads[1][1])):
        assert (got.double() - want).norm() <= 2 * (8 * half8 ** 2 + 2 * half5 ** 2) ** 0.5 * want.norm()


def test_gradient_against_differences():
    """The block's dx along a direction against differences of the unquantised block in 64 bits: the same bound as
    against the formula (differences of a step 1e-4 are off by some 1e-8)."""
    r = mx_mlp.train(tokens=120, width=128, hidden=256, seed=1)
    s = r["steps"][0]
    d = s["dx"].double() / s["dx"].double().norm()       # the direction of dx itself
    def loss(x):
        return float((mx_mlp.formula(r["w_in"], r["w_out"], x, s["dout"])[0] * s["dout"].double()).sum())
    x = s["x"].double()
    diff = (loss(x + 1e-4 * d) - loss(x - 1e-4 * d)) / 2e-4
    got = float((s["dx"].double() * d).sum())
    bound = 2 * (8 * (2.0 ** -4) ** 2 / 3 + 2 * (2.0 ** -3) ** 2 / 3) ** 0.5
    assert abs(got - diff) <= bound * abs(diff)


@pytest.mark.parametrize("rows", [1, 3, 6, 7, 40])
def test_serving(rows):
    r = mx_mlp.serve(rows=rows, width=288, hidden=600)
    for got, want in zip(r["got"], r["want"]):
        assert torch.equal(got, want) and bool(torch.isfinite(got).all()) and bool(got.any())
    assert not torch.equal(r["got"][0], r["got"][1])


class _Step:
    """One of every call, with buffers of its own."""

    def __init__(self, m=200, n=700, k=5000):
        self.x, self.dy = (torch.empty(m, k, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.w = written(data(np.random.default_rng(5), n, k, "bf16"), "e2m1")
        self.xq, self.xt, self.gq = (nc.new_mx_matrix(*s) for s in ((m, k, "e4m3"), (k, m, "e4m3"), (m, k, "e5m2")))
        self.out, self.lin, self.few = (torch.empty(r, n, device="cuda") for r in (m, m, 4))
        self.acc, self.sum = torch.zeros(k, k // 10, device="cuda"), torch.zeros(m, n, device="cuda")
        self.y, self.dg, self.back = (torch.empty_like(self.x) for _ in range(3))
        self.ws = [nc.new_mx_workspace(m, self.w), nc.new_mx_workspace(m, self.w, "e2m1"), nc.new_mx_workspace(k, self.xt)]
        # xt's bytes as a matrix of fewer rows, whose scales lie where xt has codes: any numbers, NaN among them
        self.small = nc.MxMatrix(self.xt.data, k // 10, m, "e4m3")

    def run(self, stream=None):
        kw = dict(stream=stream)
        nc.nc_mx_write(self.x, self.xq, self.xt, **kw)
        nc.nc_mx_matmul(self.xq, self.w, self.out, ws=self.ws[0], **kw)
        nc.nc_mx_linear(self.x, self.w, self.lin, fmt="e2m1", ws=self.ws[1], **kw)
        nc.nc_mx_linear(self.x[:4], self.w, self.few, fmt="e5m2", ws=self.ws[1], **kw)
        nc.nc_mx_matmul(self.xt, self.small, self.acc, accumulate=True, ws=self.ws[2], **kw)
        nc.nc_mx_matmul(self.xq, self.w, self.sum, accumulate=True, ws=self.ws[0], **kw)
        nc.nc_act_forward(self.x, None, self.y, self.gq, act="gelu", **kw)
        nc.nc_act_backward(self.dy, self.gq, None, self.dg, act="gelu", **kw)
        nc.nc_mx_read(self.gq, self.back, **kw)

    def fill(self, seed):
        rng = np.random.default_rng(seed)
        self.x.copy_(data(rng, *self.x.shape, "bf16"))
        self.dy.copy_(data(rng, *self.x.shape, "bf16"))

    def outputs(self):
        """Bit patterns: NaN compare too."""
        return [t.clone().view(torch.uint8) for t in (self.xq.data, self.xt.data, self.gq.data, self.out, self.lin, self.few, self.acc,
                                                      self.sum, self.y, self.dg, self.back)]


def test_graph_replays():
    """A captured sequence of every call, replayed with new inputs, against eager runs in between; sums that go on
    (accumulate) go on alike."""
    g, e = _Step(), _Step()
    g.fill(1)
    e.fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.run()
    torch.cuda.current_stream().wait_stream(side)
    e.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.run()
    for seed in range(2, 6):
        g.fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        e.fill(seed)
        e.run()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(g.outputs(), e.outputs())):
            assert torch.equal(a, b), (seed, i)


def test_two_graphs_share_a_workspace():
    """Two captured products with one workspace, replayed in turn: splits and quantised rows of one leave nothing that
    the other takes for its own."""
    rng = np.random.default_rng(6)
    w = written(data(rng, 130, 20000, "bf16"), "e4m3")
    xs = [data(rng, m, 20000, "bf16").cuda() for m in (40, 100)]
    ws = nc.new_mx_workspace(100, w, "e4m3")
    assert nc.mx_workspace_bytes(100, w) > 0             # it is cut along the columns
    outs = [torch.empty(x.shape[0], 130, dtype=torch.bfloat16, device="cuda") for x in xs]
    want = [o.clone() for o in outs]
    for x, o in zip(xs, want):
        nc.nc_mx_linear(x, w, o)
    graphs = []
    for x, o in zip(xs, outs):
        nc.nc_mx_linear(x, w, o, ws=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            nc.nc_mx_linear(x, w, o, ws=ws)
    ws.fill_(255)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_two_streams_at_once():
    a, b, a1, b1 = (_Step(k=3000) for _ in range(4))
    for s, seed in ((a, 1), (b, 2), (a1, 1), (b1, 2)):
        s.fill(seed)
    for _ in range(3):
        a1.run()
        b1.run()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    s1.wait_stream(torch.cuda.current_stream())
    s2.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a.run(stream=s1)
        b.run(stream=s2)
    torch.cuda.synchronize()
    for x, y in ((a, a1), (b, b1)):
        for i, (u, v) in enumerate(zip(x.outputs(), y.outputs())):
            assert torch.equal(u, v), i


def test_workspace_from_torch_on_the_calls_stream():
    """ws=None on a side stream: the same result, and the memory is that stream's."""
    rng = np.random.default_rng(7)
    w = written(data(rng, 130, 20000, "bf16"), "e2m1")
    x = data(rng, 70, 20000, "bf16").cuda()
    want = torch.empty(70, 130, device="cuda")
    nc.nc_mx_linear(x, w, want, ws=nc.new_mx_workspace(70, w, "e4m3"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        got = torch.empty(70, 130, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        nc.nc_mx_linear(x, w, got, stream=side)
        side.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("fa,fb,dtype", [("e2m1", "e2m1", "bf16"), ("e4m3", "e4m3", "bf16"), ("e5m2", "e2m1", "bf16"), ("e4m3", "e2m1", "fp32")])
def test_large_tiles(fa, fb, dtype):
    """Enough results for 256 x 256 a workgroup (bf16) or many of 128 x 128, ragged on both sides, against a product of
    the values held in 64 bits on the GPU; tolerance as in the other tests, with the dropped part bounded by eight
    neighbouring columns' largest product each, at most 2^-13 * 8 of the sum over groups of their largest factors."""
    rng = np.random.default_rng(8)
    m, n, k = 4000, 4130, 700
    xa, xb = data(rng, m, k, "bf16").cuda(), data(rng, n, k, "bf16").cuda()
    a, b = written(xa, fa), written(xb, fb)
    va, vb = (torch.empty(r, k, device="cuda") for r in (m, n))
    nc.nc_mx_read(a, va)
    nc.nc_mx_read(b, vb)
    va, vb = va.double(), vb.double()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    out = torch.full((m, n), 3.0, dtype=dt, device="cuda")
    nc.nc_mx_matmul(a, b, out)
    want, mag = va @ vb.T, va.abs() @ vb.abs().T
    tol = (k + 42) * 2.0 ** -23 * mag + torch.finfo(dt).eps / 2 * want.abs()
    if (fa, fb) != ("e2m1", "e2m1") and dtype == "bf16":
        def top(v, emin, x, fmt):                        # largest factor of each group of eight, and the smallest normal one's size
            e = torch.from_numpy(np.ldexp(1.0, mx.exponents(f64(x), fmt, "ceil") + emin)).cuda()
            w = torch.maximum(v.abs(), e)
            return torch.nn.functional.pad(w, (0, -k % 8)).unflatten(1, (-1, 8)).amax(2)
        tol = tol + 8 * 2.0 ** -13 * top(va, mx.EMIN[fa], xa, fa) @ top(vb, mx.EMIN[fb], xb, fb).T
    assert bool(((out.double() - want).abs() <= tol * 1.01).all())
