"""A gated feed-forward block in MX formats, trained and served, on cuda:0.

    python examples/mx_mlp.py [--tokens N] [--width N] [--hidden N]

Training step: every operand of every product is a matrix of MX blocks.  Activations
are cast once, with blocks along both axes from one read: the rows' matrix goes into
the forward product, the transposed one waits for the weights' gradient.  The
activation keeps its inputs in 8 bits; the backward pass takes its gradient from them
and forms its output again for the second weights' gradient, so that nothing is kept
in 16 bits.  Gradients are cast to E5M2, weights' gradients added up in fp32.

Serving: 4-bit weights, activations quantised on the way, one token's pass captured
as a HIP graph and replayed.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scaled_fp8_casting_amd as nc  # noqa: E402

BF16 = torch.bfloat16


def new(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="cuda")


class Block:
    """out = (silu(x Wg^T) * (x Wu^T)) Wd^T, Wg and Wu one matrix [2 hidden, width]."""

    def __init__(self, w_in: torch.Tensor, w_out: torch.Tensor, fmt="e4m3"):
        self.hidden, self.width = w_out.shape[1], w_out.shape[0]
        # laid out once: rows for the forward products, transposed for the backward ones
        self.w_in, self.w_in_t = nc.new_mx_matrix(*w_in.shape, fmt), nc.new_mx_matrix(*w_in.T.shape, fmt)
        self.w_out, self.w_out_t = nc.new_mx_matrix(*w_out.shape, fmt), nc.new_mx_matrix(*w_out.T.shape, fmt)
        nc.nc_mx_write(w_in, self.w_in, self.w_in_t)
        nc.nc_mx_write(w_out, self.w_out, self.w_out_t)

    @staticmethod
    def cast(x, fmt, rows=True, cols=True):
        """x as a matrix and as a transposed one, from one read."""
        m = nc.new_mx_matrix(*x.shape, fmt) if rows else None
        t = nc.new_mx_matrix(*x.T.shape, fmt) if cols else None
        nc.nc_mx_write(x, m, t)
        return m, t

    def forward(self, x):
        """The block's output and what its backward pass needs."""
        tokens, h = x.shape[0], self.hidden
        xq, xt = self.cast(x, "e4m3")
        both, y, out = new(tokens, 2 * h), new(tokens, h), new(tokens, self.width)
        nc.nc_mx_matmul(xq, self.w_in, both)
        gate_q, up_q = nc.new_mx_matrix(tokens, h, "e4m3"), nc.new_mx_matrix(tokens, h, "e4m3")
        nc.nc_act_forward(both[:, :h], both[:, h:], y, gate_q, up_q)
        yq, _ = self.cast(y, "e4m3", cols=False)
        nc.nc_mx_matmul(yq, self.w_out, out)
        return out, (xt, gate_q, up_q), {"both": both, "y": y}

    def backward(self, dout, kept, dw_in, dw_out):
        """dx; the weights' gradients are added to dw_in and dw_out (fp32)."""
        xt, gate_q, up_q = kept
        tokens, h = dout.shape[0], self.hidden
        dq, dt = self.cast(dout, "e5m2")
        dy, y, dboth, dx = new(tokens, h), new(tokens, h), new(tokens, 2 * h), new(tokens, self.width)
        nc.nc_mx_matmul(dq, self.w_out_t, dy)
        nc.nc_act_backward(dy, gate_q, up_q, dboth[:, :h], dboth[:, h:], y=y)
        _, yt = self.cast(y, "e4m3", rows=False)
        nc.nc_mx_matmul(dt, yt, dw_out, accumulate=True)
        dbq, dbt = self.cast(dboth, "e5m2")
        nc.nc_mx_matmul(dbq, self.w_in_t, dx)
        nc.nc_mx_matmul(dbt, xt, dw_in, accumulate=True)
        return dx, {"dy": dy, "y": y, "dboth": dboth}


class Server:
    """The block for a fixed number of rows with every buffer in place: its pass can be captured."""

    def __init__(self, block: Block, rows: int, fmt="e4m3"):
        self.block, self.fmt, h = block, fmt, block.hidden
        self.x, self.both, self.y, self.out = new(rows, block.width), new(rows, 2 * h), new(rows, h), new(rows, block.width)
        self.ws_in, self.ws_out = nc.new_mx_workspace(rows, block.w_in, fmt), nc.new_mx_workspace(rows, block.w_out, fmt)

    def run(self):
        b, h = self.block, self.block.hidden
        nc.nc_mx_linear(self.x, b.w_in, self.both, fmt=self.fmt, ws=self.ws_in)
        nc.nc_act_forward(self.both[:, :h], self.both[:, h:], self.y)
        nc.nc_mx_linear(self.y, b.w_out, self.out, fmt=self.fmt, ws=self.ws_out)


def train(tokens=300, width=256, hidden=640, seed=0):
    """One step over two micro-batches; inputs, results and gradients."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    w_in, w_out = (randn(2 * hidden, width) / width ** 0.5).to(BF16), (randn(width, hidden) / hidden ** 0.5).to(BF16)
    block = Block(w_in, w_out)
    dw_in, dw_out = torch.zeros(2 * hidden, width, device="cuda"), torch.zeros(width, hidden, device="cuda")
    steps = []
    for n in (tokens, tokens // 3 + 1):
        x, dout = randn(n, width).to(BF16), (1e-3 * randn(n, width)).to(BF16)
        out, kept, seen = block.forward(x)
        dx, more = block.backward(dout, kept, dw_in, dw_out)
        steps.append(dict(x=x, dout=dout, out=out, dx=dx, forward=seen, backward=more))
    return dict(w_in=w_in, w_out=w_out, dw_in=dw_in, dw_out=dw_out, steps=steps)


def serve(rows=1, width=256, hidden=640, tokens=4, seed=0):
    """`tokens` passes of the captured graph: inputs, results, and what eager passes give."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w_in = (torch.randn(2 * hidden, width, generator=g, device="cuda") / width ** 0.5).to(BF16)
    w_out = (torch.randn(width, hidden, generator=g, device="cuda") / hidden ** 0.5).to(BF16)
    block = Block(w_in, w_out, "e2m1")
    captured, eager = Server(block, rows), Server(block, rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.run()
    got, want = [], []
    for _ in range(tokens):
        x = torch.randn(rows, width, generator=g, device="cuda").to(BF16)
        captured.x.copy_(x)
        graph.replay()
        eager.x.copy_(x)
        eager.run()
        torch.cuda.synchronize()
        got.append(captured.out.clone())
        want.append(eager.out.clone())
    return dict(w_in=w_in, w_out=w_out, got=got, want=want)


def formula(w_in, w_out, x, dout):
    """Output and gradients of the unquantised block, in 64 bits."""
    with torch.enable_grad():
        a, b, x = (v.double().requires_grad_() for v in (w_in, w_out, x))
        g, u = (x @ a.T).chunk(2, 1)
        out = (torch.nn.functional.silu(g) * u) @ b.T
        grads = torch.autograd.grad(out, (x, a, b), dout.double())
    return out.detach(), *grads


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=11008)
    a = ap.parse_args()
    r = train(a.tokens, a.width, a.hidden)
    s = r["steps"][0]
    out, dx, _, _ = formula(r["w_in"], r["w_out"], s["x"], s["dout"])
    for name, got, want in (("out", s["out"], out), ("dx", s["dx"], dx)):
        print(f"{name}: {float((got.double() - want).norm() / want.norm()):.3f} of its size from the unquantised block's")
    r = serve(1, a.width, a.hidden)
    same = all(torch.equal(x, y) for x, y in zip(r["got"], r["want"]))
    print(f"served {len(r['got'])} tokens from a graph; equal to eager passes: {same}")


if __name__ == "__main__":
    main()
