"""Activations large enough that a workgroup takes a whole chunk of columns (4096 strips
by chunks and more; smaller ones take a step each), results past the caches and not."""

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc
from oracle import mx
from tests._mx import DT, close, f64
from tests.test_gpu_act import ACTS, bound

pytestmark = pytest.mark.gpu

ROWS, COLS = 8200, 4100          # 257 strips by 17 chunks; 64 MiB of bf16
PIECE = 1024                     # rows of a call that takes single steps: 32 strips by 17 chunks
SAMPLE = [0, 1, 31, 32, 4095, 4111, 8191, 8192, 8199]


def planes(n, dtype, stride, seed):
    """Normal values of unequal rows in rows `stride` apart, and what lies between them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(n):
        hold = torch.full((ROWS, stride), 3.0, dtype=DT[dtype], device="cuda")
        x = hold[:, :COLS]
        x.copy_(torch.randn(ROWS, COLS, generator=g, device="cuda") * torch.exp(torch.randn(ROWS, 1, generator=g, device="cuda")))
        out.append(x)
    return out


def room(dtype, stride):
    hold = torch.full((ROWS, stride), 3.0, dtype=DT[dtype], device="cuda")
    return hold, hold[:, :COLS]


def value(m):
    y = torch.empty(m.rows, m.cols, device="cuda")
    nc.nc_mx_read(m, y)
    return y


# rows of bf16 on 16 bytes: results go past the caches; on 8, and on any element: they do not
@pytest.mark.parametrize("stride", [4104, 4100, 4101])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gated,fmt", [(True, "e4m3"), (True, "e2m1"), (False, "e5m2"), (False, "e2m1")])
@pytest.mark.parametrize("act", ACTS)
def test_chunks_equal_steps(act, gated, fmt, dtype, stride):
    """Forward, kept values and gradients bit for bit those of pieces of the rows, and some rows against the oracle."""
    x = planes(3, dtype, stride, seed=stride)
    gate, up, dy = x[0], x[1] if gated else None, x[2]
    gq = nc.new_mx_matrix(ROWS, COLS, fmt)
    uq = nc.new_mx_matrix(ROWS, COLS, fmt) if gated else None
    for q in (gq, uq):
        if q is not None:
            q.data.fill_(255)                            # NaN where nothing is written
    y_hold, y = room(dtype, stride)
    nc.nc_act_forward(gate, up, y, gq, uq, act=act)
    bare = torch.empty(ROWS, COLS, dtype=DT[dtype], device="cuda")
    nc.nc_act_forward(gate, up, bare, act=act)
    assert torch.equal(bare, y)
    (dg_hold, dg), (du_hold, du), (again_hold, again) = (room(dtype, stride) for _ in range(3))
    nc.nc_act_backward(dy, gq, uq, dg, du if gated else None, act=act, y=again)
    for hold in (y_hold, dg_hold, du_hold, again_hold):
        assert bool((hold[:, COLS:] == 3).all())
    gv, uv = value(gq), value(uq) if gated else None
    for at in range(0, ROWS, PIECE):
        s = slice(at, min(at + PIECE, ROWS))
        n = s.stop - at
        pg, pu = nc.new_mx_matrix(n, COLS, fmt), nc.new_mx_matrix(n, COLS, fmt) if gated else None
        part = torch.empty(n, COLS, dtype=DT[dtype], device="cuda")
        nc.nc_act_forward(gate[s], up[s] if gated else None, part, pg, pu, act=act)
        assert torch.equal(part, y[s]) and torch.equal(value(pg), gv[s]) and (not gated or torch.equal(value(pu), uv[s]))
        dp, up_, ap = torch.empty_like(part), torch.empty_like(part) if gated else None, torch.empty_like(part)
        nc.nc_act_backward(dy[s], pg, pu, dp, up_, act=act, y=ap)
        assert torch.equal(dp, dg[s]) and torch.equal(ap, again[s]) and (not gated or torch.equal(up_, du[s]))
    # rows against the definition
    g64, u64, d64 = f64(gate[SAMPLE]), f64(up[SAMPLE]) if gated else 1.0, f64(dy[SAMPLE])
    f, _, sf, _ = mx.act(g64, act)
    close(y[SAMPLE], f * u64, bound(f * u64, sf * np.abs(u64), dtype))
    kept = mx.held(g64, fmt, "ceil")
    assert np.array_equal(f64(gv[SAMPLE]), kept)
    w = mx.held(u64, fmt, "ceil") if gated else 1.0
    assert not gated or np.array_equal(f64(uv[SAMPLE]), w)
    f, df, sf, sdf = mx.act(kept, act)
    close(dg[SAMPLE], d64 * w * df, bound(d64 * w * df, sdf * np.abs(d64 * w), dtype))
    close(again[SAMPLE], f * w, bound(f * w, sf * np.abs(w), dtype))
    if gated:
        close(du[SAMPLE], d64 * f, bound(d64 * f, sf * np.abs(d64), dtype))


@pytest.mark.parametrize("at", [0, 1, 2])
def test_one_result_off_16_bytes(at):
    """Results go past the caches together or not at all: one of three whose rows start on any element."""
    gate, up, dy = planes(3, "bf16", 4104, seed=7)
    gq, uq = nc.new_mx_matrix(ROWS, COLS, "e4m3"), nc.new_mx_matrix(ROWS, COLS, "e4m3")
    y = torch.empty(ROWS, COLS, dtype=torch.bfloat16, device="cuda")
    nc.nc_act_forward(gate, up, y, gq, uq)
    want = [room("bf16", 4104)[1] for _ in range(3)]
    nc.nc_act_backward(dy, gq, uq, want[0], want[1], y=want[2])
    got = [room("bf16", 4101 if i == at else 4104)[1] for i in range(3)]
    nc.nc_act_backward(dy, gq, uq, got[0], got[1], y=got[2])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    nc.nc_act_backward(dy, gq, uq, dy, got[1])           # over dy itself, y not wanted
    assert torch.equal(dy, want[0]) and torch.equal(got[1], want[1])
    nc.nc_act_forward(gate, up, gate)                    # over gate itself
    assert torch.equal(gate, y)


@pytest.mark.parametrize("rows", [70, ROWS])             # single steps, whole chunks
def test_over_their_own_inputs(rows):
    """y over up, dup over dy."""
    gate, up, dy = (x[:rows] for x in planes(3, "bf16", 4104, seed=8))
    gq, uq = nc.new_mx_matrix(rows, COLS, "e5m2"), nc.new_mx_matrix(rows, COLS, "e5m2")
    y, dg, du = (torch.empty(rows, COLS, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    nc.nc_act_forward(gate, up, y, gq, uq, act="gelu")
    nc.nc_act_backward(dy, gq, uq, dg, du, act="gelu")
    kept = value(uq)
    nc.nc_act_forward(gate, up, up, gq, uq, act="gelu")
    assert torch.equal(up, y) and torch.equal(value(uq), kept)
    got = torch.empty_like(dg)
    nc.nc_act_backward(dy, gq, uq, got, dy, act="gelu")
    assert torch.equal(dy, du) and torch.equal(got, dg)
