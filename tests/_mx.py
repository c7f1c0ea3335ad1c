"""Helpers of the MX-matrix tests: host inputs, matrices written on the GPU, and
tolerances counted from the roundings."""

import numpy as np
import torch

import scaled_fp8_casting_amd as nc
from oracle import mx

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
FMTS = ("e2m1", "e4m3", "e5m2")


def rounded(x: np.ndarray, dtype: str) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DT[dtype])


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def data(rng, rows, cols, dtype, tail=0.0) -> torch.Tensor:
    """Normal values, with `tail` log-normal spread, on the host."""
    return rounded(rng.standard_normal((rows, cols)) * np.exp(tail * rng.standard_normal((rows, cols))), dtype)


def stale(m: nc.MxMatrix, rng):
    """Random bytes, NaN codes and scales among them: what reused memory holds."""
    b = rng.integers(0, 256, m.data.numel()).astype(np.uint8)
    b[rng.random(b.size) < 0.2] = 0xFF
    m.data.copy_(torch.from_numpy(b))
    return m


def written(x: torch.Tensor, fmt: str, rule="ceil") -> nc.MxMatrix:
    m = nc.new_mx_matrix(x.shape[0], x.shape[1], fmt)
    nc.nc_mx_write(x.cuda(), m, rule=rule)
    return m


def product(xa: torch.Tensor, xb: torch.Tensor, fa, fb, dtype, rule_a="ceil", rule_b="ceil", add=None):
    """Values of a b^T (+ add) and the bound on what a product call may be off by.

    fp32 sums of n products, in any order and cut instead of rounded, are off by at
    most n + 2 times 2^-23 of the sum of magnitudes; waves' and splits' partial sums,
    bias and what is there add 40 such steps.  Then what the instruction drops (bf16
    results only), and the result's own rounding."""
    a64, b64 = f64(xa), f64(xb)
    a, b = mx.held(a64, fa, rule_a), mx.held(b64, fb, rule_b)
    out, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    if add is not None:
        out, mag = out + add, mag + np.abs(add)
    tol = (a.shape[1] + 42) * 2.0 ** -23 * mag + 1e-37
    if dtype == "bf16":
        tol = tol + mx.dropped(a, b, fa, fb, mx.exponents(a64, fa, rule_a), mx.exponents(b64, fb, rule_b))
    half = torch.finfo(DT[dtype]).eps / 2
    return out, tol * (1 + half) + half * np.abs(out)


def close(got: torch.Tensor, want: np.ndarray, tol: np.ndarray):
    g = f64(got)
    assert np.array_equal(np.isnan(g), np.isnan(want))
    ok = np.isnan(want) | (np.abs(g - np.where(np.isnan(want), 0, want)) <= tol)
    bad = np.argwhere(~ok)
    assert ok.all(), (len(bad), bad[:4].tolist(), g[tuple(bad[0])], want[tuple(bad[0])], tol[tuple(bad[0])])
