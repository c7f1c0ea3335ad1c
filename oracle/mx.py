"""MX matrices, their products and activations over what they hold, from their
definitions, in binary64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

``held`` is what a matrix holds of x [rows, cols]: 32 consecutive elements of a row
(fewer at its end) share 2^X, X from their largest finite magnitude a = m 2^e by the
rule (OCP X = e - emax; PLUS1 one more; CEIL the smallest X with a 2^-X <= max); every
element is the nearest value of the format's grid times 2^X, ties to the even code,
saturating.  All steps are exact in binary64 for fp32 inputs.
"""

import math

import numpy as np

EMAX = {"e2m1": 2, "e4m3": 8, "e5m2": 15}
EMIN = {"e2m1": 0, "e4m3": -6, "e5m2": -14}


def grid(fmt: str) -> np.ndarray:
    """Non-negative finite values in the order of their codes."""
    mb = {"e2m1": 1, "e4m3": 3, "e5m2": 2}[fmt]
    n = 1 << mb
    g = [j / n * 2.0 ** EMIN[fmt] for j in range(n)]
    g += [(n + j) / n * 2.0 ** e for e in range(EMIN[fmt], EMAX[fmt] + 1) for j in range(n)]
    return np.array(g[:-1] if fmt == "e4m3" else g)      # E4M3's last one is its NaN


def exponents(x: np.ndarray, fmt: str, rule: str) -> np.ndarray:
    """X of every element of x [rows, cols]."""
    rows, cols = x.shape
    a = np.zeros((rows, -(-cols // 32) * 32))
    a[:, :cols] = np.where(np.isfinite(x), np.abs(x), 0.0)
    a = a.reshape(rows, -1, 32).max(-1, initial=0.0)
    _, e = np.frexp(np.where(a > 0, a, 1.0))              # a = f 2^e, f in [1/2, 1)
    X = e - 1 - EMAX[fmt]
    if rule == "plus1":
        X = X + 1
    elif rule == "ceil":
        X = X + (a > np.ldexp(grid(fmt)[-1], X))
    elif rule != "ocp":
        raise ValueError(rule)
    X = np.where(a > 0, np.clip(X, -127, 127), -127)
    return np.repeat(X, 32, 1)[:, :cols]


def held(x: np.ndarray, fmt: str, rule: str) -> np.ndarray:
    """What a matrix holds of x [rows, cols] (fp32 values), as binary64."""
    x = np.asarray(x, dtype=np.float64)
    g = grid(fmt)
    fin = np.isfinite(x)
    X = exponents(x, fmt, rule)
    y = np.minimum(np.where(fin, np.ldexp(np.where(fin, np.abs(x), 0.0), -X), g[-1]), g[-1])
    hi = np.minimum(np.searchsorted(g, y), len(g) - 1)    # g[hi - 1] < y <= g[hi]
    lo = np.maximum(hi - 1, 0)
    up = (g[hi] - y < y - g[lo]) | ((g[hi] - y == y - g[lo]) & (hi % 2 == 0))
    v = np.copysign(np.ldexp(np.where(up, g[hi], g[lo]), X), x)
    nan = np.isnan(x)
    if fmt == "e2m1":                                     # no NaN code: the block reads as NaN
        rows, cols = x.shape
        n = np.zeros((rows, -(-cols // 32) * 32), dtype=bool)
        n[:, :cols] = nan
        nan = np.repeat(n.reshape(rows, -1, 32).any(-1), 32, 1)[:, :cols]
    return np.where(nan, np.nan, v)


def dropped(a, b, fa, fb, xa, xb) -> np.ndarray:
    """Bound on what the scaled matrix instruction drops of a b^T (a, b: values held, xa, xb: their exponents).
    In groups of eight columns a product keeps its bits down to 2^-13 of the largest
    exponent sum's; an element's exponent is its own, or the smallest normal one."""
    if fa == fb == "e2m1":
        return np.zeros((a.shape[0], b.shape[0]))
    pad = -a.shape[1] % 8
    a = np.maximum(np.abs(a), np.ldexp(1.0, xa + EMIN[fa]))
    b = np.maximum(np.abs(b), np.ldexp(1.0, xb + EMIN[fb]))
    a, b = (np.pad(v, ((0, 0), (0, pad))).reshape(v.shape[0], -1, 8) for v in (a, b))
    out = np.zeros((a.shape[0], b.shape[0]))
    for k in range(a.shape[1]):
        out += (a[:, None, k] * b[None, :, k]).max(-1)
    return 8 * 2.0 ** -13 * out


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1 / (1 + e), e / (1 + e))


def act(z: np.ndarray, kind: str):
    """f(z), f'(z), and what relative errors of fp32 steps move them by (in units of 2^-20)."""
    z = np.asarray(z, dtype=np.float64)
    if kind == "silu":
        s, c = _sigmoid(z), _sigmoid(-z)
        return z * s, s * (1 + z * c), np.abs(z * s), s * (1 + np.abs(z))
    if kind == "gelu":
        phi = np.array([0.5 * math.erfc(-v * math.sqrt(0.5)) for v in z.reshape(-1)]).reshape(z.shape)
        pdf = np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        grow = 1 + z * z                                  # erfc and exp of arguments off by 2^-24 of themselves
        return z * phi, phi + z * pdf, grow * np.abs(z * phi), grow * (phi + np.abs(z) * pdf)
    if kind == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        u, du = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)
        s, t = _sigmoid(u), _sigmoid(-u)
        grow = 1 + np.minimum(np.abs(u), 320.0)
        return z * s, s + z * s * t * du, grow * np.abs(z * s), s * (grow + np.abs(z * du) * (1 + grow * t))
    r = np.maximum(z, 0)
    return r * r, 2 * r, r * r, 2 * r
