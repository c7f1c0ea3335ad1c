"""The key/value cache and attention over it, from their definitions, in binary64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

``held`` is what a cache holds of a row: blocks of 32 elements share 2^X, X from
the block's largest finite magnitude a = m 2^e by the rule (OCP X = e - emax;
PLUS1 one more; CEIL the smallest X with a 2^-X <= max), and every element is the
nearest value of the format's grid times 2^X, ties to the even code, saturating.
All steps are exact in binary64 for fp32 inputs.

``attend`` is softmax attention of one sequence, row by row, in binary64; it also
returns what the tests' tolerances are made of.
"""

import numpy as np


def grid(fmt: str) -> np.ndarray:
    """Non-negative finite values in the order of their codes."""
    if fmt == "e2m1":
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    sub = [j * 2.0 ** -9 for j in range(8)]
    return np.array((sub + [(8 + j) / 8 * 2.0 ** e for e in range(-6, 9) for j in range(8)])[:127])


def block_exponent(fmt: str, a: np.ndarray, rule: str) -> np.ndarray:
    """X of blocks whose largest finite magnitude is a (binary64, >= 0)."""
    top = grid(fmt)[-1]
    emax = 2 if fmt == "e2m1" else 8
    _, e = np.frexp(np.where(a > 0, a, 1.0))              # a = f 2^e, f in [1/2, 1)
    X = e - 1 - emax
    if rule == "plus1":
        X = X + 1
    elif rule == "ceil":
        X = X + (a > np.ldexp(top, X))
    elif rule != "ocp":
        raise ValueError(rule)
    return np.where(a > 0, np.clip(X, -127, 127), -127)


def held(x: np.ndarray, fmt: str, rule: str) -> np.ndarray:
    """What the cache holds of x [..., dim] (fp32 values), as binary64."""
    g = grid(fmt)
    b = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    mag = np.abs(b)
    fin = np.isfinite(b)
    X = block_exponent(fmt, np.where(fin, mag, 0.0).max(-1, initial=0.0), rule)[..., None]
    y = np.where(fin, np.ldexp(np.where(fin, mag, 0.0), -X), g[-1])
    y = np.minimum(y, g[-1])
    hi = np.minimum(np.searchsorted(g, y), len(g) - 1)    # g[hi - 1] < y <= g[hi]
    lo = np.maximum(hi - 1, 0)
    up = (g[hi] - y < y - g[lo]) | ((g[hi] - y == y - g[lo]) & (hi % 2 == 0))
    v = np.copysign(np.ldexp(np.where(up, g[hi], g[lo]), X), b)
    nan = np.isnan(b)
    if fmt == "e2m1":                                     # no NaN code: the block reads as NaN
        nan = np.broadcast_to(nan.any(-1, keepdims=True), nan.shape)
    return np.where(nan, np.nan, v).reshape(x.shape)


def seen(n: int, n_q: int, causal: bool, window: int) -> np.ndarray:
    """[n_q, n]: which tokens each query sees."""
    end = (n - n_q + 1 + np.arange(n_q) if causal else np.full(n_q, n))[:, None]
    t = np.arange(n)[None, :]
    ok = t < end
    return ok & (t >= end - window) if window else ok


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, mask: np.ndarray, scale: float):
    """One query head over one cache head: q [n_q, dim], k and v [n, dim], mask [n_q, n].

    Returns out, lse, spread = sum_t w_t |v_t| (what a relative error of the
    weights w can move), and reach = max_t |scale| sum_d |q_d k_d| over the seen
    tokens (what a relative error of the products can move a score by)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    n_q, dim = q.shape
    out, spread = np.zeros((n_q, v.shape[1])), np.zeros((n_q, v.shape[1]))
    lse, reach = np.full(n_q, -np.inf), np.zeros(n_q)
    for i in range(n_q):
        kk, vv = k[mask[i]], v[mask[i]]
        if not len(kk):
            continue
        s = scale * (kk @ q[i])
        top = s.max()
        w = np.exp(s - top)
        lse[i] = top + np.log(w.sum())
        w /= w.sum()
        out[i], spread[i] = w @ vv, w @ np.abs(vv)
        reach[i] = abs(scale) * (np.abs(kk) @ np.abs(q[i])).max()
    return out, lse, spread, reach
