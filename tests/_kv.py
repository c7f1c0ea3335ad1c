"""Helpers of the key/value-cache tests: host inputs, the cache that a program
would keep, the oracle's results and tolerances counted from the roundings."""

import math

import numpy as np
import torch

import scaled_fp8_casting_amd as nc
from oracle import kv

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rounded(x: np.ndarray, dtype: str) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DT[dtype])


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def paged(rng, lens, page, extra=1):
    """Pages in a random order: table [batch, most pages] (unused entries far out of range),
    slots of every sequence's tokens, page count."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    ids = rng.permutation(pages)
    table = np.full((len(lens), max(max(need, default=0), 1)), 2 ** 31 - 1, dtype=np.int32)
    slots, at = [], 0
    for b, n in enumerate(lens):
        mine = ids[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = mine
        slots.append((mine[:, None] * page + np.arange(page)).reshape(-1)[:n])
    return table, slots, pages


def stale(cache: nc.KvCache, rng):
    """Fill a cache with random bytes, NaN codes and scales among them: what recycled pages hold."""
    b = rng.integers(0, 256, cache.data.numel()).astype(np.uint8)
    b[rng.random(b.size) < 0.2] = 0xFF
    cache.data.copy_(torch.from_numpy(b).view(cache.data.shape))


def tolerance(dim, dtype, out, lse, spread, reach):
    """Bounds on |out - exact| and |lse - exact|.

    A score is a sum of dim exact products in fp32 (three partial sums for fp32
    queries): each of at most dim + 2 additions, and the scaling, is off by at
    most 2^-24 of what has been added up, `reach` at most.  Twice that is a
    weight's relative error against the sum of weights; exp2 and the sums add
    2^-20 at most (1 ulp and (n + 8) roundings of sums of positive terms of
    which the long ones are cut in lanes and waves).  bf16 calls round weights
    and outputs by 2^-8 each."""
    score = (3 * dim + 4) * 2.0 ** -24 * reach + 2.0 ** -23 * np.abs(np.where(np.isfinite(lse), lse, 0))
    rel = 2 * score + 2.0 ** -20
    half = torch.finfo(DT[dtype]).eps / 2
    weights = half if dtype == "bf16" else 0.0
    t_out = (rel + weights)[..., None] * spread * (1 + half) + half * np.abs(out) + 1e-37
    return t_out, score + 2.0 ** -20


def run_case(seed, fmt, dtype, dim, heads, group, lens, q_lens, page, causal=True, window=0, rule="ceil", scale=None,
             sliced=False, max_kv=None, mutate=None, pairs=None, lose=()):
    """One attention call against the oracle; returns what came back.  pairs: so many (sequence, query head) pairs,
    the first and last among them, are compared (all where None).  lose: (sequence, page) entries of the table that
    are sent outside the cache, so that their tokens are not seen."""
    rng = np.random.default_rng(seed)
    table, slots, pages = paged(rng, lens, page)
    cache = nc.new_kv_cache(pages, page, heads, dim, fmt)
    stale(cache, rng)
    total = sum(lens)
    k = rounded(rng.standard_normal((total, heads, dim)) * np.exp(0.7 * rng.standard_normal((heads, dim))), dtype)
    v = rounded(rng.standard_normal((total, heads, dim)) + 0.4 * rng.standard_normal((heads, dim)), dtype)
    q = rounded(1.3 * rng.standard_normal((sum(q_lens), heads * group, dim)), dtype)
    if mutate:
        mutate(k, v, q)
    if total:
        nc.nc_kv_write(cache, k.cuda(), v.cuda(), torch.from_numpy(np.concatenate(slots)).cuda(), rule)
    qd = q.cuda()
    if sliced:                                     # queries inside a wider row, heads outermost in out
        wide = torch.zeros((q.shape[0], heads * group + 2 * heads, dim), dtype=q.dtype, device="cuda")
        wide[:, :heads * group] = qd
        qd = wide[:, :heads * group]
        out = torch.full((heads * group, q.shape[0], dim), 7.0, dtype=q.dtype, device="cuda").transpose(0, 1)
    else:
        out = torch.full_like(qd, 7.0)
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda")
    for b, at in lose:
        table[b, at] = -1 if at % 2 else pages
    starts = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32, device="cuda")
    nc.nc_kv_attention(cache, qd, out, starts, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                       torch.from_numpy(table).cuda(), max(q_lens), max_kv or max(lens), causal=causal, window=window,
                       scale=scale, lse=lse)
    torch.cuda.synchronize()
    hk, hv, hq = kv.held(f64(k), fmt, rule), kv.held(f64(v), fmt, rule), f64(q)
    sc = 1 / math.sqrt(dim) if scale is None else scale
    want_o, want_l = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    tol_o, tol_l = np.zeros(q.shape), np.zeros(q.shape[:2])
    got_o, got_l = f64(out), f64(lse)
    every = len(lens) * heads * group
    picked = set(range(every)) if pairs is None else {0, every - 1, *rng.choice(every, pairs, replace=False).tolist()}
    tk = tq = 0
    for b, (n, n_q) in enumerate(zip(lens, q_lens)):
        mask = kv.seen(n, n_q, causal, window)
        for s, at in lose:
            if s == b:
                mask[:, at * page:(at + 1) * page] = False
        for j in range(heads * group):
            h = j // group
            if b * heads * group + j not in picked:
                got_o[tq:tq + n_q, j], got_l[tq:tq + n_q, j], want_l[tq:tq + n_q, j] = 0, 0, 0
                continue
            r = kv.attend(hq[tq:tq + n_q, j], hk[tk:tk + n, h], hv[tk:tk + n, h], mask, sc)
            want_o[tq:tq + n_q, j], want_l[tq:tq + n_q, j] = r[0], r[1]
            tol_o[tq:tq + n_q, j], tol_l[tq:tq + n_q, j] = tolerance(dim, dtype, *r)
        tk += n
        tq += n_q
    return got_o, got_l, want_o, want_l, tol_o, tol_l


def check(got_o, got_l, want_o, want_l, tol_o, tol_l):
    empty = np.isneginf(want_l)
    assert np.array_equal(np.isneginf(got_l), empty)
    assert np.all(got_o[empty] == 0)
    assert np.array_equal(np.isnan(got_l), np.isnan(want_l))
    assert np.array_equal(np.isnan(got_o), np.isnan(want_o))
    fin = np.isfinite(want_l)
    bad = np.abs(got_l - np.where(fin, want_l, got_l)) > tol_l
    assert not np.any(bad & fin), (np.argwhere(bad & fin)[:4], got_l[bad & fin][:4], want_l[bad & fin][:4])
    d = np.where(np.isnan(want_o), 0, np.abs(got_o - want_o) - tol_o)
    d = np.where(np.isnan(d), 0, d)
    assert d.max(initial=0) <= 0, (np.unravel_index(d.argmax(), d.shape), d.max())
