"""The key/value-cache operators as they are measured: writing a cache in a narrow
format, reading it back, and attention over it for single tokens, prompts and an
encoder's states.

A cache holds keys and values of `heads` heads in pages of `page` tokens, as MX
blocks: 32 consecutive elements of a head's row share a power of two 2^X, and each
element is a code of E2M1 (4 bits: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) or of E4M3
(8 bits, largest value 448).  X follows from the block's largest magnitude a = m 2^e
by a rule: "ocp" X = e - emax, "plus1" one more, "ceil" the smallest X with
a 2^-X <= max; elements round to nearest even and saturate.  A token's place is its
slot, page * page_size + offset.

With `own` false, `run` computes everything with elementary torch operations in
fp32; with `own` true it makes the library's calls.
"""

import math

import numpy as np
import torch

own = False

FORMATS = {  # largest value, exponent of it, mantissa bits, smallest normal exponent
    "e2m1": (6.0, 2, 1, 0),
    "e4m3": (448.0, 8, 3, -6),
}
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # a step of 32 running sequences writes one token each, and reads it back
        dict(name="write_step", op="write", fmt="e2m1", dtype="bf16", rule="ceil", tokens=32, heads=8, dim=128,
             page=16, sliced=True),
        # a long prompt's keys and values, slices of one fused projection
        dict(name="write_prompt", op="write", fmt="e2m1", dtype="bf16", rule="ceil", tokens=16384, heads=8, dim=128,
             page=64, sliced=True),
        # fp32 keys and values, an odd number of tokens and heads, 8-bit codes
        dict(name="write_fp32_odd", op="write", fmt="e4m3", dtype="fp32", rule="plus1", tokens=3001, heads=5, dim=96,
             page=32, sliced=False),
        # a long shared prefix is brought back in full
        dict(name="read_prefix", op="read", fmt="e2m1", dtype="bf16", rule="ceil", tokens=131072, heads=8, dim=128,
             page=64),
        # a few hundred scattered tokens of an 8-bit cache, in fp32
        dict(name="read_scattered", op="read", fmt="e4m3", dtype="fp32", rule="ocp", tokens=777, heads=6, dim=64,
             page=16),
        # one sequence's next token over a short history: latency
        dict(name="token_short", op="attend", fmt="e2m1", dtype="bf16", batch=1, q=1, kv=517, ragged=False, heads=8,
             group=4, dim=128, page=16, causal=True, window=0),
        # the next token of 64 sequences of unequal length
        dict(name="token_batch", op="attend", fmt="e2m1", dtype="bf16", batch=64, q=1, kv=8192, ragged=True, heads=8,
             group=4, dim=128, page=64, causal=True, window=0),
        # the next token of one very long sequence
        dict(name="token_long", op="attend", fmt="e2m1", dtype="bf16", batch=1, q=1, kv=262144, ragged=False, heads=8,
             group=4, dim=128, page=64, causal=True, window=0),
        # one head of keys for each of queries, fp32, 8-bit cache
        dict(name="token_fp32", op="attend", fmt="e4m3", dtype="fp32", batch=24, q=1, kv=2500, ragged=True, heads=12,
             group=1, dim=64, page=32, causal=True, window=0),
        # five proposed tokens of each sequence are checked at once, under a sliding window
        dict(name="verify_window", op="attend", fmt="e2m1", dtype="bf16", batch=16, q=5, kv=4001, ragged=True, heads=4,
             group=8, dim=128, page=16, causal=True, window=1024),
        # a chunk of a prompt over what is cached of it
        dict(name="prompt_chunk", op="attend", fmt="e2m1", dtype="bf16", batch=1, q=4096, kv=16384, ragged=False,
             heads=8, group=4, dim=128, page=64, causal=True, window=0),
        # a decoder's prompt over an encoder's states of another, unequal length
        dict(name="cross_encoder", op="attend", fmt="e4m3", dtype="bf16", batch=8, q=448, kv=1500, ragged=True,
             heads=16, group=1, dim=64, page=16, causal=False, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes spread over the listed ones' ranges, odd ones among them."""
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    fmt = rng.choice(["e2m1", "e2m1", "e4m3"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    page = rng.choice([16, 32, 48, 64, 128])
    if op != "attend":
        heads = rng.choice([1, 2, 3, 5, 8])
        most = (16384 if op == "write" else 131072) * 8 * 128 // (heads * dim * (2 if dtype == "fp32" else 1))
        c = dict(op=op, fmt=fmt, dtype=dtype, rule=rng.choice(["ocp", "plus1", "ceil"]),
                 tokens=_log(rng, 8, min(most, 100000)), heads=heads, dim=dim, page=page)
        if op == "write":
            c["sliced"] = rng.random() < 0.5
        return c
    kind = rng.choice(["token", "token", "few", "prompt", "cross"])
    heads, group = rng.choice([(8, 4), (4, 8), (2, 6), (12, 1), (1, 16), (5, 3)])
    batch = _log(rng, 1, 48) if kind in ("token", "few") else rng.choice([1, 2, 3, 5])
    q = {"token": 1, "few": rng.randint(2, 9)}.get(kind) or _log(rng, 16, 1500)
    if kind == "cross":
        kv = _log(rng, 40, 3001)
    elif kind == "prompt":
        kv = q + rng.choice([0, 0, _log(rng, 16, 6000)])
    else:
        kv = _log(rng, 33, min(262144, 400000 // batch))
    return dict(op=op, fmt=fmt, dtype=dtype, batch=batch, q=q, kv=kv, ragged=rng.random() < 0.6, heads=heads,
                group=group, dim=dim, page=page, causal=kind != "cross",
                window=_log(rng, 32, 2048) if kind != "cross" and rng.random() < 0.25 else 0)


# ---- inputs -------------------------------------------------------------------

def _lengths(case, seed):
    """Cached tokens of each sequence (host): all `kv`, or from `kv` down to an eighth of it."""
    if not case["ragged"]:
        return [case["kv"]] * case["batch"]
    r = np.random.default_rng(seed * 7919 + case["kv"])
    low = max(min(case["q"], case["kv"]) if case["causal"] else 1, case["kv"] // 8)
    lens = r.integers(low, case["kv"] + 1, case["batch"]).tolist()
    lens[int(r.integers(case["batch"]))] = case["kv"]
    return lens


def _inputs(case, seed):
    """Everything that a pass reads, before any of it is cast or laid out."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt = "cuda", DTYPES[case["dtype"]]
    heads, dim, page = case["heads"], case["dim"], case["page"]

    def keys_and_values(tokens):
        # keys have a few strong channels per head, values a mean of their own per channel
        chan = torch.exp(0.7 * torch.randn(heads, dim, generator=g, device=dev)) * 0.6
        mean = 0.4 * torch.randn(heads, dim, generator=g, device=dev)
        k = (torch.randn(tokens, heads, dim, generator=g, device=dev) * chan).to(dt)
        v = (torch.randn(tokens, heads, dim, generator=g, device=dev) + mean).to(dt)
        return k, v

    s = {"case": case}
    if case["op"] != "attend":
        tokens = case["tokens"]
        pages = -(-tokens // page) + 2
        k, v = keys_and_values(tokens)
        if case["op"] == "write" and case["sliced"]:      # one projection's rows: queries, keys, values
            rows = torch.randn(tokens, 3 * heads, dim, generator=g, device=dev).to(dt)
            rows[:, heads:2 * heads], rows[:, 2 * heads:] = k, v
            k, v = rows[:, heads:2 * heads], rows[:, 2 * heads:]
        # whole pages in an order of their own, as a pool hands them out
        order = torch.randperm(pages, generator=g, device=dev)
        slots = (order[:, None] * page + torch.arange(page, device=dev)).reshape(-1)[:tokens].contiguous()
        s.update(k=k, v=v, slots=slots, pages=pages)
        return s
    lens = _lengths(case, seed)
    batch, q = case["batch"], case["q"]
    per = -(-case["kv"] // page)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.zeros(batch, per, dtype=torch.int32)
    slots, at = [], 0
    for b, n in enumerate(lens):
        mine = ids[at:at + need[b]]
        table[b, :need[b]] = mine
        slots.append((mine.long()[:, None] * page + torch.arange(page)).reshape(-1)[:n])
        at += need[b]
    k, v = keys_and_values(sum(lens))
    x = torch.randn(batch * q, heads * case["group"], dim, generator=g, device=dev)
    s.update(k=k, v=v, slots=torch.cat(slots).to(dev), pages=pages, lens=lens, table=table.to(dev), q=(1.3 * x).to(dt),
             kv_len=torch.tensor(lens, dtype=torch.int32, device=dev),
             q_start=(torch.arange(batch + 1, dtype=torch.int32) * q).to(dev))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    heads, dim, page, pages, dt = case["heads"], case["dim"], case["page"], s["pages"], DTYPES[case["dtype"]]
    if own:
        import scaled_fp8_casting_amd as nc
        s["cache"] = nc.new_kv_cache(pages, page, heads, dim, case["fmt"])
    else:
        s["cache"] = [torch.zeros(pages * page, heads, w, dtype=torch.uint8, device="cuda")
                      for w in (dim, dim // 32, dim, dim // 32)]
        s["table_of"] = _decode_table(case["fmt"])
    if case["op"] != "write":                             # the cache is there before the call
        if own:
            nc.nc_kv_write(s["cache"], s["k"], s["v"], s["slots"], case.get("rule", "ceil"))
        else:
            _plain_write(s["cache"], s["k"], s["v"], s["slots"], case["fmt"], case.get("rule", "ceil"))
        del s["k"], s["v"]
    if own:
        if case["op"] == "attend":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
            s["ws"] = nc.new_kv_workspace(s["cache"], s["q"], case["batch"], case["q"], case["kv"])
        else:
            s["k_out"] = torch.empty(case["tokens"], heads, dim, dtype=dt, device="cuda")
            s["v_out"] = torch.empty_like(s["k_out"])
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import scaled_fp8_casting_amd as nc
    case = s["case"]
    if case["op"] == "attend":
        nc.nc_kv_attention(s["cache"], s["q"], s["out"], s["q_start"], s["kv_len"], s["table"], case["q"], case["kv"],
                           causal=case["causal"], window=case["window"], lse=s["lse"], ws=s["ws"])
        return s["out"], s["lse"]
    if case["op"] == "write":
        nc.nc_kv_write(s["cache"], s["k"], s["v"], s["slots"], case["rule"])
    nc.nc_kv_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
    return s["k_out"], s["v_out"]


# ---- the plain form -------------------------------------------------------------

def _pow2(n):
    """2^n as fp32, exactly (n whole, clamped to the normal range: exp2 may be an ulp off)."""
    return ((n.clamp(-126, 127).to(torch.int32) + 127) << 23).view(torch.float32)


def _decode_table(fmt):
    """The value of every code as fp32, on the GPU."""
    top, _, mb, emin = FORMATS[fmt]
    half = 8 if fmt == "e2m1" else 128
    i = torch.arange(half, device="cuda")
    e, m = i >> mb, i & ((1 << mb) - 1)
    mag = torch.where(e == 0, m.float(), (m + (1 << mb)).float() * _pow2((e - 1).clamp(min=0)))
    mag = mag * 2.0 ** (emin - mb)
    if fmt == "e4m3":
        mag[half - 1] = math.nan
    return torch.cat([mag, -mag])


def _plain_codes(x, fmt, rule):
    """x [..., dim] -> codes, one a byte, and scale bytes X + 127."""
    top, emax, mb, emin = FORMATS[fmt]
    bits = 3 if fmt == "e2m1" else 7
    b = x.float().unflatten(-1, (-1, 32))
    a = b.abs().amax(-1)
    X = torch.frexp(a).exponent - 1 - emax
    if rule == "plus1":
        X = X + 1
    elif rule == "ceil":
        X = X + (a * _pow2(-X) > top)
    X = torch.where(a == 0, -127, X.clamp(-127, 127))
    y = b.abs() * _pow2(-X)[..., None]
    e = (torch.frexp(y).exponent - 1).clamp(min=emin)
    steps = torch.round(y * _pow2(mb - e))
    index = (e - emin) * (1 << mb) + steps.to(torch.int32)
    most = 7 if fmt == "e2m1" else 126
    codes = index.clamp(max=most) + (torch.signbit(b).to(torch.int32) << bits)
    return codes.flatten(-2).to(torch.uint8), (X + 127).to(torch.uint8)


def _plain_write(cache, k, v, slots, fmt, rule):
    for x, codes, scales in ((k, cache[0], cache[1]), (v, cache[2], cache[3])):
        c, sc = _plain_codes(x, fmt, rule)
        codes[slots] = c
        scales[slots] = sc


def _plain_values(codes, scales, slots, table):
    """fp32 values [tokens..., heads, dim] of the tokens at `slots`."""
    val = table[codes[slots].int()].unflatten(-1, (-1, 32))
    return (val * _pow2(scales[slots].int() - 127)[..., None]).flatten(-2)


def _plain(s):
    case, cache = s["case"], s["cache"]
    if case["op"] != "attend":
        if case["op"] == "write":
            _plain_write(cache, s["k"], s["v"], s["slots"], case["fmt"], case["rule"])
        dt = DTYPES[case["dtype"]]
        return tuple(_plain_values(cache[i], cache[i + 1], s["slots"], s["table_of"]).to(dt) for i in (0, 2))
    batch, q, kv, page, group = case["batch"], case["q"], case["kv"], case["page"], case["group"]
    heads, dim = case["heads"], case["dim"]
    at = torch.arange(kv, device="cuda")
    slots = s["table"][:, at // page].long() * page + at % page                       # [batch, kv]
    keys = _plain_values(cache[0], cache[1], slots, s["table_of"]).transpose(1, 2)     # [batch, heads, kv, dim]
    vals = _plain_values(cache[2], cache[3], slots, s["table_of"]).transpose(1, 2)
    x = s["q"].float().view(batch, q, heads, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, heads, q * group, dim)
    score = torch.matmul(x, keys.transpose(2, 3)) * (1.0 / math.sqrt(dim))             # [batch, heads, rows, kv]
    # a query at place i of q sees keys up to kv_len - q + i, and `window` of them at most
    last = s["kv_len"].long()[:, None] - 1
    if case["causal"]:
        last = last - (q - 1) + torch.arange(q, device="cuda")
    else:
        last = last.expand(batch, q)
    seen = at <= last[..., None]
    if case["window"]:
        seen = seen & (at > last[..., None] - case["window"])
    seen = seen[:, None, :, None].expand(batch, 1, q, group, kv).reshape(batch, 1, q * group, kv)
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, vals) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.view(batch, heads, q, group, dim).permute(0, 2, 1, 3, 4).reshape(batch * q, heads * group, dim)
    lse = lse.view(batch, heads, q, group).permute(0, 2, 1, 3).reshape(batch * q, heads * group)
    return out.to(s["q"].dtype), lse


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    bits = 4 if case["fmt"] == "e2m1" else 8
    size = 2 if case["dtype"] == "bf16" else 4
    heads, dim = case["heads"], case["dim"]
    row = dim * bits // 8 + dim // 32                     # a head's cached row
    if case["op"] != "attend":
        n = case["tokens"]
        moved = 2 * n * heads * (row + dim * size) + 8 * n
        if case["op"] == "write":
            moved += 2 * n * heads * (row + dim * size)
        return {"bytes": moved, "flops": 0}
    # lengths are those of seed 1; other seeds' differ little in sum
    lens, q, group = _lengths(case, 1), case["q"], case["group"]
    pairs = rows = 0
    for n in lens:
        lo = n
        for i in range(q):
            end = max(0, n - q + 1 + i) if case["causal"] else n
            start = max(0, end - case["window"]) if case["window"] else 0
            pairs += end - start
            if end:
                lo = min(lo, start)
        rows += n - lo
    io = len(lens) * q * heads * group * (2 * dim * size + 4)
    return {"bytes": 2 * rows * heads * row + io, "flops": 4 * pairs * heads * group * dim}


# ---- the definition in 64 bits -----------------------------------------------------

def _exact_grid(fmt):
    """The non-negative finite values, ascending; a value's place is its code."""
    if fmt == "e2m1":
        return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    sub = [j * 2.0 ** -9 for j in range(8)]
    nor = [(8 + j) / 8 * 2.0 ** e for e in range(-6, 9) for j in range(8)]
    return torch.tensor((sub + nor)[:127], dtype=torch.float64, device="cuda")


def _exact_pow2(n):
    """2^n as a 64-bit float, by its exponent field."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_values(x, fmt, rule):
    """What the cache holds for x [tokens, heads, dim]: the nearest grid value, ties to the even code."""
    grid = _exact_grid(fmt)
    top = grid[-1]
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    a = b.abs().max(-1, keepdim=True).values
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0)))
    e = torch.where(_exact_pow2(e) > a, e - 1, torch.where(_exact_pow2(e + 1) <= a, e + 1, e))
    X = e - torch.floor(torch.log2(top))
    if rule == "plus1":
        X = X + 1
    if rule == "ceil":
        X = torch.where(a > top * _exact_pow2(X), X + 1, X)
    X = torch.where(a > 0, X.clamp(-127, 127), -127.0)
    unit = _exact_pow2(X)
    y = (b.abs() / unit).clamp(max=top)
    hi = torch.searchsorted(grid, y.contiguous()).clamp(max=len(grid) - 1)   # grid[hi - 1] < y <= grid[hi]
    lo = (hi - 1).clamp(min=0)
    below, above = y - grid[lo], grid[hi] - y
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    val = torch.where(up, grid[hi], grid[lo]) * unit
    return torch.copysign(val, b).reshape(x.shape)


def exact(case, seed):
    s = _inputs(case, seed)
    rule = case.get("rule", "ceil")
    if case["op"] != "attend":
        return _exact_values(s["k"], case["fmt"], rule), _exact_values(s["v"], case["fmt"], rule)
    q, group, heads, dim = case["q"], case["group"], case["heads"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, n in enumerate(s["lens"]):
        mine = slice(at, at + n)
        at += n
        pos = torch.arange(n, device="cuda")[None, :]
        end = torch.full((q, 1), n, device="cuda")
        if case["causal"]:
            end = end - q + 1 + torch.arange(q, device="cuda")[:, None]
        hidden = pos >= end
        if case["window"]:
            hidden = hidden | (pos < end - case["window"])
        for h in range(heads):
            k = _exact_values(s["k"][mine, h], case["fmt"], rule)
            v = _exact_values(s["v"][mine, h], case["fmt"], rule)
            for j in range(group):
                col = h * group + j
                x = s["q"][b * q:(b + 1) * q, col].double()
                score = (x @ k.T) / math.sqrt(dim)
                score[hidden] = -math.inf
                some = ~hidden.all(1)
                if bool(some.any()):
                    rows = torch.arange(b * q, (b + 1) * q, device="cuda")[some]
                    out[rows, col] = torch.softmax(score[some], 1) @ v
                    lse[rows, col] = torch.logsumexp(score[some], 1)
    return out, lse
