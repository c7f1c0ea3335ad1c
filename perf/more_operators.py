"""Matrices of MX blocks as they are measured: casting a matrix to 4 or 8 bits with blocks
along its rows, its columns or both, products of such matrices, linear layers over
unquantised rows, and activations that keep their inputs in 8 bits for the backward pass.

An MX matrix [rows, cols] has blocks of 32 consecutive elements of a row (the last one of a
row may be shorter) that share a power of two 2^X; each element is a code of E2M1 (4 bits:
0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), E4M3 (largest value 448) or E5M2 (57344).  X follows
from the block's largest magnitude a = m 2^e by a rule: "ocp" X = e - emax, "plus1" one more,
"ceil" the smallest X with a 2^-X <= max; elements round to nearest even and saturate.

With `own` false, `run` computes everything with elementary torch operations in fp32; with
`own` true it makes the library's calls.
"""

import math

import torch

own = False

FORMATS = {  # largest value, exponent of it, mantissa bits, smallest normal exponent
    "e2m1": (6.0, 2, 1, 0),
    "e4m3": (448.0, 8, 3, -6),
    "e5m2": (57344.0, 15, 2, -14),
}
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # a decoding step's activations of 32 sequences, ahead of several products with the same input
        dict(name="write_step", op="write", fmt="e2m1", dtype="bf16", rule="ceil", rows=32, cols=4096, sides="rows",
             sliced=False),
        # a training step's activations: rows for the forward product, columns for the weights' gradient
        dict(name="write_both", op="write", fmt="e4m3", dtype="bf16", rule="ocp", rows=8192, cols=4096, sides="both",
             sliced=False),
        # an fp32 gradient of odd size, a slice of a wider tensor, for both products of the backward pass
        dict(name="write_odd", op="write", fmt="e5m2", dtype="fp32", rule="plus1", rows=3001, cols=1357, sides="both",
             sliced=True),
        # one token through a square projection with a bias: 4-bit weights, 8-bit activations
        dict(name="linear_token", op="linear", x_fmt="e4m3", w_fmt="e2m1", dtype="bf16", m=1, n=4096, k=4096, bias=True),
        # a decoding step of 24 sequences through a wide projection, 4 bits on both sides
        dict(name="linear_batch", op="linear", x_fmt="e2m1", w_fmt="e2m1", dtype="bf16", m=24, n=11008, k=4096,
             bias=False),
        # a prompt of 4096 tokens through the same projection
        dict(name="linear_prompt", op="linear", x_fmt="e2m1", w_fmt="e2m1", dtype="bf16", m=4096, n=11008, k=4096,
             bias=False),
        # a middle-sized product of odd sizes, 8 by 4 bits, kept in fp32
        dict(name="matmul_odd", op="matmul", x_fmt="e4m3", w_fmt="e2m1", dtype="fp32", m=777, n=1000, k=1357, bias=True),
        # the weights' gradient over a step's 16384 tokens: gradients in E5M2, activations in E4M3
        dict(name="matmul_wgrad", op="matmul", x_fmt="e5m2", w_fmt="e4m3", dtype="bf16", m=4096, n=4096, k=16384,
             bias=False),
        # the gated activation of a step's tokens, its inputs kept in 8 bits
        dict(name="act_forward", op="act_forward", act="silu", gated=True, fmt="e4m3", dtype="bf16", rule="ceil",
             rows=8192, cols=11008, sliced=True),
        # a plain activation of odd size, in fp32
        dict(name="act_forward_odd", op="act_forward", act="gelu", gated=False, fmt="e4m3", dtype="fp32", rule="plus1",
             rows=1001, cols=1365, sliced=False),
        # its gradient from what was kept, with the output formed again for the next layer's weight gradient
        dict(name="act_backward", op="act_backward", act="silu", gated=True, fmt="e4m3", dtype="bf16", rule="ceil",
             rows=8192, cols=11008, sliced=True, again=True),
        # a short sequence's gradient: latency
        dict(name="act_backward_short", op="act_backward", act="gelu_tanh", gated=False, fmt="e5m2", dtype="bf16",
             rule="ocp", rows=100, cols=4096, sliced=False, again=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes spread over the listed ones' ranges, odd ones among them."""
    op = rng.choice(["write", "linear", "linear", "matmul", "matmul", "act_forward", "act_backward"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    rule = rng.choice(["ocp", "plus1", "ceil"])
    size = 2 if dtype == "bf16" else 4
    if op == "write":
        cols = _log(rng, 33, 11008)
        rows = _log(rng, 1, 8192 * 4096 * 2 // (size * cols))
        return dict(op=op, fmt=rng.choice(["e2m1", "e2m1", "e4m3", "e5m2"]), dtype=dtype, rule=rule,
                    rows=min(rows, 60000), cols=cols, sides=rng.choice(["rows", "cols", "both"]),
                    sliced=rng.random() < 0.5)
    if op in ("linear", "matmul"):
        n, k = _log(rng, 40, 11008), _log(rng, 70, 16384 if op == "matmul" else 11008)
        kind = rng.choice(["token", "few", "many"]) if op == "linear" else "many"
        m = {"token": 1, "few": rng.randint(2, 200)}.get(kind) or _log(rng, 100, 8192)
        m = min(m, max(1, 4096 * 4096 * 16384 // (n * k)))
        return dict(op=op, x_fmt=rng.choice(["e2m1", "e4m3", "e5m2"]), w_fmt=rng.choice(["e2m1", "e2m1", "e4m3"]),
                    dtype=dtype, m=m, n=n, k=k, bias=rng.random() < 0.4)
    cols = _log(rng, 40, 11008)
    rows = min(_log(rng, 1, 8192 * 11008 * 2 // (size * cols)), 60000)
    c = dict(op=op, act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu2"]), gated=rng.random() < 0.6,
             fmt=rng.choice(["e4m3", "e4m3", "e5m2", "e2m1"]), dtype=dtype, rule=rule, rows=rows, cols=cols,
             sliced=rng.random() < 0.5)
    if op == "act_backward":
        c["again"] = rng.random() < 0.5
    return c


# ---- inputs -------------------------------------------------------------------

def _inputs(case, seed):
    """Everything that a pass reads, before any of it is cast or laid out."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def activations(rows, cols, sliced=False, spread=0.8):
        # channels of unequal strength, tokens too, as behind a norm
        x = randn(rows, cols) * torch.exp(spread * randn(cols)) * torch.exp(0.3 * randn(rows, 1))
        if not sliced:
            return x.to(dt)
        wide = torch.zeros(rows, cols + 3, dtype=dt, device="cuda")   # a slice of a wider tensor: an odd row stride
        wide[:, 3:] = x
        return wide[:, 3:]

    s = {"case": case}
    op = case["op"]
    if op == "write":
        s["x"] = activations(case["rows"], case["cols"], case["sliced"])
    elif op in ("linear", "matmul"):
        s["x"] = activations(case["m"], case["k"])
        s["w"] = (randn(case["n"], case["k"]) * torch.exp(0.3 * randn(case["n"], 1)) / math.sqrt(case["k"])).to(dt)
        s["bias"] = (0.2 * randn(case["n"])).to(dt) if case["bias"] else None
    else:
        rows, cols = case["rows"], case["cols"]
        if case["gated"] and case["sliced"]:              # both halves of one projection's output
            both = torch.cat([activations(rows, cols, spread=0.4), activations(rows, cols, spread=0.4)], 1)
            s["gate"], s["up"] = both[:, :cols], both[:, cols:]
        else:
            s["gate"] = activations(rows, cols, spread=0.4)
            s["up"] = activations(rows, cols, spread=0.4) if case["gated"] else None
        if op == "act_backward":
            s["dy"] = (randn(rows, cols) * torch.exp(0.5 * randn(rows, 1))).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    if own:
        import scaled_fp8_casting_amd as nc

        def written(x, fmt, rule):
            m = nc.new_mx_matrix(x.shape[0], x.shape[1], fmt)
            nc.nc_mx_write(x, m, rule=rule)
            return m
    else:
        written = _plain_matrix

    def like(x):
        return torch.empty(x.shape, dtype=dt, device="cuda")

    if op in ("linear", "matmul"):                        # weights are laid out once, a product's operands are there
        s["w"] = written(s["w"], case["w_fmt"], "ceil")
        if op == "matmul":
            s["x"] = written(s["x"], case["x_fmt"], "ceil")
        if own:
            s["out"] = torch.empty(case["m"], case["n"], dtype=dt, device="cuda")
            s["ws"] = nc.new_mx_workspace(case["m"], s["w"], case["x_fmt"] if op == "linear" else None)
    elif op == "act_backward":                            # what the forward pass kept
        s["gate"] = written(s["gate"], case["fmt"], case["rule"])
        if case["gated"]:
            s["up"] = written(s["up"], case["fmt"], case["rule"])
        if own:
            s["dgate"], s["dup"] = like(s["dy"]), like(s["dy"]) if case["gated"] else None
            s["y"] = like(s["dy"]) if case["again"] else None
    elif own:
        rows, cols = case["rows"], case["cols"]
        if op == "write":
            s["m"] = nc.new_mx_matrix(rows, cols, case["fmt"]) if case["sides"] != "cols" else None
            s["t"] = nc.new_mx_matrix(cols, rows, case["fmt"]) if case["sides"] != "rows" else None
            s["m_out"] = like(s["x"]) if s["m"] is not None else None
            s["t_out"] = torch.empty(cols, rows, dtype=dt, device="cuda") if s["t"] is not None else None
        else:
            s["y"] = like(s["gate"])
            s["gate_q"] = nc.new_mx_matrix(rows, cols, case["fmt"])
            s["up_q"] = nc.new_mx_matrix(rows, cols, case["fmt"]) if case["gated"] else None
            s["gate_out"], s["up_out"] = like(s["gate"]), like(s["gate"]) if case["gated"] else None
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _given(*outputs):
    return tuple(x for x in outputs if x is not None)


def _own(s):
    import scaled_fp8_casting_amd as nc
    case = s["case"]
    op = case["op"]
    if op == "write":
        nc.nc_mx_write(s["x"], s["m"], s["t"], rule=case["rule"])
        if s["m"] is not None:
            nc.nc_mx_read(s["m"], s["m_out"])
        if s["t"] is not None:
            nc.nc_mx_read(s["t"], s["t_out"])
        return _given(s["m_out"], s["t_out"])
    if op == "linear":
        nc.nc_mx_linear(s["x"], s["w"], s["out"], fmt=case["x_fmt"], rule="ceil", bias=s["bias"], ws=s["ws"])
        return s["out"]
    if op == "matmul":
        nc.nc_mx_matmul(s["x"], s["w"], s["out"], bias=s["bias"], ws=s["ws"])
        return s["out"]
    if op == "act_forward":
        nc.nc_act_forward(s["gate"], s["up"], s["y"], s["gate_q"], s["up_q"], act=case["act"], rule=case["rule"])
        nc.nc_mx_read(s["gate_q"], s["gate_out"])
        if case["gated"]:
            nc.nc_mx_read(s["up_q"], s["up_out"])
        return _given(s["y"], s["gate_out"], s["up_out"])
    nc.nc_act_backward(s["dy"], s["gate"], s["up"], s["dgate"], s["dup"], act=case["act"], y=s["y"])
    return _given(s["dgate"], s["dup"], s["y"])


# ---- the plain form -------------------------------------------------------------

def _pow2(n):
    """2^n as fp32, exactly (n whole, clamped to the normal range: exp2 may be an ulp off)."""
    return ((n.clamp(-126, 127).to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_matrix(x, fmt, rule):
    """x [rows, cols] -> codes, one a byte, scale bytes X + 127, and what decodes them."""
    top, emax, mb, emin = FORMATS[fmt]
    cols = x.shape[1]
    b = torch.nn.functional.pad(x.float(), (0, -cols % 32)).unflatten(-1, (-1, 32))
    a = b.abs().amax(-1)
    X = torch.frexp(a).exponent - 1 - emax
    if rule == "plus1":
        X = X + 1
    elif rule == "ceil":
        X = X + (a * _pow2(-X) > top)
    X = torch.where(a == 0, -127, X.clamp(-127, 127))
    y = b.abs() * _pow2(-X)[..., None]
    e = torch.where(y > 0, torch.frexp(y).exponent - 1, emin).clamp(min=emin)
    index = (e - emin) * (1 << mb) + torch.round(y * _pow2(mb - e)).to(torch.int32)
    most = (int(math.log2(top)) - emin + 1) * (1 << mb) + (1 << mb) - 1 - (fmt == "e4m3")   # the largest value's code
    codes = index.clamp(max=most) + (torch.signbit(b).to(torch.int32) << (3 if fmt == "e2m1" else 7))
    return codes.to(torch.uint8), (X + 127).to(torch.uint8), _decode_table(fmt), cols


def _decode_table(fmt):
    """The value of every code as fp32, on the GPU."""
    _, _, mb, emin = FORMATS[fmt]
    i = torch.arange(8 if fmt == "e2m1" else 128, device="cuda")
    e, m = i >> mb, i & ((1 << mb) - 1)
    mag = torch.where(e == 0, m.float(), (m + (1 << mb)).float() * _pow2((e - 1).clamp(min=0))) * 2.0 ** (emin - mb)
    return torch.cat([mag, -mag])


def _plain_values(matrix):
    codes, scales, table, cols = matrix
    return (table[codes.int()] * _pow2(scales.int() - 127)[..., None]).flatten(-2)[:, :cols]


def _plain_act(z, act):
    """f(z) and f'(z), fp32."""
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        return z * sig, sig * (1.0 + z * (1.0 - sig))
    if act == "gelu":
        phi = 0.5 * torch.erfc(z * -math.sqrt(0.5))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        sig = 1.0 / (1.0 + torch.exp(-2.0 * c * (z + 0.044715 * z * z * z)))    # (1 + tanh u) / 2
        return z * sig, sig + 2.0 * z * sig * (1.0 - sig) * c * (1.0 + 3.0 * 0.044715 * z * z)
    r = z.clamp(min=0)
    return r * r, 2.0 * r


def _plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "write":
        x, fmt, rule = s["x"], case["fmt"], case["rule"]
        m = _plain_values(_plain_matrix(x, fmt, rule)).to(dt) if case["sides"] != "cols" else None
        t = _plain_values(_plain_matrix(x.T, fmt, rule)).to(dt) if case["sides"] != "rows" else None
        return _given(m, t)
    if op in ("linear", "matmul"):
        x = _plain_matrix(s["x"], case["x_fmt"], "ceil") if op == "linear" else s["x"]
        out = torch.matmul(_plain_values(x), _plain_values(s["w"]).T)
        if s["bias"] is not None:
            out = out + s["bias"].float()
        return out.to(dt)
    if op == "act_forward":
        f, _ = _plain_act(s["gate"].float(), case["act"])
        y = f * s["up"].float() if case["gated"] else f
        kept = [_plain_values(_plain_matrix(x, case["fmt"], case["rule"])).to(dt) for x in _given(s["gate"], s["up"])]
        return (y.to(dt), *kept)
    dy = s["dy"].float()
    f, df = _plain_act(_plain_values(s["gate"]), case["act"])
    up = _plain_values(s["up"]) if case["gated"] else None
    dgate = dy * up * df if case["gated"] else dy * df
    dup = dy * f if case["gated"] else None
    y = (f * up if case["gated"] else f) if case["again"] else None
    return tuple(x.to(dt) for x in _given(dgate, dup, y))


# ---- what a pass cannot do without -------------------------------------------------

def _kept(rows, cols, fmt):
    """Bytes of an MX matrix."""
    return rows * (cols * (4 if fmt == "e2m1" else 8) // 8 + -(-cols // 32))


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("linear", "matmul"):
        m, n, k = case["m"], case["n"], case["k"]
        moved = _kept(n, k, case["w_fmt"]) + m * n * size + (n * size if case["bias"] else 0)
        moved += m * k * size if op == "linear" else _kept(m, k, case["x_fmt"])
        return {"bytes": moved, "flops": 2 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    plane, kept = rows * cols * size, _kept(rows, cols, case["fmt"])
    if op == "write":                                     # written, read back
        sides = (case["sides"] != "cols") * kept + (case["sides"] != "rows") * _kept(cols, rows, case["fmt"])
        planes = 3 if case["sides"] == "both" else 2
        return {"bytes": planes * plane + 2 * sides, "flops": 0}
    n = 2 if case["gated"] else 1
    if op == "act_forward":                               # inputs read, output and codes written, these read back
        return {"bytes": (2 * n + 1) * plane + 2 * n * kept, "flops": 0}
    return {"bytes": (n + 1 + (1 if case["again"] else 0)) * plane + n * kept, "flops": 0}


# ---- the definition in 64 bits -----------------------------------------------------

def _exact_grid(fmt):
    """The non-negative finite values, ascending; a value's place is its code."""
    if fmt == "e2m1":
        values = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    elif fmt == "e4m3":
        values = [j / 8 * 2.0 ** -6 for j in range(8)]
        values += [(8 + j) / 8 * 2.0 ** e for e in range(-6, 9) for j in range(8)][:-1]
    else:
        values = [j / 4 * 2.0 ** -14 for j in range(4)]
        values += [(4 + j) / 4 * 2.0 ** e for e in range(-14, 16) for j in range(4)]
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _exact_pow2(n):
    """2^n as a 64-bit float, by its exponent field."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_values(x, fmt, rule):
    """What an MX matrix holds for x [rows, cols]: the nearest grid value, ties to the even code."""
    grid = _exact_grid(fmt)
    top = grid[-1]
    rows, cols = x.shape
    full = torch.zeros(rows, (cols + 31) // 32 * 32, dtype=torch.float64, device="cuda")
    full[:, :cols] = x
    b = full.reshape(rows, -1, 32)
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
    return torch.copysign(val, b).reshape(rows, -1)[:, :cols]


def _exact_act(z, act):
    """f(z), and f'(z) as torch differentiates f, in 64 bits."""
    with torch.enable_grad():
        z = z.detach().requires_grad_()
        if act == "silu":
            f = z * torch.sigmoid(z)
        elif act == "gelu":
            f = z * torch.special.ndtr(z)
        elif act == "gelu_tanh":
            f = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        else:
            f = torch.relu(z) ** 2
        df, = torch.autograd.grad(f.sum(), z)
    return f.detach(), df


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "write":
        x, fmt, rule = s["x"], case["fmt"], case["rule"]
        m = _exact_values(x, fmt, rule) if case["sides"] != "cols" else None
        t = _exact_values(x.T, fmt, rule) if case["sides"] != "rows" else None
        return _given(m, t)
    if op in ("linear", "matmul"):
        out = _exact_values(s["x"], case["x_fmt"], "ceil") @ _exact_values(s["w"], case["w_fmt"], "ceil").T
        return out if s["bias"] is None else out + s["bias"].double()
    if op == "act_forward":
        f, _ = _exact_act(s["gate"].double(), case["act"])
        y = f * s["up"].double() if case["gated"] else f
        return (y, *(_exact_values(x, case["fmt"], case["rule"]) for x in _given(s["gate"], s["up"])))
    dy = s["dy"].double()
    f, df = _exact_act(_exact_values(s["gate"], case["fmt"], case["rule"]), case["act"])
    up = _exact_values(s["up"], case["fmt"], case["rule"]) if case["gated"] else torch.ones_like(dy)
    return _given(dy * up * df, dy * f if case["gated"] else None, f * up if case["again"] else None)
