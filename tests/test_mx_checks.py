"""Refusals of the MX matrices, their products and the activations over them, at the
C-ABI and in the binding, sizes, and pins of the oracle.  Nothing here launches a
kernel: every call fails its checks (or is empty) first, so these run without a GPU."""

import ctypes

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc
from oracle import E4M3, E5M2, bulk, kv, mx
from scaled_fp8_casting_amd import _lib
from scaled_fp8_casting_amd._lib import NcMxMatrix, NcMxOut, NcPlane

A = 0x10000          # an aligned address that no call reaches
W = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def matrix(**kw):
    f = dict(data=A, rows=40, cols=100, fmt=_lib.NC_E2M1, reserved=0)
    f.update(kw)
    return ctypes.byref(NcMxMatrix(**f))


def plane(p=A, stride=1000):
    return ctypes.byref(NcPlane(p, stride))


def out(**kw):
    f = dict(data=A, stride=1000, dtype=1, accumulate=0, bias=None)
    f.update(kw)
    return ctypes.byref(NcMxOut(**f))


BAD = [
    (dict(fmt=3), _lib.NC_E_UNSUPPORTED), (dict(fmt=-1), _lib.NC_E_UNSUPPORTED),
    (dict(rows=-1), _lib.NC_E_ARG), (dict(cols=-1), _lib.NC_E_ARG), (dict(rows=1 << 31), _lib.NC_E_ARG),
    (dict(cols=1 << 31), _lib.NC_E_ARG), (dict(rows=1 << 30, cols=1 << 20), _lib.NC_E_ARG),
    (dict(data=None), _lib.NC_E_ARG), (dict(data=A + 8), _lib.NC_E_ALIGN),
]


@pytest.mark.parametrize("kw,status", BAD)
def test_matrices(lib, kw, status):
    bad = matrix(**kw)
    rows, cols = kw.get("rows", 40), kw.get("cols", 100)
    good = matrix(rows=40, cols=100)
    assert lib.nc_mx_write(bad, None, plane(), 1, 2, None) == status
    assert lib.nc_mx_write(None, bad, plane(), 1, 2, None) == status
    assert lib.nc_mx_read(bad, plane(), 1, None) == status
    assert lib.nc_mx_matmul(bad, good, out(), A, W, None) == status
    assert lib.nc_mx_matmul(good, bad, out(), A, W, None) == status
    assert lib.nc_mx_linear(plane(), 4, 1, 0, 2, bad, out(), A, W, None) == status
    assert lib.nc_act_backward(0, plane(), 1, bad, None, plane(), None, None, None) == status
    assert lib.nc_act_backward(0, plane(), 1, good, bad, plane(), plane(), None, None) == status
    if "data" not in kw:
        assert lib.nc_mx_bytes(rows, cols, kw.get("fmt", _lib.NC_E2M1)) == 0
        assert lib.nc_mx_workspace_bytes(bad, 100, -1) == 0


def test_no_matrix(lib):
    good = matrix()
    assert lib.nc_mx_write(None, None, plane(), 1, 2, None) == _lib.NC_E_ARG
    assert lib.nc_mx_read(None, plane(), 1, None) == _lib.NC_E_ARG
    assert lib.nc_mx_matmul(None, good, out(), A, W, None) == _lib.NC_E_ARG
    assert lib.nc_mx_matmul(good, None, out(), A, W, None) == _lib.NC_E_ARG
    assert lib.nc_mx_linear(plane(), 4, 1, 0, 2, None, out(), A, W, None) == _lib.NC_E_ARG
    assert lib.nc_act_backward(0, plane(), 1, None, None, plane(), None, None, None) == _lib.NC_E_ARG
    assert lib.nc_mx_workspace_bytes(None, 5, -1) == 0


def test_write_and_read(lib):
    m, t = matrix(), matrix(rows=100, cols=40)
    for dt in (2, -1):
        assert lib.nc_mx_write(m, t, plane(), dt, 2, None) == _lib.NC_E_UNSUPPORTED
        assert lib.nc_mx_read(m, plane(), dt, None) == _lib.NC_E_UNSUPPORTED
    assert lib.nc_mx_write(m, t, plane(), 1, 3, None) == _lib.NC_E_UNSUPPORTED
    for other in (matrix(rows=100, cols=41), matrix(rows=99, cols=40), matrix(rows=100, cols=40, fmt=0)):
        assert lib.nc_mx_write(m, other, plane(), 1, 2, None) == _lib.NC_E_SHAPE
    assert lib.nc_mx_write(m, t, None, 1, 2, None) == _lib.NC_E_ARG
    assert lib.nc_mx_write(m, t, plane(None), 1, 2, None) == _lib.NC_E_ARG
    assert lib.nc_mx_write(m, t, plane(A, -1), 1, 2, None) == _lib.NC_E_ARG
    assert lib.nc_mx_write(m, t, plane(A + 1), 1, 2, None) == _lib.NC_E_ALIGN
    assert lib.nc_mx_write(m, t, plane(A + 2), 0, 2, None) == _lib.NC_E_ALIGN
    assert lib.nc_mx_read(m, plane(A, 99), 1, None) == _lib.NC_E_ARG          # rows would overlap
    assert lib.nc_mx_read(m, None, 1, None) == _lib.NC_E_ARG
    assert lib.nc_mx_read(m, plane(A + 1), 1, None) == _lib.NC_E_ALIGN
    empty = matrix(rows=0, data=None)
    assert lib.nc_mx_write(empty, None, None, 1, 2, None) == lib.nc_mx_read(empty, None, 1, None) == _lib.NC_OK
    # the transposed write's workgroups would not fit a launch: many rows of few columns
    assert lib.nc_mx_write(None, matrix(rows=3, cols=(1 << 31) - 1), plane(), 1, 2, None) == _lib.NC_E_ARG


def test_products(lib):
    a, b = matrix(), matrix(rows=70)
    assert lib.nc_mx_matmul(a, matrix(cols=99), out(), A, W, None) == _lib.NC_E_SHAPE
    for bad, status in ((dict(data=None), _lib.NC_E_ARG), (dict(stride=69), _lib.NC_E_ARG), (dict(dtype=2), _lib.NC_E_UNSUPPORTED),
                        (dict(data=A + 1), _lib.NC_E_ALIGN), (dict(bias=A + 1), _lib.NC_E_ALIGN),
                        (dict(dtype=0, data=A + 2), _lib.NC_E_ALIGN), (dict(dtype=0, bias=A + 2), _lib.NC_E_ALIGN)):
        assert lib.nc_mx_matmul(a, b, out(**bad), A, W, None) == status
        assert lib.nc_mx_linear(plane(), 4, 1, 0, 2, b, out(**bad), A, W, None) == status
    assert lib.nc_mx_matmul(a, b, None, A, W, None) == _lib.NC_E_ARG
    for x_dtype, fmt, rule in ((2, 0, 2), (1, 3, 2), (1, 0, 3), (1, -1, 2)):
        assert lib.nc_mx_linear(plane(), 4, x_dtype, fmt, rule, b, out(), A, W, None) == _lib.NC_E_UNSUPPORTED
    assert lib.nc_mx_linear(plane(), -1, 1, 0, 2, b, out(), A, W, None) == _lib.NC_E_ARG
    assert lib.nc_mx_linear(None, 4, 1, 0, 2, b, out(), A, W, None) == _lib.NC_E_ARG
    assert lib.nc_mx_linear(plane(A, -5), 4, 1, 0, 2, b, out(), A, W, None) == _lib.NC_E_ARG
    # a workspace that is missing, not aligned, too small
    big = matrix(rows=64, cols=20000)
    for args in ((None, W), (A + 8, W)):
        assert lib.nc_mx_matmul(a, b, out(), *args, None) == _lib.NC_E_WORKSPACE
        assert lib.nc_mx_linear(plane(), 40, 1, 0, 2, b, out(), *args, None) == _lib.NC_E_WORKSPACE
    need = lib.nc_mx_workspace_bytes(big, 40, 0)
    assert need >= nc.mx_bytes(40, 20000, "e4m3")
    assert lib.nc_mx_linear(plane(A, 20000), 40, 1, 0, 2, big, out(), None, 0, None) == _lib.NC_E_WORKSPACE
    assert lib.nc_mx_linear(plane(A, 20000), 40, 1, 0, 2, big, out(), A, nc.mx_bytes(40, 20000, "e4m3") - 1, None) == _lib.NC_E_WORKSPACE
    # nothing to write
    assert lib.nc_mx_matmul(matrix(rows=0, data=None), b, out(data=None), None, 0, None) == _lib.NC_OK
    assert lib.nc_mx_matmul(a, matrix(rows=0, data=None), out(data=None), None, 0, None) == _lib.NC_OK
    assert lib.nc_mx_linear(None, 0, 1, 0, 2, b, out(data=None), None, 0, None) == _lib.NC_OK
    # more results than any launch has workgroups for
    wide = matrix(rows=1 << 26, cols=1)
    assert lib.nc_mx_matmul(wide, wide, out(stride=1 << 26), None, 0, None) == _lib.NC_E_ARG
    none = matrix(rows=1 << 26, cols=0, data=None)
    assert lib.nc_mx_matmul(none, none, out(stride=1 << 26), None, 0, None) == _lib.NC_E_ARG


def test_workspace_serves_fewer_rows(lib):
    """One for more rows is enough for fewer, for a matrix product's splits and a linear layer's rows alike."""
    for n, k in ((256, 16384), (4096, 4096), (1000, 100000), (70, 300)):
        for fmt in (-1, 0, 2):
            w = matrix(rows=n, cols=k)
            sizes = [lib.nc_mx_workspace_bytes(w, m, fmt) for m in range(1, 3000, 37)]
            assert sizes == sorted(sizes)


def test_activations(lib):
    g, u = matrix(fmt=0), matrix(fmt=0)
    def fwd(act=0, rows=40, cols=100, gate=plane(), up=plane(), y=plane(), dt=1, gq=g, uq=u, rule=2):
        return lib.nc_act_forward(act, rows, cols, gate, up, y, dt, gq, uq, rule, None)
    for kw in (dict(act=4), dict(act=-1), dict(dt=2), dict(rule=3)):
        assert fwd(**kw) == _lib.NC_E_UNSUPPORTED
    for kw in (dict(gate=None), dict(y=None), dict(gate=plane(None)), dict(up=plane(None)), dict(y=plane(A, 99)), dict(rows=-1),
               dict(uq=None), dict(up=None), dict(gq=None), dict(gate=plane(A, -1)), dict(cols=1 << 31)):
        assert fwd(**kw) == _lib.NC_E_ARG
    for kw in (dict(rows=41), dict(cols=99), dict(uq=matrix(fmt=1)), dict(uq=matrix(rows=41, fmt=0)), dict(gq=matrix(cols=99, fmt=0))):
        assert fwd(**kw) == _lib.NC_E_SHAPE
    for kw in (dict(gate=plane(A + 1)), dict(up=plane(A + 1)), dict(y=plane(A + 1)), dict(gq=matrix(data=A + 8, fmt=0))):
        assert fwd(**kw) == _lib.NC_E_ALIGN
    assert fwd(rows=0, gate=None, y=None, up=None, gq=None, uq=None) == _lib.NC_OK

    def bwd(act=0, dy=plane(), dt=1, gq=g, uq=u, dg=plane(), du=plane(), y=None):
        return lib.nc_act_backward(act, dy, dt, gq, uq, dg, du, y, None)
    for kw in (dict(act=4), dict(dt=2)):
        assert bwd(**kw) == _lib.NC_E_UNSUPPORTED
    for kw in (dict(dy=None), dict(dg=None), dict(du=None), dict(uq=None), dict(dg=plane(A, 99)), dict(du=plane(A, 99)), dict(y=plane(A, 99)),
               dict(dy=plane(None)), dict(y=plane(None))):
        assert bwd(**kw) == _lib.NC_E_ARG
    for kw in (dict(uq=matrix(fmt=1)), dict(uq=matrix(rows=41, fmt=0)), dict(uq=matrix(cols=99, fmt=0))):
        assert bwd(**kw) == _lib.NC_E_SHAPE
    for kw in (dict(dy=plane(A + 1)), dict(dg=plane(A + 1)), dict(du=plane(A + 1)), dict(y=plane(A + 1))):
        assert bwd(**kw) == _lib.NC_E_ALIGN


def test_struct_sizes():
    assert ctypes.sizeof(NcMxMatrix) == 32 and ctypes.sizeof(NcPlane) == 16 and ctypes.sizeof(NcMxOut) == 32


def test_bytes():
    """Strips of 32 rows by chunks of 256 columns, and 256 bytes of scales for each."""
    for rows, cols in ((1, 1), (32, 256), (33, 257), (4096, 11008), (7, 1000)):
        tiles = -(-rows // 32) * -(-cols // 256)
        assert nc.mx_bytes(rows, cols, "e2m1") == tiles * (4096 + 256)
        assert nc.mx_bytes(rows, cols, "e4m3") == nc.mx_bytes(rows, cols, "e5m2") == tiles * (8192 + 256)
    assert nc.mx_bytes(0, 50, "e2m1") == nc.mx_bytes(50, 0, "e2m1") == 0
    for args in ((1, 1, "e3m2"), (-1, 5, "e2m1"), (5, -1, "e2m1"), (1 << 31, 1, "e2m1"), (1, 1 << 31, "e2m1"), (1 << 40, 1, "e2m1"),
                 (1 << 30, 1 << 20, "e2m1")):
        with pytest.raises(ValueError):
            nc.mx_bytes(*args)


# ---- the binding: tensors that only say that they are on a GPU, a library that notes its calls ----

class OnGpu(torch.Tensor):
    """Host memory that gives a GPU as its device."""
    device = property(lambda self: torch.device("cuda", 0))


def on_gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Library:
    def __init__(self):
        self.calls, self.real = [], _lib.load()

    def nc_mx_bytes(self, *args):
        return self.real.nc_mx_bytes(*args)

    def nc_mx_workspace_bytes(self, *args):
        return self.real.nc_mx_workspace_bytes(*args)

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(_lib, "load", lambda: lib)
    monkeypatch.setattr(nc, "_kv_stream", lambda stream, dev: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return lib


def new(rows, cols, fmt="e4m3"):
    return nc.MxMatrix(on_gpu(max(nc.mx_bytes(rows, cols, fmt), 16), dtype=torch.uint8), rows, cols, fmt)


def test_binding_passes_on(library):
    m, t, w = new(8, 100), new(100, 8), new(70, 100, "e2m1")
    x = on_gpu(8, 103)[:, 3:]
    nc.nc_mx_write(x, m, t, rule="ocp")
    name, (md, td, p, code, rule, _) = library.calls[-1]
    assert name == "nc_mx_write" and (md.rows, md.cols, md.fmt) == (8, 100, _lib.NC_E4M3) and td.rows == 100
    assert (p.data, p.stride, code, rule) == (x.data_ptr(), 103, _lib.NC_BF16, _lib.NC_MX_OCP)
    ws = on_gpu(nc.mx_workspace_bytes(8, w, "e4m3"), dtype=torch.uint8)
    y, bias = on_gpu(8, 70, dtype=torch.float32), on_gpu(70, dtype=torch.float32)
    nc.nc_mx_linear(x, w, y, bias=bias, accumulate=True, ws=ws)
    _, (p, rows, xd, xf, rule, wd, o, at, n, _) = library.calls[-1]
    assert (p.stride, rows, xd, xf, rule, wd.rows) == (103, 8, _lib.NC_BF16, _lib.NC_E4M3, _lib.NC_MX_CEIL, 70)
    assert (o.data, o.stride, o.dtype, o.accumulate, o.bias) == (y.data_ptr(), 70, _lib.NC_F32, 1, bias.data_ptr())
    assert (at, n) == (ws.data_ptr(), ws.numel())
    nc.nc_mx_matmul(m, w, y, ws=ws)
    _, (ad, bd, o, *_rest) = library.calls[-1]
    assert (ad.data, bd.data, o.accumulate, o.bias) == (m.data.data_ptr(), w.data.data_ptr(), 0, None)
    row = on_gpu(1, 100).expand(8, 100)
    nc.nc_mx_write(row, m)
    assert library.calls[-1][1][2].stride == 0
    # another buffer in a matrix's place, and one resized in place
    m.data = on_gpu(nc.mx_bytes(8, 100, "e4m3") + 64, dtype=torch.uint8)
    nc.nc_mx_write(x, m)
    assert library.calls[-1][1][0].data == m.data.data_ptr()
    m.data.resize_(8)
    with pytest.raises(ValueError):
        nc.nc_mx_write(x, m)


def test_binding_refuses(library):
    m, t, w = new(8, 100), new(100, 8), new(70, 100, "e2m1")
    x, y = on_gpu(8, 100), on_gpu(8, 70)
    bad = [
        lambda: nc.nc_mx_write(x), lambda: nc.nc_mx_write(x, m, rule="up"), lambda: nc.nc_mx_write(on_gpu(8, 99), m),
        lambda: nc.nc_mx_write(on_gpu(800), m), lambda: nc.nc_mx_write(x, m, new(100, 9)), lambda: nc.nc_mx_write(x, m, new(100, 8, "e5m2")),
        lambda: nc.nc_mx_write(on_gpu(100, 8).T, m), lambda: nc.nc_mx_write(x.as_subclass(torch.Tensor), m),
        lambda: nc.nc_mx_read(m, on_gpu(8, 101)), lambda: nc.nc_mx_read(m, on_gpu(1, 100).expand(8, 100)),
        lambda: nc.nc_mx_read(m, on_gpu(100, 8).T), lambda: nc.nc_mx_read(m, on_gpu(1000).as_strided((8, 100), (99, 1))),
        lambda: nc.nc_mx_matmul(m, new(70, 101), y), lambda: nc.nc_mx_matmul(m, w, on_gpu(8, 71)),
        lambda: nc.nc_mx_matmul(m, w, y, bias=on_gpu(71)), lambda: nc.nc_mx_matmul(m, w, y, bias=on_gpu(70, dtype=torch.float32)),
        lambda: nc.nc_mx_matmul(m, w, y, bias=on_gpu(140)[::2]), lambda: nc.nc_mx_matmul(m, w, y, ws=on_gpu(64)),
        lambda: nc.nc_mx_matmul(m, w, y, ws=torch.zeros(64, dtype=torch.uint8)),
        lambda: nc.nc_mx_linear(x, w, y, fmt="e3m2"), lambda: nc.nc_mx_linear(x, w, y, rule=7), lambda: nc.nc_mx_linear(on_gpu(100), w, on_gpu(1, 70)),
        lambda: nc.nc_mx_linear(on_gpu(8, 99), w, y), lambda: nc.nc_mx_linear(x, w, on_gpu(9, 70)),
        lambda: nc.nc_act_forward(x, None, on_gpu(8, 100), m, t), lambda: nc.nc_act_forward(x, x, on_gpu(8, 100), m),
        lambda: nc.nc_act_forward(x, None, on_gpu(8, 100), None, m), lambda: nc.nc_act_forward(x, None, on_gpu(8, 100), new(8, 99)),
        lambda: nc.nc_act_forward(x, x, on_gpu(8, 100), m, new(8, 100, "e5m2")), lambda: nc.nc_act_forward(x, None, on_gpu(8, 100), act="tanh"),
        lambda: nc.nc_act_forward(x, None, on_gpu(8, 100, dtype=torch.float32)), lambda: nc.nc_act_forward(x, on_gpu(8, 99), on_gpu(8, 100)),
        lambda: nc.nc_act_forward(on_gpu(800), None, on_gpu(800)),
        lambda: nc.nc_act_backward(x, m, None, x, x), lambda: nc.nc_act_backward(x, m, m, x), lambda: nc.nc_act_backward(x, m, new(8, 99), x, x),
        lambda: nc.nc_act_backward(x, m, None, on_gpu(8, 99)), lambda: nc.nc_act_backward(x, m, None, x, y=on_gpu(8, 99)),
        lambda: nc.new_mx_workspace(-1, w), lambda: nc.new_mx_workspace(1 << 31, w), lambda: nc.new_mx_workspace(4, w, "e3m2"),
        lambda: nc.MxMatrix(on_gpu(64, dtype=torch.uint8), 8, 100, "e4m3"), lambda: nc.MxMatrix(on_gpu(1 << 16), 8, 100, "e4m3"),
        lambda: nc.MxMatrix(on_gpu(2, 1 << 16, dtype=torch.uint8), 8, 100, "e4m3"),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print(i)
    for call in (lambda: nc.nc_mx_write(on_gpu(8, 100, dtype=torch.float16), m), lambda: nc.nc_mx_read(m, on_gpu(8, 100, dtype=torch.float64)),
                 lambda: nc.nc_mx_matmul(m, w, on_gpu(8, 70, dtype=torch.float16)), lambda: nc.nc_mx_linear(on_gpu(8, 100, dtype=torch.float16), w, y),
                 lambda: nc.nc_act_forward(on_gpu(8, 100, dtype=torch.float16), None, x), lambda: nc.nc_act_backward(on_gpu(8, 100, dtype=torch.float16), m, None, x)):
        with pytest.raises(TypeError):
            call()
    assert not library.calls


def test_binding_refuses_host_tensors():
    m = nc.MxMatrix(torch.zeros(nc.mx_bytes(8, 100, "e4m3"), dtype=torch.uint8), 8, 100, "e4m3")
    x = torch.zeros(8, 100)
    for call in (lambda: nc.nc_mx_write(x, m), lambda: nc.nc_mx_read(m, x), lambda: nc.nc_mx_matmul(m, m, torch.zeros(8, 8)),
                 lambda: nc.nc_mx_linear(x, m, torch.zeros(8, 8)), lambda: nc.nc_act_forward(x, None, x), lambda: nc.nc_act_backward(x, m, None, x)):
        with pytest.raises(ValueError, match="no CPU path"):
            call()


# ---- pins of the oracle ----------------------------------------------------------

@pytest.mark.parametrize("rule", ["ocp", "plus1", "ceil"])
def test_oracle_against_the_casts(rule):
    """Whole blocks: what the oracles of the MX cast and of the cache hold."""
    x = np.random.default_rng(1).standard_normal((16, 96)).astype(np.float32) * np.float32(3)
    x[0, 0], x[1, 5], x[2, 40:] = 0.0, -0.0, 0.0
    for fmt, name in ((E4M3, "e4m3"), (E5M2, "e5m2")):
        codes, scales, _ = bulk.cast_mx_f64(fmt, x.astype(np.float64).reshape(-1), 96, rule)
        want = bulk.represented_f64(fmt, codes, np.repeat(127 - scales.astype(np.int64), 32))
        assert np.array_equal(mx.held(x, name, rule).reshape(-1), want)
    assert np.array_equal(mx.held(x, "e2m1", rule), kv.held(x, "e2m1", rule))


def test_oracle_short_blocks():
    """A row's last block is of what is left of it: the same as with zeros behind."""
    x = np.random.default_rng(2).standard_normal((5, 45))
    wide = np.zeros((5, 64))
    wide[:, :45] = x
    for fmt in ("e2m1", "e4m3", "e5m2"):
        assert np.array_equal(mx.held(x, fmt, "ceil"), mx.held(wide, fmt, "ceil")[:, :45])


def test_oracle_activations():
    """Against torch's own functions in binary64, and its derivatives."""
    z = torch.linspace(-12, 12, 481, dtype=torch.float64, requires_grad=True)
    for kind, f in (("silu", torch.nn.functional.silu), ("gelu", torch.nn.functional.gelu),
                    ("gelu_tanh", lambda v: torch.nn.functional.gelu(v, approximate="tanh")), ("relu2", lambda v: torch.relu(v) ** 2)):
        y = f(z)
        d, = torch.autograd.grad(y.sum(), z)
        got, df, _, _ = mx.act(z.detach().numpy(), kind)
        np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-15)
        np.testing.assert_allclose(df, d.numpy(), rtol=1e-9, atol=1e-12)


# More workgroups than a launch has, where a strip or a tile is not full: 600000001 rows
# of b are 18750001 strips, 9375001 tiles of 64 (more than 2^23), with one row of a.
def test_products_past_a_launch(lib):
    rows = 600000001
    none, one = matrix(rows=rows, cols=0, data=None), matrix(rows=1, cols=0, data=None)
    assert lib.nc_mx_matmul(one, none, out(stride=rows), None, 0, None) == _lib.NC_E_ARG
    assert lib.nc_mx_matmul(none, one, out(stride=1), None, 0, None) == _lib.NC_E_ARG
    assert lib.nc_mx_linear(None, 1, 1, 0, 2, none, out(stride=rows), A, W, None) == _lib.NC_E_ARG
