"""What the key/value cache's binding passes to the library: sizes beyond 32 bits.
The library is a stand-in and the tensors only say that they are on a GPU, so
these run without one."""

import pytest
import torch

import scaled_fp8_casting_amd as nc
from scaled_fp8_casting_amd import _lib


class OnGpu(torch.Tensor):
    """Host memory that gives a GPU as its device."""
    device = property(lambda self: torch.device("cuda", 0))


def on_gpu(t):
    return t.as_subclass(OnGpu)


class Library:
    """Notes the calls' arguments; sizes are the real library's."""

    def __init__(self):
        self.calls, self.real = [], _lib.load()

    def nc_kv_cache_bytes(self, *args):
        return self.real.nc_kv_cache_bytes(*args)

    def nc_status_string(self, status):
        return self.real.nc_status_string(status)

    def nc_kv_workspace_bytes(self, *args):
        self.calls.append(("workspace", args))
        return 0

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


def new_cache(heads=2, dim=64, pages=4):
    return nc.KvCache(on_gpu(torch.zeros((pages, nc.kv_page_bytes(16, heads, dim, "e2m1")), dtype=torch.uint8)), 16, heads,
                      dim, "e2m1")


def rows(*shape):
    return on_gpu(torch.zeros(shape, dtype=torch.bfloat16))


def i32(*x):
    return on_gpu(torch.tensor(x, dtype=torch.int32))


def attend(cache, **kw):
    args = dict(q=rows(3, 4, 64), out=rows(3, 4, 64), q_start=i32(0, 1, 3), kv_len=i32(9, 9),
                table=on_gpu(torch.zeros((2, 2), dtype=torch.int32)), max_q=2, max_kv=9)
    nc.nc_kv_attention(cache, **{**args, **kw})


LARGE = [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63, 2 ** 70]


@pytest.mark.parametrize("n", LARGE)
@pytest.mark.parametrize("name", ["max_q", "max_kv"])
def test_bounds_beyond_32_bits_are_refused(library, name, n):
    with pytest.raises(ValueError, match=name):
        attend(new_cache(), **{name: n})
    assert not library.calls


@pytest.mark.parametrize("window,passed", [(n, 2 ** 31 - 1) for n in LARGE] + [(2 ** 31 - 1, 2 ** 31 - 1), (7, 7), (0, 0)])
def test_a_window_beyond_32_bits_is_no_limit(library, window, passed):
    """No sequence has more than 2^31 - 1 tokens."""
    attend(new_cache(), window=window)
    name, args = library.calls[-1]
    assert name == "nc_kv_attention" and args[1].window == passed
    assert (args[1].max_q, args[1].max_kv, args[1].total_q, args[1].batch) == (2, 9, 3, 2)


@pytest.mark.parametrize("n", LARGE)
def test_workspace_sizes_beyond_32_bits_are_refused(library, n):
    cache, q = new_cache(), rows(3, 4, 64)
    for args in ((n, 1, 1), (1, n, 1), (1, 1, n)):
        with pytest.raises(ValueError):
            nc.kv_workspace_bytes(cache, q, *args)
        with pytest.raises(ValueError):
            nc.new_kv_workspace(cache, q, *args)
    with pytest.raises(ValueError):
        nc.kv_workspace_bytes(cache, rows(3, 1, 64).expand(3, 2 ** 32 + 2, 64), 1, 1, 1)
    assert not library.calls
    nc.kv_workspace_bytes(cache, q, 2 ** 31 - 1, 1, 2 ** 31 - 1)
    assert library.calls[-1][1][2:] == (4, 2 ** 31 - 1, 1, 2 ** 31 - 1)


@pytest.mark.parametrize("page,heads", [(2 ** 32 + 16, 1), (2 ** 31, 1), (16, 2 ** 32 + 1), (16, 2 ** 31)])
def test_page_sizes_beyond_32_bits_are_refused(page, heads):
    with pytest.raises(ValueError, match="too large"):
        nc.kv_page_bytes(page, heads, 64, "e2m1")


# -- a cache's memory ------------------------------------------------------------

def passed(library, cache):
    """What the calls pass on of the cache."""
    seen = []
    x = rows(3, 2, 64)
    nc.nc_kv_write(cache, x, x, on_gpu(torch.arange(3)))
    nc.nc_kv_read(cache, on_gpu(torch.arange(3)), x, rows(3, 2, 64))
    attend(cache)
    for name, args in library.calls:
        seen.append((args[0].data, args[0].pages, args[0].page, args[0].heads, args[0].dim))
    library.calls.clear()
    assert seen
    return set(seen)


def test_calls_follow_assigned_memory(library):
    cache = new_cache()
    assert passed(library, cache) == {(cache.data.data_ptr(), 4, 16, 2, 64)}
    old = cache.data
    cache.data = on_gpu(torch.zeros((7, old.shape[1]), dtype=torch.uint8))
    assert cache.pages == 7 and old.data_ptr() != cache.data.data_ptr()
    assert passed(library, cache) == {(cache.data.data_ptr(), 7, 16, 2, 64)}
    for bad in (on_gpu(torch.zeros((7, old.shape[1] - 1), dtype=torch.uint8)), on_gpu(torch.zeros((7, old.shape[1]))),
                on_gpu(torch.zeros(old.shape[1], dtype=torch.uint8))):
        with pytest.raises(ValueError, match="data: shape"):
            cache.data = bad
    assert passed(library, cache) == {(cache.data.data_ptr(), 7, 16, 2, 64)}


def test_calls_follow_resized_memory(library):
    cache = new_cache()
    each = cache.data.shape[1]
    for pages in (2000, 3, 0):
        cache.data.resize_(pages, each)
        assert passed(library, cache) == {(cache.data.data_ptr() if pages else None, pages, 16, 2, 64)}
        assert cache.pages == pages
    cache = new_cache()
    cache.data.resize_(4, each - 1)
    with pytest.raises(ValueError, match="data: shape"):
        attend(cache)
    assert not [c for c in library.calls if c[0] != "workspace"]


@pytest.mark.parametrize("name", ["page", "heads", "dim", "fmt", "pages", "device", "descriptor"])
def test_sizes_are_fixed(name):
    cache = new_cache()
    with pytest.raises(AttributeError):
        setattr(cache, name, getattr(cache, name))


# -- the GPU that a call is made on -------------------------------------------------

class Devices:
    """Stands for torch.cuda's current device."""

    def __init__(self, monkeypatch, now):
        self.now = now
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.now, raising=False)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.now)
        devices = self

        class Device:
            def __init__(self, to):
                self.to = to.index if isinstance(to, torch.device) else to

            def __enter__(self):
                self.before, devices.now = devices.now, self.to

            def __exit__(self, *exc):
                devices.now = self.before

        monkeypatch.setattr(torch.cuda, "device", Device)


@pytest.mark.parametrize("now", [0, 1])
def test_calls_are_made_on_the_caches_gpu(monkeypatch, library, now):
    """A stream's number 0 means the current device's default stream, so the cache's has to be current."""
    devices = Devices(monkeypatch, now)
    on = []
    monkeypatch.setattr(library, "calls", type("Calls", (list,), {"append": lambda self, call: on.append(
        (call[0], devices.now))})())
    cache, x = new_cache(), rows(3, 2, 64)
    nc.nc_kv_write(cache, x, x, on_gpu(torch.arange(3)))
    nc.nc_kv_read(cache, on_gpu(torch.arange(3)), x, rows(3, 2, 64))
    attend(cache)
    attend(cache, ws=on_gpu(torch.zeros(16, dtype=torch.uint8)), stream=0)
    assert {name for name, _ in on} >= {"nc_kv_write", "nc_kv_read", "nc_kv_attention"}
    assert all(at == 0 for name, at in on if name != "workspace"), on
    assert devices.now == now


def test_the_device_is_set_back_after_a_refusal(monkeypatch, library):
    devices = Devices(monkeypatch, 1)
    library.nc_kv_write = lambda *args: 5
    with pytest.raises(nc.NarrowcastError):
        nc.nc_kv_write(new_cache(), rows(3, 2, 64), rows(3, 2, 64), on_gpu(torch.arange(3)))
    assert devices.now == 1


# -- strides ---------------------------------------------------------------------

def test_a_single_head_has_no_stride(library):
    """Rows of one head as the transpose of columns: torch gives the axis of length 1 the stride 1."""
    cache = new_cache(heads=1)
    x = rows(5, 64, 1).transpose(1, 2)
    assert x.shape == (5, 1, 64) and x.stride() == (64, 1, 1)
    slots = on_gpu(torch.arange(5))
    nc.nc_kv_write(cache, x, x, slots)
    nc.nc_kv_read(cache, slots, x, rows(5, 64, 1).transpose(1, 2))
    attend(cache, q=rows(3, 64, 1).transpose(1, 2), out=rows(3, 64, 1).transpose(1, 2))
    write, read, attention = (args for name, args in library.calls if name != "workspace")
    assert [(r.token_stride, r.head_stride) for r in (*write[1:3], *read[1:3])] == [(64, 0)] * 4
    assert (attention[1].q_token_stride, attention[1].q_head_stride, attention[1].out_head_stride) == (64, 0, 0)
