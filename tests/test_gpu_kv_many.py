"""nc_kv_attention where a workgroup for each 128 rows fills the card, and where its
shares cut sequences: against softmax attention in binary64 over what the cache holds."""

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc
from tests._kv import check, run_case

pytestmark = pytest.mark.gpu

# 16 sequences x 16 heads: queries of all cached tokens, of the last ones, none, and more than there are tokens
LENS = [190, 300, 70, 129, 64, 257, 31, 500, 128, 200, 77, 1, 320, 96, 150, 403]
QS = [190, 131, 150, 129, 65, 128, 31, 70, 100, 66, 77, 90, 0, 96, 150, 99]


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompts(fmt, dtype, dim):
    check(*run_case(dim, fmt, dtype, dim, 16, 1, LENS, QS, 16, pairs=30))


@pytest.mark.parametrize("group", [1, 3, 8])
@pytest.mark.parametrize("page", [16, 48, 64])
def test_groups_and_pages(group, page):
    check(*run_case(group + page, "e2m1", "bf16", 64, 16, group, LENS, QS, page, pairs=30))


@pytest.mark.parametrize("fmt,dtype,dim", [("e2m1", "bf16", 128), ("e4m3", "bf16", 64), ("e4m3", "fp32", 96)])
def test_cross(fmt, dtype, dim):
    check(*run_case(3, fmt, dtype, dim, 16, 1, LENS, [100] * 16, 16, causal=False, pairs=30))


@pytest.mark.parametrize("window", [1, 16, 65, 130, 1000])
@pytest.mark.parametrize("causal", [True, False])
def test_window(window, causal):
    check(*run_case(window, "e2m1", "bf16", 64, 16, 2, LENS, QS, 32, causal=causal, window=window, pairs=30))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [0.0, -0.4, 3.0])
def test_scale_and_strides(dtype, scale):
    check(*run_case(5, "e4m3", dtype, 96, 16, 1, LENS, QS, 16, scale=scale, sliced=True, pairs=30))


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_nan_reaches_only_rows_that_see_it(fmt):
    """One in the part of the keys that every row sees, others where only some rows see them."""
    at = np.cumsum([0] + LENS)

    def mutate(k, v, q):
        v[at[1] + 10, :, 5] = float("nan")      # seen by every row of a sequence of 300
        v[at[1] + 280, :, 37] = float("nan")    # by its last ones
        v[at[7] + 460, :, 60] = float("nan")
        k[at[0] + 150, :, 3] = float("nan")
    check(*run_case(6, fmt, "bf16", 64, 16, 1, LENS, QS, 16, mutate=mutate, pairs=60))


def test_pages_outside_the_cache():
    check(*run_case(7, "e2m1", "bf16", 64, 16, 1, LENS, QS, 16, lose=((0, 3), (0, 11), (1, 0), (7, 20), (15, 25)), pairs=60))


@pytest.mark.parametrize("fmt,dtype,dim", [("e2m1", "bf16", 64), ("e4m3", "fp32", 64)])
def test_long(fmt, dtype, dim):
    """More than 64 steps of 64 keys."""
    check(*run_case(8, fmt, dtype, dim, 128, 1, [5000, 4300], [130, 200], 64, pairs=8))


@pytest.mark.parametrize("fmt,dtype,dim", [("e2m1", "bf16", 128), ("e2m1", "bf16", 256), ("e4m3", "bf16", 96),
                                           ("e4m3", "fp32", 192), ("e2m1", "fp32", 64)])
@pytest.mark.parametrize("n_q", [1, 7])
@pytest.mark.parametrize("causal", [True, False])
def test_shares(fmt, dtype, dim, n_q, causal):
    """Shares that begin and end inside sequences, whole sequences inside a share, empty ones between."""
    lens = [3000, 1, 40, 2100, 17, 300, 0, 5, 900, 2700, 16, 33]
    qs = [n_q] * 4 + [0, n_q, n_q, 0, n_q, n_q, n_q, 0]
    check(*run_case(n_q, fmt, dtype, dim, 4, 3, lens, qs, 32, causal=causal, pairs=50))


def test_shares_over_many_sequences():
    """More sequences than a wave has lanes."""
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 400, 150).tolist()
    lens[70], lens[149] = 2500, 2300
    qs = rng.integers(0, 3, 150).tolist()
    qs[70], qs[149] = 2, 1
    check(*run_case(2, "e2m1", "bf16", 64, 2, 2, lens, qs, 16, pairs=200))


@pytest.mark.parametrize("window", [100, 2500])
def test_shares_with_window(window):
    check(*run_case(4, "e4m3", "bf16", 64, 2, 4, [5000, 60, 3100], [5, 3, 9], 64, window=window))


def test_shares_and_pages_outside_the_cache():
    check(*run_case(9, "e2m1", "bf16", 128, 2, 4, [4000, 2500], [2, 1], 64, lose=((0, 0), (0, 31), (0, 62), (1, 7))))


def test_offsets_past_32_bits():
    """The last pages of a cache of more than 4 GiB."""
    dim, page, heads = 128, 64, 8
    each = nc.kv_page_bytes(page, heads, dim, "e4m3")
    pages = (9 << 29) // each + 3
    cache = nc.new_kv_cache(pages, page, heads, dim, "e4m3")
    assert cache.data.numel() > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(128, heads, dim, generator=g, device="cuda") for _ in range(2))
    q = torch.randn(3, heads, dim, generator=g, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = []
    for first in (0, pages - 2):
        nc.nc_kv_write(cache, k, v, torch.arange(first * page, first * page + 128, device="cuda"))
        out, lse = torch.empty_like(q), torch.empty(3, heads, device="cuda")
        nc.nc_kv_attention(cache, q, out, i32(0, 3), i32(128), i32([first, first + 1]), 3, 128, lse=lse)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        nc.nc_kv_read(cache, torch.arange(first * page, first * page + 128, device="cuda"), ko, vo)
        got.append((out, lse, ko, vo))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    del cache
    torch.cuda.empty_cache()


def test_many_rows_graph_and_same_bits():
    dim, page, heads, n_q, kv = 64, 64, 64, 600, 900
    g = torch.Generator(device="cuda").manual_seed(4)
    pages = -(-kv // page)
    cache = nc.new_kv_cache(pages, page, heads, dim, "e2m1")
    k, v = (torch.randn(kv, heads, dim, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(n_q, heads, dim, generator=g, device="cuda").bfloat16()
    starts = torch.tensor([0, n_q], dtype=torch.int32, device="cuda")
    lens = torch.tensor([kv], dtype=torch.int32, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    slots = torch.arange(kv, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(n_q, heads, device="cuda")

    def step(o, l):
        nc.nc_kv_write(cache, k, v, slots)
        nc.nc_kv_attention(cache, q, o, starts, lens, table, n_q, kv, lse=l)

    step(out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, lse)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    for i in range(4):
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        v.copy_(torch.randn(v.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        step(o2, l2)
        torch.cuda.synchronize()
        assert torch.equal(got[0], o2) and torch.equal(got[1], l2), i
