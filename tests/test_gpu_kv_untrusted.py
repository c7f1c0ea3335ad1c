"""Lengths, offsets and tables that do not fit, in the many-row kernel and where shares cut
sequences: what they are cut to, bit for bit, and nothing outside it."""

import numpy as np
import pytest
import torch

import scaled_fp8_casting_amd as nc

pytestmark = pytest.mark.gpu

DIM, PAGE = 64, 16


class Calls:
    """batch sequences of n_q queries over kv tokens, the arrays as given."""

    def __init__(self, batch, heads, group, n_q, kv, fmt="e2m1"):
        g = torch.Generator(device="cuda").manual_seed(3)
        self.batch, self.n_q, self.kv, self.per = batch, n_q, kv, -(-kv // PAGE)
        self.cache = nc.new_kv_cache(batch * self.per, PAGE, heads, DIM, fmt)
        tokens = batch * self.per * PAGE
        k, v = (torch.randn(tokens, heads, DIM, generator=g, device="cuda").bfloat16() for _ in range(2))
        nc.nc_kv_write(self.cache, k, v, torch.arange(tokens, device="cuda"))
        self.q = torch.randn(batch * n_q, heads * group, DIM, generator=g, device="cuda").bfloat16()
        self.starts = np.arange(batch + 1) * n_q
        self.lens = kv - 5 * np.arange(batch)
        self.table = np.arange(batch * self.per).reshape(batch, self.per)

    def __call__(self, starts=None, lens=None, table=None, n_q=None, kv=None, causal=True):
        i32 = lambda x, own: torch.tensor(np.ascontiguousarray(own if x is None else x), dtype=torch.int32, device="cuda")  # noqa: E731
        out = torch.full_like(self.q, 5.0)
        lse = torch.full(self.q.shape[:2], 5.0, device="cuda")
        nc.nc_kv_attention(self.cache, self.q, out, i32(starts, self.starts), i32(lens, self.lens), i32(table, self.table),
                           n_q or self.n_q, kv or self.kv, causal=causal, lse=lse)
        torch.cuda.synchronize()
        return out, lse


def same(a, b):
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.fixture(scope="module", params=[dict(batch=16, heads=16, group=1, n_q=100, kv=150),
                                        dict(batch=3, heads=2, group=4, n_q=1, kv=4000),
                                        dict(batch=3, heads=2, group=4, n_q=9, kv=4000, fmt="e4m3")],
                ids=["many", "shares", "shares_rows"])
def calls(request):
    return Calls(**request.param)


@pytest.mark.parametrize("causal", [True, False])
def test_lengths(calls, causal):
    at, cut = calls.lens.copy(), calls.lens.copy()
    at[0], at[1], at[2] = 2 ** 31 - 1, -7, -2 ** 31
    cut[0], cut[1], cut[2] = calls.kv, 0, 0
    got = calls(lens=at, causal=causal)
    same(got, calls(lens=cut, causal=causal))
    n = calls.n_q
    assert not got[0][n:3 * n].any() and torch.isneginf(got[1][n:3 * n]).all()
    assert torch.isfinite(got[1][:n].min(0).values).any()


def test_lengths_above_the_table(calls):
    """Two pages fewer than the lengths need."""
    table = calls.table[:, :-2]
    held = np.minimum(calls.lens, table.shape[1] * PAGE)
    assert (held < calls.lens).any()
    same(calls(table=table), calls(lens=held))


@pytest.mark.parametrize("page", [-1, -2 ** 31, 2 ** 31 - 1, None])
def test_no_page_of_a_sequence_is_there(calls, page):
    table = calls.table.copy()
    table[1] = calls.cache.pages if page is None else page
    got, n = calls(table=table), calls.n_q
    assert not got[0][n:2 * n].any() and torch.isneginf(got[1][n:2 * n]).all()
    whole = calls()
    for part in (slice(0, n), slice(2 * n, None)):
        assert torch.equal(got[0][part], whole[0][part]) and torch.equal(got[1][part], whole[1][part])


@pytest.mark.parametrize("end", ["past q", "before its start", "negative", "largest"])
def test_offsets(calls, end):
    """The last sequence's: it has no queries, and its rows are left alone."""
    starts, none = calls.starts.copy(), calls.starts.copy()
    starts[-1] = {"past q": starts[-1] + 1, "before its start": starts[-2] - 1, "negative": -1, "largest": 2 ** 31 - 1}[end]
    none[-1] = none[-2]
    got = calls(starts=starts)
    same(got, calls(starts=none))
    assert (got[0][-calls.n_q:] == 5).all() and (got[1][-calls.n_q:] == 5).all()
    assert not (got[1][:-calls.n_q] == 5).any()


def test_more_queries_than_max_q():
    """The first max_q of them, as the sequence's last tokens; the others' rows are left alone."""
    for c, most in ((Calls(16, 16, 1, 100, 150), 70), (Calls(3, 2, 4, 9, 4000), 5)):
        got = c(n_q=most)
        for b in range(c.batch):
            rows = slice(b * c.n_q + most, (b + 1) * c.n_q)
            assert (got[0][rows] == 5).all() and (got[1][rows] == 5).all()
        starts = [0, most] + [c.batch * c.n_q] * (c.batch - 1)     # the first sequence alone
        alone = c(starts=starts, n_q=most)
        if c.batch == 16:                                          # a workgroup to itself: the same bits
            assert torch.equal(got[0][:most], alone[0][:most]) and torch.equal(got[1][:most], alone[1][:most])
        else:
            assert not (got[1][:most] == 5).any()
