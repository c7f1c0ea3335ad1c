"""nc_kv_attention where arguments are at the ends of their ranges."""

import pytest
import torch

import scaled_fp8_casting_amd as nc
from tests._kv import check, run_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 60])
@pytest.mark.parametrize("lens,q_lens,heads", [([67, 20], [150, 90], 2), ([67, 3000, 9], [150, 4, 80], 2),
                                               ([190, 70, 64, 500] * 4, [131, 150, 65, 70] * 4, 16)])
def test_windows_without_a_limit(lens, q_lens, heads, window):
    """The largest windows, over fewer tokens than queries: the first queries' ends lie before the cache."""
    check(*run_case(1, "e2m1", "bf16", 64, heads, 2, lens, q_lens, 16, window=window, pairs=min(30, len(lens) * heads)))


def served(max_q, max_kv, batch, lens, q_lens, heads):
    """A call with bounds far above its real sizes against the same call with its own; most sequences are empty."""
    dim, page = 64, 16
    g = torch.Generator(device="cuda").manual_seed(7)
    per = max(-(-n // page) for n in lens)
    cache = nc.new_kv_cache(per * len(lens), page, heads, dim, "e2m1")
    tokens = per * len(lens) * page
    k, v = (torch.randn(tokens, heads, dim, generator=g, device="cuda") for _ in range(2))
    nc.nc_kv_write(cache, k, v, torch.arange(tokens, device="cuda"))
    table = torch.zeros((batch, per), dtype=torch.int32, device="cuda")
    table[:len(lens)] = torch.arange(per * len(lens), dtype=torch.int32, device="cuda").reshape(len(lens), per)
    fill = lambda x: torch.tensor(list(x) + [0] * (batch - len(x)), dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(sum(q_lens), heads, dim, generator=g, device="cuda")
    start = torch.cat([fill([])[:1], fill(q_lens).cumsum(0, dtype=torch.int32)])
    got, want = [], []
    for o, b, mq, mk in ((got, batch, max_q, max_kv), (want, len(lens), max(q_lens), max(lens))):
        o += [torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")]
        nc.nc_kv_attention(cache, q, o[0], start[:b + 1], fill(lens)[:b], table[:b], mq, mk, lse=o[1])
    torch.cuda.synchronize()
    # either call: a score is off by at most (3 dim + 4) 2^-24 of the magnitudes it adds up (below 64 here, 8 sigma of
    # |q| |k| / 8), a weight by twice that relative to their sum, and exp2 and the sums by 2^-20
    score = (3 * dim + 4) * 2.0 ** -24 * 64
    assert ((got[1] - want[1]).abs() <= 2 * (score + 2.0 ** -20 + 2.0 ** -23 * want[1].abs())).all()
    assert ((got[0] - want[0]).abs() <= 2 * (2 * score + 2.0 ** -20) * v.abs().max()).all()


def test_many_sequences_of_possibly_long_prompts():
    """640 sequences of up to 32768 queries over as many tokens: 2.7e9 tiles of row groups, though few are there."""
    served(32768, 32768, 640, [500, 300], [200, 1], 8)


def test_many_sequences_of_possibly_long_caches():
    """Single tokens of 4096 sequences of up to 2^20: 2.1e9 tiles."""
    served(1, 1 << 20, 4096, [3000, 77], [1, 1], 8)


LONG = 1 << 20       # tokens of a page that stands for every page of a sequence of 2^31


def long_cache(batch):
    g = torch.Generator(device="cuda").manual_seed(9)
    cache = nc.new_kv_cache(1, LONG, 1, 64, "e2m1")
    k, v = (torch.randn(LONG, 1, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    nc.nc_kv_write(cache, k, v, torch.arange(LONG, device="cuda"))
    return g, cache, torch.zeros((batch, 2 ** 31 // LONG), dtype=torch.int32, device="cuda")


def last(cache, q, table, batch, n_q, n, **kw):
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    start = torch.arange(0, batch * n_q + 1, n_q, dtype=torch.int32, device="cuda")
    nc.nc_kv_attention(cache, q, out, start, torch.full((batch,), n, dtype=torch.int32, device="cuda"), table, n_q, n, lse=lse,
                       **kw)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("n", [2 ** 31 - 16, 2 ** 31 - 1])
def test_the_longest_sequence(n):
    """2^31 - 16 tokens, a cache's most: one page 2047 times and, but for its last 16 tokens, once more."""
    g, cache, table = long_cache(1)
    q = torch.randn(1, 2, 64, generator=g, device="cuda")
    out, lse = last(cache, q, table, 1, 1, n)
    (o1, l1), (o2, l2) = (last(cache, q, table[:, :1].contiguous(), 1, 1, m) for m in (LONG, LONG - 16))
    w1, w2 = 2047 * torch.exp(l1.double()), torch.exp(l2.double())
    want = (o1 * w1[..., None] + o2 * w2[..., None]) / (w1 + w2)[..., None]
    # a lane sums the weights of 1 of 4 keys, of a wave of at least 4 x 256: 2^31 / 2^12 terms, each addition off by
    # 2^-24 of the sum at most
    off = 2.0 ** 19 * 2.0 ** -24
    assert ((lse - torch.log(w1 + w2)).abs() <= off).all()
    assert ((out - want).abs() <= 2 * off * 6).all()      # no value is above 6


@pytest.mark.parametrize("n_q,batch,group", [(130, 128, 2), (3, 2, 4)])
@pytest.mark.parametrize("window", [100, 116, 132, 148])
def test_the_last_tokens_of_the_longest_sequences(window, n_q, batch, group):
    """The same tokens, in the same places of their tiles and steps, as those of a sequence of one page."""
    g, cache, table = long_cache(batch)
    q = torch.randn(batch * n_q, group, 64, generator=g, device="cuda").bfloat16()
    got = last(cache, q, table, batch, n_q, 2 ** 31 - 16, window=window)
    want = last(cache, q, table[:, :1].contiguous(), batch, n_q, LONG - 16, window=window)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
