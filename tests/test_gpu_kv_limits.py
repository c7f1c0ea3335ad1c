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
