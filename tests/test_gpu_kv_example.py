"""examples/kv_cache_decode.py: prompts, graph-replayed tokens and cross attention over one cache."""

import pytest
import torch

from examples import kv_cache_decode as ex

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,apart", [("e2m1", 0.5), ("e4m3", 0.125)])
def test_example(fmt, apart):
    """What comes back differs from the unquantised by at most the format's half step: relative to a
    value 1/4 for E2M1 (from 1 to 1.5 is a whole step; 1/2 below its smallest normal, where it is
    absolute) and 2^-4 for E4M3, doubled for the weights that the scores' errors move."""
    r = ex.run(fmt, prompts=(300, 16, 1), encoder=(40, 65, 7), tokens=6)
    for name in ("keys", "values", "own", "cross"):
        got, want = (x.float() for x in r[name])
        assert torch.isfinite(got).all()
        assert (got - want).norm() <= apart * want.norm(), name
