"""The example's last step against attention in binary64 over what its caches hold, for a
sequence and an encoder short enough that every token counts."""

import math

import numpy as np
import pytest

from examples import kv_cache_decode as ex
from oracle import kv
from tests._kv import f64, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_every_token_counts(fmt):
    r = ex.run(fmt, prompts=(3, 300), encoder=(5, 40), tokens=4)
    q, scale = f64(r["query"][0]), 1 / math.sqrt(ex.DIM)
    for name, keys, values in (("own", r["keys"][1], r["values"][1]), ("cross", *r["encoder"])):
        k, v, got = kv.held(f64(keys), fmt, "ceil"), kv.held(f64(values), fmt, "ceil"), f64(r[name][0][0])
        n = len(k)
        assert n == {"own": 7, "cross": 5}[name]
        missed = 0
        for j in range(ex.HEADS * ex.GROUP):
            h = j // ex.GROUP
            out, lse, spread, reach = kv.attend(q[j:j + 1], k[:, h], v[:, h], np.ones((1, n), bool), scale)
            off = tolerance(ex.DIM, "bf16", out, lse, spread, reach)[0][0]
            assert (np.abs(got[j] - out[0]) <= off).all(), (name, j)
            # one token fewer would show, at either end
            for part in (slice(1, n), slice(0, n - 1)):
                less = kv.attend(q[j:j + 1], k[part, h], v[part, h], np.ones((1, n - 1), bool), scale)[0][0]
                missed += (np.abs(less - out[0]) <= 2 * off).all()
        assert missed == 0
