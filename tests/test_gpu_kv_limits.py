"""nc_kv_attention where arguments are at the ends of their ranges."""

import pytest

from tests._kv import check, run_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 60])
@pytest.mark.parametrize("lens,q_lens,heads", [([67, 20], [150, 90], 2), ([67, 3000, 9], [150, 4, 80], 2),
                                               ([190, 70, 64, 500] * 4, [131, 150, 65, 70] * 4, 16)])
def test_windows_without_a_limit(lens, q_lens, heads, window):
    """The largest windows, over fewer tokens than queries: the first queries' ends lie before the cache."""
    check(*run_case(1, "e2m1", "bf16", 64, heads, 2, lens, q_lens, 16, window=window, pairs=min(30, len(lens) * heads)))
