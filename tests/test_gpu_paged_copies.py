"""The lanes that copy a step's two halves in the kernel of few rows go by one test for a free stage: with the testing build's
switch that makes every second lane's own test fail, the results are the same bits (needs a GB300)."""
import numpy as np
import pytest

from attention_tools import cache, cache_case
from paged_tools import attend, queries
from test_gpu_paged_probabilities import Q  # noqa: F401 (a fixture: the testing build)

pytestmark = pytest.mark.gpu


# several parts a CTA and one; clusters; rings that come round many times
@pytest.mark.parametrize("batch,lens,hq,hkv,dim", [(1, 20000, 8, 1, 128), (3, 3001, 16, 2, 64), (160, 400, 16, 8, 64), (5, 700, 9, 3, 64)])
@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("Q", [1], indirect=True, ids=["few"])
def test_pairs_of_lanes_agree(Q, batch, lens, hq, hkv, dim, window):  # noqa: F811
    case = cache_case(batch=batch, s1=1, seq_lens_k=[lens - b for b in range(batch)], block_size=64, sparse_count=1, sparse_mode=3,
                      seed=batch)
    pool, q = cache(case, hkv, dim, True, 1), queries(case.rows, hq, dim, False, 2)
    want = attend(Q, case, q, pool, hkv, True, False, window=window)
    Q.lib.qli_testing_set_stall(3)
    try:
        got = attend(Q, case, q, pool, hkv, True, False, window=window)
    finally:
        Q.lib.qli_testing_set_stall(0)
    assert got[2] == want[2] == 0
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
