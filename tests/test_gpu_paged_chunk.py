"""The same calls as in test_gpu_paged_attention.py, all of them through the kernel of many rows (the testing build's
switch), and a few that are its own: wide groups of query heads, CTAs that take over pending ones (needs a GB300)."""
import numpy as np
import pytest

import test_gpu_paged_attention as base
from attention_tools import cache, cache_case
from paged_tools import attend, check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_token_block_gb300 import build as B
    B.build()
    import sparse_attention_token_block_gb300 as Q
    saved = Q._lib_handle, Q._lib_path
    Q._lib_handle, Q._lib_path = None, Q.TESTING_LIB_PATH
    Q.lib.qli_testing_set_paged(2)
    yield Q
    Q.lib.qli_testing_set_paged(0)
    Q._lib_handle, Q._lib_path = saved


for name in dir(base):
    if name.startswith("test_") and name not in ("test_long_and_many", "test_far_pool_offsets", "test_chunks_over_many_tiles"):
        globals()[name] = getattr(base, name)


@pytest.mark.parametrize("hq", [256, 255, 254, 201, 129])
def test_wide_groups(Q, hq):
    case = cache_case(layout_q="TND", q_lens=[3, 1, 2], seq_lens_k=[150, 30, 400], block_size=16, sparse_count=1, sparse_mode=3,
                      seed=hq)
    base._both(Q, case, hq, 1, 64)


def test_rows_of_many_blocks(Q):
    """More blocks than CTAs that fit the GPU: each CTA takes several, of different lengths, some without positions."""
    import torch
    lens = [300, 1, 0, 700, 129, 40, 5] * 8
    q_lens = [150, 0, 3, 20, 129, 41, 33] * 8
    case = cache_case(layout_q="TND", q_lens=q_lens, seq_lens_k=lens, block_size=32, sparse_count=1, sparse_mode=3, seed=3)
    hkv, hq, dim = 8, 16, 64
    pool, q = cache(case, hkv, dim, True, 1), queries(case.rows, hq, dim, False, 2)
    got = attend(Q, case, q, pool, hkv, True, False, window=200, sinks=3)
    # the first seven sequences against the oracle, the others (the same lengths) against the kernel of few rows
    rows = sum(q_lens[:7])
    part = cache_case(layout_q="TND", q_lens=q_lens[:7], seq_lens_k=lens[:7], block_size=32, sparse_count=1, sparse_mode=3, seed=3)
    part.block_table, part.num_blocks = case.block_table[:7], case.num_blocks
    check(part, (got[0][:rows], got[1][:rows], got[2]), q[:rows], pool, hkv, True, False, window=200, sinks=3)
    Q.lib.qli_testing_set_paged(1)
    try:
        other = attend(Q, case, q, pool, hkv, True, False, window=200, sinks=3)
    finally:
        Q.lib.qli_testing_set_paged(2)
    assert np.array_equal(np.isinf(got[1]), np.isinf(other[1]))
    # (each within its own rounding of the exact result: two bfloat16 roundings and the probabilities' 2^-11 twice)
    assert np.abs(got[0] - other[0]).max() <= (2.0 ** -8 + 2.0 ** -10) * 2 * np.abs(other[0]).max()
    torch.cuda.synchronize()
