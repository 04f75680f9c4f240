"""Calls padded with tens of thousands of sequences without new tokens, through both kernels of the dense paged attention
(needs a GB300)."""
import numpy as np
import pytest

from attention_tools import cache, cache_case
from paged_tools import attend, check, queries
from test_gpu_paged_probabilities import Q  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sequences", [1000, 50000])
def test_sequences_without_new_tokens(Q, sequences):  # noqa: F811
    q_lens, lens = np.zeros(sequences, int), np.zeros(sequences, int)
    for b, (new, total) in {0: (3, 40), 1: (200, 700), sequences // 2: (1, 300), sequences - 1: (150, 150)}.items():
        q_lens[b], lens[b] = new, total
    case = cache_case(layout_q="TND", q_lens=q_lens.tolist(), seq_lens_k=lens.tolist(), block_size=64, sparse_count=1,
                      sparse_mode=3, seed=1)
    hkv, hq, dim = 8, 16, 64
    pool, q = cache(case, hkv, dim, True, 1), queries(case.rows, hq, dim, False, 2)
    check(case, attend(Q, case, q, pool, hkv, True, False), q, pool, hkv, True, False)
