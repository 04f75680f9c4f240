"""Sequences long enough for the largest clusters of the kernel of few rows, and chunks over many tiles through the kernel of
many rows (needs a GB300)."""
import pytest

import test_gpu_paged_attention as base
from attention_tools import cache_case
from test_gpu_paged_chunk import Q as many_rows  # noqa: F401 (a fixture)
from test_gpu_paged_attention import Q  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


# 16 CTAs of 8 warps that keep 16 steps of 32 positions each: 65536 positions and more
@pytest.mark.parametrize("hq,hkv,dim", [(8, 1, 128), (16, 1, 128), (8, 1, 64), (16, 1, 64), (10, 2, 128)])
@pytest.mark.parametrize("f16", [False, True])
def test_clusters_of_sixteen(Q, hq, hkv, dim, f16):  # noqa: F811
    case = cache_case(batch=1, s1=1, seq_lens_k=[66001], block_size=64, sparse_count=1, sparse_mode=3, seed=hq)
    base._both(Q, case, hq, hkv, dim, e2m1=hq == 8, f16=f16)


@pytest.mark.parametrize("q_lens,lens", [([300], [2000]), ([33, 129, 1], [1300, 129, 700]), ([64], [4001])])
@pytest.mark.parametrize("hq,hkv,dim", [(4, 2, 64), (3, 3, 128), (8, 1, 128)])
@pytest.mark.parametrize("e2m1,f16", [(True, False), (False, True)])
def test_chunks_over_many_tiles(many_rows, q_lens, lens, hq, hkv, dim, e2m1, f16):  # noqa: F811
    case = cache_case(layout_q="TND", q_lens=q_lens, seq_lens_k=lens, block_size=64, sparse_count=1, sparse_mode=3, seed=dim)
    base._both(many_rows, case, hq, hkv, dim, e2m1, f16)
    base._both(many_rows, case, hq, hkv, dim, e2m1, f16, window=333, sinks=20)
