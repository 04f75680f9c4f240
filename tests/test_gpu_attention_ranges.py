"""Sparse attention of blocks of neighbouring rows where a CTA carries several KV heads, with one or
several ranges of positions, against the 64-bit oracle on a sample of the rows (needs a GB300).

A mask holds the positions of one range: 4096 for groups of 6 query heads and more, fewer for smaller
groups; lists that reach further take a mask per range.  As many blocks of rows as the GPU has SMs, times
8 KV heads, are twice the CTAs that the launch asks for, so each CTA takes two heads one after another."""
import dataclasses

import numpy as np
import pytest

from attention_tools import cache, cache_case
from test_gpu_sparse_attention import Q, _check, _query, _run  # noqa: F401 (Q is a fixture)

pytestmark = pytest.mark.gpu


def _sms():
    import torch
    return torch.cuda.get_device_properties(0).multi_processor_count


def _lists(case, seed):
    """int32 [rows, sparse_count]: distinct positions of the row's sequence in random order, then -1."""
    rng = np.random.default_rng(seed)
    idx = np.full((case.total_q, case.sparse_count), -1, np.int32)
    first = 0
    for end, n in zip(case.seq_lens_q, case.seq_lens_k):
        m = min(case.sparse_count, int(n))
        idx[first:end, :m] = np.argsort(rng.random((end - first, int(n)), np.float32), axis=1)[:, :m]
        first = end
    return idx


def _sample(case, got, q, idx, rows):
    """The same call's case, results, queries and lists for these rows alone."""
    rows = np.unique(rows)
    out, lse, bits = got
    part = dataclasses.replace(case, seq_lens_q=np.searchsorted(rows, case.seq_lens_q).astype(np.int32), total_q=len(rows))
    return part, (out[rows], lse[rows], bits), q[rows], idx[rows]


# query heads, KV heads: groups of 8 and 4
@pytest.mark.parametrize("hq,hkv", [(64, 8), (32, 8)])
@pytest.mark.parametrize("e2m1,f16", [(True, False), (False, True)])
@pytest.mark.parametrize("keys,k", [(5000, 1300), (900, 512)])
@pytest.mark.parametrize("again", [False, True])
def test_heads_of_a_cta(Q, hq, hkv, e2m1, f16, keys, k, again):
    """Every head of a CTA attends to all ranges of its rows' lists; some lists name a position of the first
    range twice."""
    per = min(32, 128 * hkv // hq)                           # rows of a block
    rows = per * _sms()
    case = cache_case(layout_q="TND", q_lens=[rows - 100, 100], seq_lens_k=[keys, keys // 7], block_size=64, sparse_count=k,
                      seed=hq)
    pool = cache(case, hkv, 128, e2m1, seed=1)
    idx = _lists(case, 2)
    sample = np.concatenate([np.random.default_rng(3).integers(0, rows, 8), [0, per, rows - 101, rows - 100, rows - 1]])
    if again:
        for r in sample[:6]:
            low = np.flatnonzero((idx[r] >= 0) & (idx[r] < 100))[:2]
            idx[r, low[0]] = idx[r, low[1]]
    q = _query(rows, hq, 128, f16, 4)
    got = _run(Q, case, q, idx, pool, hkv, e2m1, f16)
    part, got, q, idx = _sample(case, got, q, idx, sample)
    _check(part, got, q, idx, pool, hkv, e2m1, f16)
