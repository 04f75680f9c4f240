"""Pins of the oracle's dense paged attention and append: hand-worked visibility, the sparse attention over
complete lists, closed forms, and what invalid lengths and pages leave (no GPU)."""
import math

import numpy as np
import pytest

from attention_tools import cache, cache_case, round_to, table
from oracle import ERR_LENGTH, ERR_PAGE
from oracle import attention as A


def _case(**kw):
    args = dict(batch=2, s1=3, seq_lens_k=[50, 7], block_size=16, sparse_count=1, sparse_mode=3, seed=1)
    args.update(kw)
    return cache_case(**args)


def _q(case, hq, dim, seed=0):
    return round_to(np.random.default_rng(seed).normal(size=(case.rows, hq, dim)), False)


def test_visibility_by_hand():
    c = _case()
    assert A.visible(c, 3, 7, 0) == [0, 1, 2, 3, 4]                       # position 4 of 7
    assert A.visible(c, 3, 7, 2, window=2) == [5, 6]
    assert A.visible(c, 3, 7, 2, window=2, sinks=1) == [0, 5, 6]
    assert A.visible(c, 3, 7, 2, window=2, sinks=6) == [0, 1, 2, 3, 4, 5, 6]
    assert A.visible(c, 3, 2, 0) == [] and A.visible(c, 3, 2, 1) == [0]   # fewer cached than new
    c.cmp_ratio = 4
    assert A.visible(c, 3, 10, 0) == [0, 1] and A.visible(c, 3, 10, 1) == [0, 1, 2]      # positions 7, 8 of 10
    assert A.visible(c, 3, 10, 0, complete=True) == [0, 1] and A.visible(c, 3, 10, 2, complete=True) == [0, 1]
    c.sparse_mode = 0
    assert A.visible(c, 3, 10, 0) == [0, 1, 2] and A.visible(c, 3, 10, 0, window=1, sinks=1) == [0, 2]


@pytest.mark.parametrize("e2m1", [True, False])
@pytest.mark.parametrize("layout", ["BSND", "TND"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 2)])
def test_sparse_attention_over_complete_lists(e2m1, layout, window, sinks):
    more = dict(layout_q="TND", q_lens=[5, 3]) if layout == "TND" else {}
    case = _case(**more)
    pool, q = cache(case, 2, 64, e2m1, 3), _q(case, 6, 64)
    idx = np.full((case.rows, 60), -1, np.int32)
    for b in range(2):
        first, sq, _ = A.sequence_rows(case, b)
        for r in range(sq):
            seen = A.visible(case, sq, int(case.seq_lens_k[b]), r, window, sinks)
            idx[first + r, :len(seen)] = seen
    want = A.sparse_attention(case, q, idx, pool, 2, e2m1, 0.2, 0.5, 3.0)
    got = A.paged_attention(case, q, pool, 2, e2m1, 0.2, 0.5, 3.0, window=window, sinks=sinks)
    assert got[2] == want[2] == 0
    assert np.allclose(got[0], want[0], rtol=1e-12, atol=0) and np.allclose(got[1], want[1], rtol=1e-12, atol=0)


def test_flat_logits_average_the_values():
    case = _case(sparse_mode=0)
    pool, q = cache(case, 1, 64, True, 3), np.zeros((case.rows, 2, 64), np.float32)
    out, lse, err, _ = A.paged_attention(case, q, pool, 1, True, 1.0)
    for b, n in enumerate(case.seq_lens_k):
        v = A.decode(np.stack([pool[A.entry_of(case, b, j, n)[0]] for j in range(n)]), 1, 64, True)[1]
        assert np.allclose(out[3 * b], v.mean(0)) and np.allclose(lse[3 * b], math.log(n))


def test_invalid_lengths_and_pages():
    case = _case(batch=3, q_lens=[3, 4, 2], seq_lens_k=[50, 20, 33])
    pool, q = cache(case, 1, 64, True, 3), _q(case, 1, 64)
    out, lse, err, _ = A.paged_attention(case, q, pool, 1, True, 1.0)
    assert err == ERR_LENGTH and not out[3:6].any() and np.isinf(lse[3:6]).all()          # 4 tokens of at most 3
    assert out[:3].any(1).all() and out[6:8].any(-1).all() and not out[8].any()           # 2 of 3
    case.seq_lens_q[1] = 3
    case.block_table[0, 1] = -1
    out, lse, err, _ = A.paged_attention(case, q, pool, 1, True, 1.0)
    assert err == ERR_PAGE
    assert A.paged_attention(case, q, pool, 1, True, 1.0, window=10)[2] == 0              # positions 38 ... 49
    assert A.paged_attention(case, q, pool, 1, True, 1.0, window=10, sinks=16)[2] == 0
    assert A.paged_attention(case, q, pool, 1, True, 1.0, window=10, sinks=17)[2] == ERR_PAGE
    tnd = _case(layout_q="TND", q_lens=[2, 3])
    tnd.seq_lens_q = np.array([4, 3], np.int32)
    got = A.paged_attention(tnd, _q(tnd, 1, 64), pool, 1, True, 1.0)
    assert got[2] == ERR_LENGTH and not got[0].any()


def test_append_is_the_two_steps():
    case = _case()
    rng = np.random.default_rng(0)
    x = rng.normal(size=(4, 5, 64)).astype(np.float32)
    tb, tp, pos = np.array([0, 1, 0, 5]), np.array([3, 6, 40, 0]), np.array([7, 2, 99, 1])
    cs = table(50, 32)
    w = rng.normal(size=64).astype(np.float32)
    pool = cache(case, 2, 64, True, 3)
    other = pool.copy()
    q, k, err = A.append(case, pool, x[:, :1], x[:, 1:3], x[:, 3:], w, w, pos, cs, 32, False, 1e-6, tb, tp, True)
    assert err == ERR_LENGTH
    assert A.cache_write(case, other, k[:2].astype(np.float32), x[:2, 3:], tb[:2], tp[:2], True) == 0
    assert np.array_equal(pool, other)                     # the token off the table and the one of no batch: not written
    assert not q[2].any() and q[3].any()
