"""Sparse attention of blocks of neighbouring rows whose lists name positions several times, against the
64-bit oracle on a sample of the rows, and what such lists may cost (needs a GB300)."""
import numpy as np
import pytest

from attention_tools import cache, cache_case
from test_gpu_attention_ranges import _lists, _sample, _sms
from test_gpu_sparse_attention import Q, _check, _dev, _query, _run  # noqa: F401 (Q is a fixture)

pytestmark = pytest.mark.gpu


def _repeat(idx, row, times, rng, first=0):
    """Row `row` lists position first + i times[i] times, the rest of it is -1, in random order."""
    flat = np.repeat(first + np.arange(len(times)), times)
    assert len(flat) <= idx.shape[1]
    idx[row] = -1
    idx[row, rng.permutation(idx.shape[1])[:len(flat)]] = flat


@pytest.mark.parametrize("e2m1,f16", [(True, False), (False, True)])
@pytest.mark.parametrize("keys,k", [(2300, 2048), (5000, 1300)])
def test_multiplicities(Q, e2m1, f16, keys, k):
    """Counts of every binary digit up to the whole list, in one block of rows and beside plain lists, in the
    first range of positions and in the next."""
    hq, hkv, per = 64, 8, 16
    rows = per * -(-_sms() // hkv)
    case = cache_case(layout_q="TND", q_lens=[rows], seq_lens_k=[keys], block_size=16, sparse_count=k, seed=5)
    pool = cache(case, hkv, 128, e2m1, seed=1)
    rng = np.random.default_rng(6)
    idx = _lists(case, 2)
    last = keys - 70
    n = 63 if k == 2048 else 50
    _repeat(idx, 1, np.arange(1, n + 1), rng)                                  # 1, 2, 3, ... times
    _repeat(idx, 2, [k], rng, 7)                                               # one position alone
    _repeat(idx, 3, [k // 2, k // 2], rng, last)
    _repeat(idx, 4, [k - 1, 1], rng, last)
    _repeat(idx, 6, [1 << i for i in range(10)], rng, keys - 10)               # a digit each
    idx[7, k // 2:] = 0                                                        # padded with a valid position
    idx[8, ::2] = idx[8, 1::2]                                                 # all twice: no odd count
    _repeat(idx, per + 3, [0, 3, 0, 2, 256, 255], rng, 60)
    idx[per + 4, 5:9] = idx[per + 4, 4]
    sample = np.array([0, 1, 2, 3, 4, 5, 6, 7, 8, 15, per, per + 3, per + 4, rows - 1])
    q = _query(rows, hq, 128, f16, 4)
    got = _run(Q, case, q, idx, pool, hkv, e2m1, f16)
    part, got, q, idx = _sample(case, got, q, idx, sample)
    _check(part, got, q, idx, pool, hkv, e2m1, f16)


def test_cost_of_a_repeated_position(Q):
    """A list that names one position 2048 times has counts of twelve binary digits at most, each a round over
    the masks beside the first look at the lists: the block that holds it takes at most 13 times as long,
    and so does the call."""
    import torch
    hq, hkv, rows, keys, k = 64, 8, 16 * _sms(), 2300, 2048
    case = cache_case(layout_q="TND", q_lens=[rows], seq_lens_k=[keys], block_size=64, sparse_count=k, seed=5)
    p = Q.make_problem(batch=1, layout_q=Q.TND, total_q_tokens=rows, num_blocks=case.num_blocks, block_size=64,
                       max_blocks_per_seq=case.max_blocks_per_seq, sparse_count=k, sparse_mode=0, cmp_ratio=1,
                       max_seqlen_q=rows, max_seqlen_k=keys)
    a = Q.make_attention(num_heads_q=hq, num_heads_kv=hkv, head_dim=128)
    pool = _dev(cache(case, hkv, 128, True, seed=1))
    q = torch.randn(rows, hq, 128, device="cuda").bfloat16()
    out = torch.empty_like(q)
    args = _dev(case.seq_lens_q), _dev(case.seq_lens_k), _dev(case.block_table)
    idx = _dev(_lists(case, 2))

    def us():
        times = []
        for _ in range(5):
            start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            Q.check(Q.sparse_attention(p, a, q, *args, idx, pool, out), "sparse_attention")
            stop.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(stop) * 1e3)
        return min(times[2:])

    plain = us()
    idx[5] = 7
    once = us()
    idx[7, 1024:] = 0
    assert max(once, us()) < 13 * plain
