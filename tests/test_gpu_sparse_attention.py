"""Attention over listed entries of the 4-bit cache on the GPU (qli_sparse_attention) against the
64-bit oracle (needs a GB300)."""
import math

import numpy as np
import pytest

import workloads as W
from attention_tools import attention_bounds, cache, cache_case, round_to
from oracle import attention as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_token_block_gb300 import build as B
    B.build()
    import sparse_attention_token_block_gb300 as Q
    return Q


def _dev(a, f16=None):
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if f16 is None else t.to(torch.float16 if f16 else torch.bfloat16)


def _attention(Q, case, hq, hkv, dim, e2m1, f16, **kw):
    return (Q.make_problem(**W.problem_kwargs(case)),
            Q.make_attention(num_heads_q=hq, num_heads_kv=hkv, head_dim=dim, dtype=Q.ACT_F16 if f16 else Q.ACT_BF16,
                             kv_dtype=Q.KV_E2M1 if e2m1 else Q.KV_INT4, **kw))


def _run(Q, case, query, idx, pool, hkv, e2m1, f16, scale=0.0, factors=(1.0, 1.0), kv_stride=0, with_k=True, q_pad=0):
    """The call on fresh buffers: (out, lse, error bits)."""
    import torch
    rows, hq, dim = query.shape
    p, a = _attention(Q, case, hq, hkv, dim, e2m1, f16, softmax_scale=scale, k_scale=factors[0], v_scale=factors[1],
                      kv_stride=kv_stride)
    qd = _dev(np.concatenate([query, np.ones((rows, q_pad, dim), np.float32)], 1), f16)[:, :hq]
    out = torch.full((rows, hq, dim), 5.0, dtype=qd.dtype, device="cuda")
    lse = torch.full((rows, hq), 5.0, dtype=torch.float32, device="cuda")
    ws = torch.zeros(64, dtype=torch.int32, device="cuda")
    args = (_dev(case.seq_lens_q), _dev(case.seq_lens_k) if with_k else None, _dev(case.block_table), _dev(idx), _dev(pool))
    Q.check(Q.sparse_attention(p, a, qd, *args, out, lse, ws), "sparse_attention")
    bits = Q.get_device_error(ws)[1]
    again = torch.empty_like(out)
    Q.check(Q.sparse_attention(p, a, qd, *args, again), "sparse_attention")    # no lse, no workspace
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))         # and the same result
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), bits


def _check(case, got, query, idx, pool, hkv, e2m1, f16, scale=0.0, factors=(1.0, 1.0), with_k=True):
    out, lse, bits = got
    d = query.shape[2]
    ref, rl, err, spread = A.sparse_attention(case, query, idx, pool, hkv, e2m1, scale or 1 / math.sqrt(d), *factors,
                                              use_seq_lens_k=with_k)
    assert bits == err
    tol, ltol = attention_bounds(ref, rl, spread, d, f16)
    bad = ~(np.abs(out - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], out[bad][:3], ref[bad][:3], tol[bad][:3])
    empty = np.isinf(rl)
    assert np.array_equal(np.isinf(lse), empty) and (lse[empty] < 0).all()
    assert np.all(np.abs(lse - rl)[~empty] <= ltol[~empty])
    assert not out[empty].any()


def _query(rows, hq, dim, f16, seed, std=1.0):
    return round_to(np.random.default_rng(seed).normal(size=(rows, hq, dim)) * std, f16)


# query heads, KV heads, D: groups of 1 ... 64, odd numbers of heads on both sides
HEADS = [(8, 1, 128), (64, 8, 128), (4, 4, 64), (7, 1, 64), (15, 3, 128), (10, 5, 64), (28, 4, 64), (16, 1, 128),
         (33, 3, 64), (32, 16, 128), (40, 2, 128), (64, 1, 128), (64, 2, 64), (64, 64, 64), (9, 9, 128), (256, 2, 64)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("e2m1,f16", [(True, False), (False, True)])
def test_head_layouts(Q, heads, e2m1, f16):
    hq, hkv, dim = heads
    case = cache_case(batch=2, s1=2, seq_lens_k=[150, 77], block_size=16, sparse_count=100, seed=hq)
    pool = cache(case, hkv, dim, e2m1, seed=1)
    idx = W.random_indices(case, seed=2)
    q = _query(4, hq, dim, f16, 3)
    _check(case, _run(Q, case, q, idx, pool, hkv, e2m1, f16, q_pad=1), q, idx, pool, hkv, e2m1, f16)


@pytest.mark.parametrize("k", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 257, 511, 513, 1000, 1025, 2047, 2048])
@pytest.mark.parametrize("rows", [1, 3])
def test_list_lengths(Q, k, rows):
    case = cache_case(batch=rows, s1=1, seq_lens_k=[3000, 1900, 60][:rows], block_size=64, sparse_count=k, seed=k)
    pool = cache(case, 2, 128, True, seed=1)
    idx = W.random_indices(case, seed=2, frac_pad=0.0)
    q = _query(rows, 16, 128, False, 3)
    _check(case, _run(Q, case, q, idx, pool, 2, True, False), q, idx, pool, 2, True, False)


@pytest.mark.parametrize("e2m1", [True, False])
@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
def test_many_rows_tnd_compressed(Q, e2m1, f16, dim):
    """More rows than the GPU takes at once, ragged sequences (one empty), compressed positions, pages with
    a gap, factors that are no powers of two, a logit factor of its own."""
    case = cache_case(layout_q="TND", q_lens=[201, 0, 150, 3], seq_lens_k=[801, 60, 333, 3], block_size=48,
                      sparse_count=70, cmp_ratio=4, seed=7)
    hkv, factors = 3, (0.7, 3.0)
    pool = cache(case, hkv, dim, e2m1, 1, *factors)
    eb = pool.shape[2]
    gap = np.random.default_rng(4).integers(0, 256, (case.num_blocks, 48 * eb + 32), dtype=np.uint8)
    gap[:, :48 * eb] = pool.reshape(case.num_blocks, -1)
    idx = W.random_indices(case, seed=2)
    q = _query(354, 6, dim, f16, 3)
    got = _run(Q, case, q, idx, gap, hkv, e2m1, f16, 0.11, factors, 48 * eb + 32)
    _check(case, got, q, idx, pool, hkv, e2m1, f16, 0.11, factors)


@pytest.mark.parametrize("heads", [(8, 1, 128), (64, 8, 128), (24, 3, 64), (32, 4, 64)])
@pytest.mark.parametrize("gap", [0, 1, 3])
def test_page_strides_of_whole_entries(Q, heads, gap):
    """Pages that lie a whole number of entries apart."""
    hq, hkv, dim = heads
    case = cache_case(batch=3, s1=1, seq_lens_k=[300, 90, 33], block_size=32, sparse_count=96, seed=hq)
    pool = cache(case, hkv, dim, True, seed=1)
    eb = pool.shape[2]
    raw = np.random.default_rng(4).integers(0, 256, (case.num_blocks, (32 + gap) * eb), dtype=np.uint8)
    raw[:, :32 * eb] = pool.reshape(case.num_blocks, -1)
    idx = W.random_indices(case, seed=2)
    q = _query(3, hq, dim, False, 3)
    got = _run(Q, case, q, idx, raw, hkv, True, False, kv_stride=(32 + gap) * eb)
    _check(case, got, q, idx, pool, hkv, True, False)


def test_scattered_padding_duplicates_and_empty_rows(Q):
    """-1 anywhere in a list, whole tiles of it, rows of nothing else, one entry listed many times."""
    rng = np.random.default_rng(8)
    case = cache_case(batch=8, s1=1, seq_lens_k=[400] * 8, block_size=16, sparse_count=300, seed=8)
    pool = cache(case, 4, 64, True, seed=1)
    idx = W.random_indices(case, seed=2, frac_pad=0.0)
    idx[0, rng.random(300) < 0.5] = -1
    idx[1, :] = -1
    idx[2, :299] = -1                                        # only the last
    idx[3, 1:] = -1                                          # only the first
    idx[4, 32:260] = -1                                      # whole tiles in the middle
    idx[5, :] = 17                                           # one entry 300 times
    idx[6, ::2] = -1
    q = _query(8, 32, 64, False, 3)
    _check(case, _run(Q, case, q, idx, pool, 4, True, False), q, idx, pool, 4, True, False)


def test_unlisted_and_padding_bytes_are_never_used(Q):
    """Slots that no list names, and scale bytes of NaN in them, do not reach the result."""
    case = cache_case(batch=3, s1=1, seq_lens_k=[90, 33, 50], block_size=32, sparse_count=40, seed=9)
    pool = cache(case, 3, 64, True, seed=1)
    idx = W.random_indices(case, seed=2)
    idx[1, 5:] = -1
    used = np.zeros(pool.shape[:2], bool)
    for b in range(3):
        j = idx[b][idx[b] >= 0]
        used[case.block_table[b, j // 32], j % 32] = True
    poisoned = np.where(used[..., None], pool, np.uint8(0x7F))
    poisoned[..., 3 * 72:] = 0xFF
    q = _query(3, 6, 64, True, 3)
    _check(case, _run(Q, case, q, idx, poisoned, 3, True, True), q, idx, pool, 3, True, True)


@pytest.mark.parametrize("order", ["rising", "falling", "spike"])
def test_large_logits(Q, order):
    """Logits of several hundred whose maximum comes first, last, or alone in the middle."""
    case = cache_case(batch=1, s1=1, seq_lens_k=[700], block_size=64, sparse_count=700, seed=3)
    n = case.num_blocks * 64
    rng = np.random.default_rng(1)
    size = {"rising": np.linspace(0.1, 6, 700), "falling": np.linspace(6, 0.1, 700), "spike": np.full(700, 0.2)}[order]
    if order == "spike":
        size[333] = 6.0
    k = np.zeros((n, 1, 128), np.float32)
    base = rng.choice([-1.0, 1.0], 128)
    slot = np.array([case.block_table[0, j // 64] * 64 + j % 64 for j in range(700)])
    k[slot, 0] = size[:, None] * base
    v = rng.normal(size=(n, 1, 128)).astype(np.float32)
    pool = A.encode(k, v, True).reshape(case.num_blocks, 64, -1)
    q = round_to(np.stack([base * s for s in (8.0, -8.0, 0.01, 1.0, 0.0)])[None], False)
    idx = np.arange(700, dtype=np.int32)[None]
    _check(case, _run(Q, case, q, idx, pool, 1, True, False), q, idx, pool, 1, True, False)


def test_query_magnitudes(Q):
    """Heads of very different sizes, some beyond fp16's range (bfloat16 queries), some all zero."""
    case = cache_case(batch=2, s1=1, seq_lens_k=[200, 200], block_size=16, sparse_count=128, seed=3)
    pool = cache(case, 1, 128, False, seed=1)
    q = _query(2, 8, 128, False, 3)
    q[0] *= np.array([1, 1e-6, 1e-30, 1e5, 0, 1e-3, 3e38 / 8, 2.0 ** -133], np.float32)[:, None]
    q = round_to(q, False)
    idx = W.random_indices(case, seed=2)
    for scale in (0.05, 1e-37):
        keep = np.abs(q).max(-1, keepdims=True) < 1e30 if scale == 0.05 else np.ones((2, 8, 1), bool)
        qq = np.where(keep, q, np.float32(0))
        _check(case, _run(Q, case, qq, idx, pool, 1, False, False, scale), qq, idx, pool, 1, False, False, scale)


def test_invalid_indices_and_pages(Q):
    case = cache_case(batch=2, s1=1, seq_lens_k=[100, 40], block_size=32, sparse_count=8, seed=5)
    pool = cache(case, 2, 128, True, seed=6)
    idx = np.array([[0, 99, -1, -1, -1, -1, -1, -1], [40, -5, 3, 63, 64, -1, 2147483647, -2147483648]], np.int32)
    q = _query(2, 4, 128, False, 3)
    for with_k in (True, False):
        _check(case, _run(Q, case, q, idx, pool, 2, True, False, with_k=with_k), q, idx, pool, 2, True, False,
               with_k=with_k)
    case.block_table[0, 3] = case.num_blocks + 2
    case.block_table[1, 0] = -3
    _check(case, _run(Q, case, q, idx, pool, 2, True, False), q, idx, pool, 2, True, False)


def test_tnd_rows_past_the_last_prefix_sum(Q):
    case = cache_case(layout_q="TND", q_lens=[2, 2], seq_lens_k=[64, 64], block_size=32, sparse_count=4, seed=7)
    case.total_q = 6
    pool = cache(case, 1, 64, True, seed=8)
    idx = np.full((6, 4), -1, np.int32)
    idx[:, 0] = 1
    idx[5, 0] = -1
    q = _query(6, 2, 64, False, 3)
    _check(case, _run(Q, case, q, idx, pool, 1, True, False), q, idx, pool, 1, True, False)


def test_rows_without_any_batch(Q):
    """TND rows of an empty batch: no lengths, table or cache at all."""
    import torch
    p = Q.make_problem(batch=0, layout_q=Q.TND, total_q_tokens=5, num_blocks=1, block_size=16, max_blocks_per_seq=0,
                       sparse_count=40, sparse_mode=0, cmp_ratio=1, max_seqlen_q=0, max_seqlen_k=0)
    a = Q.make_attention(num_heads_q=64, num_heads_kv=8, head_dim=128)
    out = torch.full((5, 64, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(5, 64, device="cuda")
    ws = torch.zeros(64, dtype=torch.int32, device="cuda")
    for last, bits in ((-1, 0), (7, 1)):
        idx = torch.full((5, 40), -1, dtype=torch.int32, device="cuda")
        idx[4, 39] = last
        Q.check(Q.sparse_attention(p, a, torch.ones_like(out), None, None, None, idx, None, out, lse, ws), "sparse_attention")
        assert Q.get_device_error(ws)[1] == bits
        assert not out.any() and (lse == -math.inf).all()


def test_offsets_past_32_bits(Q):
    """Entries on the last pages of a pool of over 4 GB."""
    import torch
    bs, nb, hkv = 1024, 20, 8
    page = bs * 1152 + (1 << 28)
    case = cache_case(batch=1, s1=1, seq_lens_k=[2 * bs], block_size=bs, sparse_count=64, seed=1)
    case.num_blocks = nb
    case.block_table = np.array([[nb - 1, nb - 2]], np.int32)
    small = cache(case, hkv, 128, True, seed=1)
    pool = torch.zeros(nb * page, dtype=torch.uint8, device="cuda")
    for pg in (nb - 1, nb - 2):
        pool[pg * page:pg * page + bs * 1152] = _dev(small[pg].reshape(-1))
    idx = np.random.default_rng(2).permutation(2 * bs)[:64].astype(np.int32)[None]
    q = _query(1, 64, 128, False, 3)
    p, a = _attention(Q, case, 64, hkv, 128, True, False, kv_stride=page)
    out = torch.empty(1, 64, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 64, dtype=torch.float32, device="cuda")
    Q.check(Q.sparse_attention(p, a, _dev(q, False), None, _dev(case.seq_lens_k), _dev(case.block_table), _dev(idx), pool, out,
                               lse), "sparse_attention")
    _check(case, (out.double().cpu().numpy(), lse.double().cpu().numpy(), 0), q, idx, small, hkv, True, False)


def test_runs_on_its_stream_and_in_a_graph(Q):
    """Captured on a stream of its own and replayed on new queries, lists and cache contents."""
    import torch
    case = cache_case(batch=4, s1=1, seq_lens_k=[300] * 4, block_size=16, sparse_count=128, seed=2)
    p, a = _attention(Q, case, 16, 2, 128, True, False)
    shape = cache(case, 2, 128, True, seed=1).shape
    pool = torch.zeros(shape, dtype=torch.uint8, device="cuda")
    q = torch.zeros(4, 16, 128, dtype=torch.bfloat16, device="cuda")
    idx = torch.full((4, 128), -1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    lse = torch.empty(4, 16, dtype=torch.float32, device="cuda")
    sk, bt = _dev(case.seq_lens_k), _dev(case.block_table)
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            Q.check(Q.sparse_attention(p, a, q, None, sk, bt, idx, pool, out, lse), "sparse_attention")
    for seed in (1, 2):
        hp, hq, hi = cache(case, 2, 128, True, seed), _query(4, 16, 128, False, seed), W.random_indices(case, seed)
        pool.copy_(_dev(hp))
        q.copy_(_dev(hq, False))
        idx.copy_(_dev(hi))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _check(case, (out.double().cpu().numpy(), lse.double().cpu().numpy(), 0), hq, hi, hp, 2, True, False)


def test_after_the_indexer_on_one_stream(Q):
    """The whole layer step: rotate, write the cache, select, attend, without a synchronisation between."""
    import torch
    case = cache_case(batch=3, s1=2, seq_lens_k=[500, 260, 90], block_size=32, sparse_count=64, sparse_mode=3, seed=4)
    hq, hkv, dim = 16, 2, 128
    p, a = _attention(Q, case, hq, hkv, dim, True, False)
    pool = cache(case, hkv, dim, True, seed=1)
    d = W.to_device(case)
    ix = Q.Indexer(p)
    dp = _dev(pool)
    k = round_to(np.random.default_rng(9).normal(size=(3, hkv, dim)), False)
    tb, tp = np.arange(3, dtype=np.int32), (case.seq_lens_k - 1).astype(np.int32)
    q = _query(6, hq, dim, False, 3)
    out = torch.empty(6, hq, dim, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(6, hq, dtype=torch.float32, device="cuda")
    kd, qd, tbd, tpd = _dev(k, False), _dev(q, False), _dev(tb), _dev(tp)
    Q.check(Q.kv_write(p, a, kd, kd, tbd, tpd, d["block_table"], dp, ix.workspace), "kv_write")
    idx = ix.run(**d)
    Q.check(Q.sparse_attention(p, a, qd, d["seq_lens_q"], d["seq_lens_k"], d["block_table"], idx, dp, out, lse, ix.workspace),
            "sparse_attention")
    assert ix.device_error() == (0, 0)
    assert A.cache_write(case, pool, k, k, tb, tp, True) == 0
    _check(case, (out.double().cpu().numpy(), lse.double().cpu().numpy(), 0), q, idx.cpu().numpy(), pool, hkv, True, False)
