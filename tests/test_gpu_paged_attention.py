"""Dense attention of new tokens over the paged 4-bit cache (qli_paged_attention) against the 64-bit oracle (needs
a GB300)."""
import numpy as np
import pytest

from attention_tools import cache, cache_case
from oracle import attention as A
from paged_tools import attend, check, dev, queries, round_to, settings

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


def _both(Q, case, hq, hkv, dim, e2m1=True, f16=False, seed=1, factors=(1.0, 1.0), std=1.0, **kw):
    pool = cache(case, hkv, dim, e2m1, seed, *factors)
    q = queries(case.rows, hq, dim, f16, seed + 1, std)
    more = {k: v for k, v in kw.items() if k in ("kv_stride", "q_pad")}
    rest = {k: v for k, v in kw.items() if k not in more}
    sent = pool
    if "kv_stride" in more:
        flat = pool.reshape(pool.shape[0], -1)
        sent = np.random.default_rng(5).integers(0, 256, (pool.shape[0], more["kv_stride"]), dtype=np.uint8)
        sent[:, :flat.shape[1]] = flat
    check(case, attend(Q, case, q, sent, hkv, e2m1, f16, factors=factors, **more, **rest), q, pool, hkv, e2m1, f16,
          factors=factors, **rest)


# query heads, KV heads, D: groups of 1 ... 64, odd numbers of heads on both sides
HEADS = [(8, 1, 128), (64, 8, 128), (4, 4, 64), (7, 1, 64), (15, 3, 128), (10, 5, 64), (28, 4, 64), (16, 1, 128),
         (33, 3, 64), (32, 16, 128), (40, 2, 128), (64, 1, 128), (64, 2, 64), (64, 64, 64), (9, 9, 128), (256, 2, 64)]


@pytest.mark.parametrize("hq,hkv,dim", HEADS)
@pytest.mark.parametrize("e2m1,f16", [(True, False), (False, True)])
def test_heads(Q, hq, hkv, dim, e2m1, f16):
    case = cache_case(batch=2, s1=2, seq_lens_k=[75, 130], block_size=16, sparse_count=1, sparse_mode=3, seed=hq)
    _both(Q, case, hq, hkv, dim, e2m1, f16)


@pytest.mark.parametrize("lens", [[1], [0, 1, 2], [15, 16, 17], [31, 32, 33], [63, 64, 65], [127, 128, 129], [1, 700, 0, 257]])
@pytest.mark.parametrize("s1", [1, 2, 5])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 3)])
def test_lengths(Q, lens, s1, window, sinks):
    case = cache_case(batch=len(lens), s1=s1, seq_lens_k=lens, block_size=32, sparse_count=1, sparse_mode=3, seed=s1)
    _both(Q, case, 8, 2, 128, window=window, sinks=sinks)


@pytest.mark.parametrize("block_size", [16, 48, 64, 80, 128, 1024])
@pytest.mark.parametrize("cmp_ratio,complete", [(1, False), (4, False), (4, True), (128, False)])
@pytest.mark.parametrize("mode", [0, 3])
def test_pages_and_compression(Q, block_size, cmp_ratio, complete, mode):
    case = cache_case(batch=3, s1=3, seq_lens_k=[900, 5, 333], block_size=block_size, sparse_count=1, sparse_mode=mode,
                      cmp_ratio=cmp_ratio, seed=block_size, extra_pages=1)
    _both(Q, case, 6, 2, 64, e2m1=False, complete=complete)
    _both(Q, case, 6, 2, 64, complete=complete, window=50, sinks=7)


@pytest.mark.parametrize("window", [1, 15, 16, 17, 31, 33, 64, 100, 500, 2000])
@pytest.mark.parametrize("sinks", [0, 1, 16, 33, 500, 3000])
def test_windows(Q, window, sinks):
    case = cache_case(layout_q="TND", q_lens=[70, 1, 9], seq_lens_k=[411, 700, 9], block_size=48, sparse_count=1, sparse_mode=3,
                      seed=window)
    _both(Q, case, 8, 2, 128, window=window, sinks=sinks)


@pytest.mark.parametrize("window", [699, 700, 701, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 2 ** 31 - 1])
def test_windows_as_long_as_the_sequences(Q, window, sinks):
    case = cache_case(layout_q="TND", q_lens=[40, 3, 1], seq_lens_k=[700, 2, 130], block_size=16, sparse_count=1, sparse_mode=3, seed=6)
    _both(Q, case, 8, 2, 64, window=window, sinks=sinks)


def _check_finite(Q, case, q, pool, e2m1, f16, scale=0.0):
    """Rows and heads whose queries hold NaN or infinities are NaN, the others as if those were zeros."""
    bad = ~np.isfinite(q).all(-1)
    out, lse, bits = attend(Q, case, q, pool, 2, e2m1, f16, scale=scale)
    assert np.isnan(out[bad]).all() and np.isnan(lse[bad]).all()
    clean = np.where(bad[..., None], np.float32(0), q)
    want = attend(Q, case, clean, pool, 2, e2m1, f16, scale=scale)
    out[bad], lse[bad] = want[0][bad], want[1][bad]
    check(case, (out, lse, bits), clean, pool, 2, e2m1, f16, scale=scale)


@pytest.mark.parametrize("e2m1,f16", [(True, False), (False, True), (True, True), (False, False)])
def test_queries_of_no_numbers(Q, e2m1, f16):
    case = cache_case(layout_q="TND", q_lens=[40, 3], seq_lens_k=[300, 77], block_size=32, sparse_count=1, sparse_mode=3, seed=7)
    pool, q = cache(case, 2, 64, e2m1, 1), queries(case.rows, 8, 64, f16, 2)
    q[1] = 0
    q[5, 3, 7], q[9, 2], q[41, 0, 0], q[39, 6, 63] = np.nan, np.inf, -np.inf, np.nan
    _check_finite(Q, case, q, pool, e2m1, f16)


@pytest.mark.parametrize("size,scale", [(1e38, 2e-39), (1e-38, 1e37), (2.0 ** -130, 2.0 ** 120)])
def test_queries_of_any_size(Q, size, scale):
    case = cache_case(layout_q="TND", q_lens=[40, 3], seq_lens_k=[300, 77], block_size=32, sparse_count=1, sparse_mode=3, seed=8)
    pool, q = cache(case, 2, 64, True, 1), round_to(queries(case.rows, 8, 64, False, 2) * np.float64(size), False)
    _check_finite(Q, case, q, pool, True, False, scale=scale)            # (a few of the largest are infinite)


@pytest.mark.parametrize("q_lens,lens", [([1, 1, 1], [40, 1, 600]), ([5, 0, 3, 0, 0, 17], [5, 3, 900, 0, 7, 17]),
                                         ([0, 0], [0, 5]), ([33, 200], [33, 1000]), ([7], [3])])
@pytest.mark.parametrize("spare", [0, 1, 40])
def test_chunks_and_rows_behind(Q, q_lens, lens, spare):
    case = cache_case(layout_q="TND", q_lens=q_lens, seq_lens_k=lens, block_size=16, sparse_count=1, sparse_mode=3, seed=3)
    case.total_q += spare
    if case.rows == 0:
        pytest.skip("no rows")
    _both(Q, case, 14, 2, 128)
    _both(Q, case, 4, 4, 64, f16=True, window=20, sinks=2)


def test_fewer_tokens_than_rows(Q):
    case = cache_case(batch=4, s1=6, q_lens=[6, 0, 3, 1], seq_lens_k=[50, 40, 2, 0], block_size=16, sparse_count=1,
                      sparse_mode=3, seed=2)
    _both(Q, case, 16, 2, 128)


@pytest.mark.parametrize("e2m1", [True, False])
@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
def test_factors_strides_and_scales(Q, e2m1, f16, dim):
    case = cache_case(batch=3, s1=1, seq_lens_k=[300, 17, 90], block_size=32, sparse_count=1, sparse_mode=3, seed=4)
    page = 32 * A.entry_bytes(3, dim)
    _both(Q, case, 9, 3, dim, e2m1, f16, factors=(0.3, 5.0), kv_stride=page + 80, q_pad=2)
    _both(Q, case, 9, 3, dim, e2m1, f16, scale=2.0)                           # sharp: most weight on one position
    _both(Q, case, 9, 3, dim, e2m1, f16, scale=1e-30)                         # flat


@pytest.mark.parametrize("batch,lens", [(1, 20000), (5, 9000), (70, 400)])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 1, 128), (16, 8, 128), (8, 4, 64)])
def test_long_and_many(Q, batch, lens, hq, hkv, dim):
    rng = np.random.default_rng(batch)
    case = cache_case(batch=batch, s1=1, seq_lens_k=rng.integers(lens // 2, lens, batch).tolist(), block_size=64,
                      sparse_count=1, sparse_mode=3, seed=5)
    _both(Q, case, hq, hkv, dim)


@pytest.mark.parametrize("q_lens,lens", [([300], [2000]), ([33, 129, 1], [1300, 129, 700]), ([64], [4001])])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 1, 128), (4, 2, 64), (3, 3, 128), (32, 1, 64), (12, 1, 128)])
@pytest.mark.parametrize("e2m1,f16", [(True, False), (False, False), (True, True)])
def test_chunks_over_many_tiles(Q, q_lens, lens, hq, hkv, dim, e2m1, f16):
    case = cache_case(layout_q="TND", q_lens=q_lens, seq_lens_k=lens, block_size=64, sparse_count=1, sparse_mode=3, seed=dim)
    _both(Q, case, hq, hkv, dim, e2m1, f16)
    if e2m1:
        _both(Q, case, hq, hkv, dim, e2m1, f16, window=333, sinks=20)


def test_growing_logits(Q):
    """Each position's logit above the last one's: the maximum rises at every step."""
    case = cache_case(batch=1, s1=1, seq_lens_k=[1500], block_size=64, sparse_count=1, sparse_mode=3, seed=6, permute=False)
    hkv, dim = 2, 128
    rng = np.random.default_rng(0)
    n = case.num_blocks * case.block_size
    base = rng.normal(size=(1, hkv, dim))
    k = base * np.linspace(0.05, 6, n)[:, None, None]
    pool = A.encode(k.astype(np.float32), rng.normal(size=(n, hkv, dim)).astype(np.float32), True).reshape(case.num_blocks, 64, -1)
    q = np.repeat(base, 4, 1).astype(np.float32)
    q = (np.ascontiguousarray(q).view(np.uint32) & 0xFFFF0000).view(np.float32)
    for tokens in (1, 20):
        case.s1 = tokens
        many = np.repeat(q, tokens, 0)
        for sign in (1, -1):
            check(case, attend(Q, case, sign * many, pool, hkv, True, False), sign * many, pool, hkv, True, False)


@pytest.mark.parametrize("window,sinks", [(0, 0), (64, 5)])
def test_bad_lengths_and_pages(Q, window, sinks):
    case = cache_case(batch=4, s1=2, q_lens=[2, 3, 1, 2], seq_lens_k=[200, 100, 500, 90], block_size=16, sparse_count=1,
                      sparse_mode=3, seed=7)
    case.seq_lens_q[1] = -1                                                   # an invalid sequence
    case.seq_lens_k[3] = 1 << 20
    case.block_table[0, 11] = case.num_blocks                                 # visible pages outside the pool
    case.block_table[2, 30] = -1
    case.block_table[2, 5] = -7                                               # seen without a window only
    _both(Q, case, 8, 2, 128, max_seqlen_k=500, window=window, sinks=sinks)
    _both(Q, case, 8, 8, 64, e2m1=False, max_seqlen_k=500, window=window, sinks=sinks)


@pytest.mark.parametrize("cum", [[3, 2, 8], [-1, 2, 8], [3, 5, 9]])
def test_bad_prefix_sums(Q, cum):
    case = cache_case(layout_q="TND", q_lens=[3, 2, 3], seq_lens_k=[30, 20, 50], block_size=16, sparse_count=1, sparse_mode=3,
                      seed=8)
    case.seq_lens_q = np.array(cum, np.int32)
    _both(Q, case, 8, 2, 128)


def test_unseen_pages_are_not_looked_at(Q):
    """A window's cache gives up its middle pages: their table entries are -1, and no error is reported."""
    case = cache_case(batch=2, s1=2, seq_lens_k=[400, 333], block_size=16, sparse_count=1, sparse_mode=3, seed=9)
    case.block_table[:, 2:18] = -1
    pool = cache(case, 2, 128, True, 1)
    q = queries(case.rows, 8, 128, False, 2)
    got = attend(Q, case, q, pool, 2, True, False, window=30, sinks=20)
    assert got[2] == 0
    check(case, got, q, pool, 2, True, False, window=30, sinks=20)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("values", [False, True])
def test_nan_scales(Q, dim, window, sinks, values):
    """What lies beyond the rows' positions may hold NaN scales; a NaN that a row sees is its and no other row's."""
    hkv, hq = 2, 8
    case = cache_case(batch=2, s1=4, seq_lens_k=[203, 77], block_size=16, sparse_count=1, sparse_mode=3, seed=10, permute=False)
    pool = cache(case, hkv, dim, True, 3)
    q = queries(case.rows, hq, dim, False, 4)
    unit = A.unit_bytes(dim)
    used = np.zeros(case.num_blocks * case.block_size, bool)
    for b, n in enumerate(case.seq_lens_k):
        for j in range(n):
            used[case.block_table[b, j // 16] * 16 + j % 16] = True
    flat = pool.reshape(-1, pool.shape[-1])
    for h in range(hkv):
        flat[~used, h * unit + dim:(h + 1) * unit] = 0x7F
    check(case, attend(Q, case, q, pool, hkv, True, False, window=window, sinks=sinks), q, pool, hkv, True, False, window=window,
          sinks=sinks)
    # position 201 of sequence 0: seen by its last two tokens, in KV head 1 alone
    clean = attend(Q, case, q, pool, hkv, True, False, window=window, sinks=sinks)
    at = case.block_table[0, 201 // 16] * 16 + 201 % 16
    flat[at, unit + dim + (dim // 16 if values else 0) + 1] = 0xFF
    out, lse, bits = attend(Q, case, q, pool, hkv, True, False, window=window, sinks=sinks)
    hit = np.zeros((case.rows, hq), bool)
    hit[2:4, hq // 2:] = True
    assert bits == 0 and np.isnan(out).any(-1)[hit].all()
    assert np.array_equal(out[~hit], clean[0][~hit]) and np.array_equal(lse[~hit], clean[1][~hit])


def test_own_stream_and_graph(Q):
    import torch
    case = cache_case(batch=3, s1=2, seq_lens_k=[300, 41, 900], block_size=64, sparse_count=1, sparse_mode=3, seed=11)
    pool, q = cache(case, 2, 128, True, 1), queries(case.rows, 16, 128, False, 2)
    want = attend(Q, case, q, pool, 2, True, False)[0]
    p, a = settings(Q, case, 16, 2, 128, True, False)
    args = (dev(case.seq_lens_q), dev(case.seq_lens_k), dev(case.block_table), dev(pool))
    qd = dev(q, False)
    out = torch.empty_like(qd)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        Q.check(Q.paged_attention(p, a, qd, *args, out))
    for sign in (1, -1):                                                      # the graph reads what is there when it runs
        out.fill_(9)
        qd.copy_(dev(sign * q, False))
        graph.replay()
        torch.cuda.synchronize()
        ref = want if sign == 1 else attend(Q, case, -q, pool, 2, True, False)[0]
        assert np.array_equal(out.double().cpu().numpy(), ref)
    out2 = torch.empty_like(qd)
    torch.cuda.synchronize()
    Q.check(Q.paged_attention(p, a, qd, *args, out2, stream=side))
    side.synchronize()
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))


def test_far_pool_offsets(Q):
    """Pages whose byte offsets pass 32 bits."""
    import torch
    hkv, dim, bs = 64, 128, 1024
    entry = A.entry_bytes(hkv, dim)                                            # 9216 bytes: 9.4 MB a page
    blocks = 600
    case = cache_case(batch=1, s1=1, seq_lens_k=[2500], block_size=bs, sparse_count=1, sparse_mode=3, seed=12)
    small = cache(case, hkv, dim, True, 1)
    pool = torch.zeros((blocks, bs, entry), dtype=torch.uint8, device="cuda")
    far = [599, 470, 17][:case.max_blocks_per_seq]
    for i, page in enumerate(far):
        pool[page] = dev(small[case.block_table[0, i]])
    q = queries(1, 64, dim, False, 2)
    p, a = settings(Q, case, 64, hkv, dim, True, False)
    p.num_blocks = blocks
    out = torch.empty(1, 64, dim, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 64, dtype=torch.float32, device="cuda")
    table = dev(np.array([far], np.int32))
    Q.check(Q.paged_attention(p, a, dev(q, False), None, dev(case.seq_lens_k), table, pool, out, lse))
    check(case, (out.double().cpu().numpy(), lse.double().cpu().numpy(), 0), q, small, hkv, True, False)
