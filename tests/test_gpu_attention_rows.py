"""Sparse attention of many neighbouring rows, whose lists become masks over shared tiles of keys
(calls of lists of at least 512, at least as many blocks of rows as fill the GPU), against the 64-bit oracle (needs a GB300)."""
import os
import subprocess
import sys

import numpy as np
import pytest

import workloads as W
from attention_tools import cache, cache_case
from oracle import attention as A
from test_gpu_sparse_attention import Q, _check, _dev, _query, _run  # noqa: F401 (Q is a fixture)

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _ragged(q_lens, k_lens, **kw):
    return cache_case(layout_q="TND", q_lens=q_lens, seq_lens_k=k_lens, **kw)


def _wide(case, idx, seed=0, k=512):
    """The lists spread over k places of which the others are -1."""
    if idx.shape[1] >= k:
        return idx
    place = np.sort(np.random.default_rng(seed).permutation(k)[:idx.shape[1]])
    wide = np.full((idx.shape[0], k), -1, np.int32)
    wide[:, place] = idx
    case.sparse_count = k
    return wide


# query heads, KV heads, rows that give at least 152 blocks of rows and KV heads
@pytest.mark.parametrize("hq,hkv,q_lens", [(64, 8, [300, 17, 5]), (16, 16, [200, 130]), (40, 8, [333, 150]), (7, 1, [2738]),
                                           (32, 1, [640]), (10, 5, [993, 1]), (96, 32, [150, 118]),
                                           (33, 1, [470]), (64, 1, [310]), (128, 1, [160])])
@pytest.mark.parametrize("e2m1,f16", [(True, False), (False, True)])
def test_head_layouts(Q, hq, hkv, q_lens, e2m1, f16):
    rows = sum(q_lens)
    case = _ragged(q_lens, [257, 130, 70][:len(q_lens)], block_size=48, sparse_count=90, seed=hq)
    pool = cache(case, hkv, 128, e2m1, seed=1)
    idx = _wide(case, W.random_indices(case, seed=2))
    q = _query(rows, hq, 128, f16, 3)
    _check(case, _run(Q, case, q, idx, pool, hkv, e2m1, f16, q_pad=1), q, idx, pool, hkv, e2m1, f16)


@pytest.mark.parametrize("k,keys", [(1, 4), (33, 129), (64, 64), (500, 2000), (2048, 2300)])
def test_list_lengths(Q, k, keys):
    """One position, lists of all positions, an odd key past a tile, many tiles."""
    case = _ragged([330], [keys], block_size=16, sparse_count=k, seed=k)
    pool = cache(case, 16, 128, True, seed=1)
    idx = _wide(case, W.random_indices(case, seed=2, frac_pad=0.0))
    q = _query(330, 32, 128, False, 3)
    _check(case, _run(Q, case, q, idx, pool, 16, True, False), q, idx, pool, 16, True, False)


@pytest.mark.parametrize("with_k", [True, False])
def test_compressed_factors_and_page_gaps(Q, with_k):
    case = _ragged([301, 0, 250, 3], [801, 60, 333, 3], block_size=32, sparse_count=70, cmp_ratio=4, seed=7)
    hkv, factors = 8, (0.7, 3.0)
    pool = cache(case, hkv, 128, True, 1, *factors)
    eb = pool.shape[2]
    gap = np.random.default_rng(4).integers(0, 256, (case.num_blocks, 32 * eb + 32), dtype=np.uint8)
    gap[:, :32 * eb] = pool.reshape(case.num_blocks, -1)
    idx = _wide(case, W.random_indices(case, seed=2))
    q = _query(554, 64, 128, False, 3)
    got = _run(Q, case, q, idx, gap, hkv, True, False, 0.11, factors, 32 * eb + 32, with_k=with_k)
    _check(case, got, q, idx, pool, hkv, True, False, 0.11, factors, with_k=with_k)


def test_padding_duplicates_and_empty_rows(Q):
    rng = np.random.default_rng(8)
    case = _ragged([320], [400], block_size=16, sparse_count=300, seed=8)
    pool = cache(case, 8, 128, True, seed=1)
    idx = W.random_indices(case, seed=2, frac_pad=0.0)
    idx[0, rng.random(300) < 0.5] = -1
    idx[1, :] = -1
    idx[2, :299] = -1                                        # only the last
    idx[3, 1:] = -1                                          # only the first
    idx[5, :] = 17                                           # one entry 300 times
    idx[6, ::2] = 399
    idx[32:48] = -1                                          # a block of nothing
    idx[48:64, 1:] = -1                                      # one entry a row
    idx[64:80] = np.sort(idx[64:80], axis=1)
    idx = _wide(case, idx)
    q = _query(320, 64, 128, False, 3)
    _check(case, _run(Q, case, q, idx, pool, 8, True, False), q, idx, pool, 8, True, False)


def test_unlisted_bytes_and_other_rows_nan_are_never_used(Q):
    """Slots that no list names hold scale bytes of NaN; so does one that a single row lists: that row is NaN,
    the others of its block are not."""
    case = _ragged([320], [190], block_size=32, sparse_count=60, seed=9)
    pool = cache(case, 8, 128, True, seed=1)
    idx = W.random_indices(case, seed=2)
    idx[idx == 150] = -1                                     # listed by one row only
    idx[21, 0] = 150
    idx = _wide(case, idx)
    used = np.zeros(pool.shape[:2], bool)
    j = idx[idx >= 0]
    used[case.block_table[0, j // 32], j % 32] = True
    poisoned = np.where(used[..., None], pool, np.uint8(0x7F))
    q = _query(320, 64, 128, False, 3)
    _check(case, _run(Q, case, q, idx, poisoned, 8, True, False), q, idx, pool, 8, True, False)
    pg, at = case.block_table[0, 150 // 32], 150 % 32
    for byte in (128 + 3, 136 + 5):                          # a key's and a value's scale of the first head
        bad = poisoned.copy()
        bad[pg, at, byte] = 0xFF
        out, lse, bits = _run(Q, case, q, idx, bad, 8, True, False)
        assert bits == 0 and np.isnan(out[21, :8]).any(-1).all()
        ref = idx.copy()
        ref[21] = -1
        out[21], lse[21] = 0, -np.inf
        _check(case, (out, lse, 0), q, ref, pool, 8, True, False)


@pytest.mark.parametrize("order", ["rising", "falling", "spike"])
def test_large_logits(Q, order):
    n, rows = 700, 304
    case = _ragged([rows], [n], block_size=64, sparse_count=n, seed=3)
    rng = np.random.default_rng(1)
    size = {"rising": np.linspace(0.1, 6, n), "falling": np.linspace(6, 0.1, n), "spike": np.full(n, 0.2)}[order]
    if order == "spike":
        size[333] = 6.0
    base = rng.choice([-1.0, 1.0], 128)
    j = np.arange(n)
    slot = case.block_table[0, j // 64] * 64 + j % 64
    k = np.zeros((case.num_blocks * 64, 8, 128), np.float32)
    k[slot] = size[:, None, None] * base
    v = rng.normal(size=k.shape).astype(np.float32)
    pool = A.encode(k, v, True).reshape(case.num_blocks, 64, -1)
    q = np.zeros((rows, 64, 128), np.float32)
    q[:] = np.resize([8.0, -8.0, 0.01, 1.0, 0.0], (rows, 64))[..., None] * base
    q[:] = np.float32(np.float16(q))
    idx = np.stack([rng.permutation(n) for _ in range(rows)]).astype(np.int32)
    _check(case, _run(Q, case, q, idx, pool, 8, True, True), q, idx, pool, 8, True, True)


def test_query_magnitudes(Q):
    case = _ragged([304], [200], block_size=16, sparse_count=128, seed=3)
    pool = cache(case, 8, 128, False, seed=1)
    q = _query(304, 64, 128, False, 3)
    q *= np.resize(np.array([1, 1e-6, 1e-30, 1e3, 0, 1e-3, 2.0 ** -100], np.float32), (304, 64))[..., None]
    q = (q.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    idx = _wide(case, W.random_indices(case, seed=2))
    _check(case, _run(Q, case, q, idx, pool, 8, False, False, 0.05), q, idx, pool, 8, False, False, 0.05)


def test_invalid_indices_and_pages(Q):
    case = _ragged([300, 20], [100, 40], block_size=32, sparse_count=28, seed=5)
    pool = cache(case, 8, 128, True, seed=6)
    good = _wide(case, W.random_indices(case, seed=2))
    q = _query(320, 64, 128, False, 3)
    for row, bad in ((7, 100), (7, -5), (319, 40), (0, 2147483647), (5, -2147483648)):
        idx = good.copy()
        idx[row, 3] = bad
        _check(case, _run(Q, case, q, idx, pool, 8, True, False), q, idx, pool, 8, True, False)
    case.block_table[0, 3] = case.num_blocks + 2
    case.block_table[0, 1] = -3
    _check(case, _run(Q, case, q, good, pool, 8, True, False), q, good, pool, 8, True, False)


def test_rows_past_the_last_prefix_sum(Q):
    case = _ragged([200, 90], [64, 64], block_size=32, sparse_count=20, seed=7)
    case.total_q = 310
    pool = cache(case, 8, 128, True, seed=8)
    idx = np.full((310, 20), -1, np.int32)
    idx[:, 0], idx[:, 9] = 1, 60
    idx[300] = -1
    idx = _wide(case, idx)
    q = _query(310, 64, 128, False, 3)
    _check(case, _run(Q, case, q, idx, pool, 8, True, False), q, idx, pool, 8, True, False)


def test_a_length_above_its_bound(Q):
    """seq_lens_k larger than max_seqlen_k promises (the table holds them): the masks, made for the bound, are
    filled once per range of positions; some positions are listed twice."""
    case = _ragged([304], [600], block_size=64, sparse_count=150, seed=4)
    pool = cache(case, 8, 128, True, seed=1)
    idx = _wide(case, W.random_indices(case, seed=2))
    idx[9, 200:400] = idx[9, :200]
    q = _query(304, 64, 128, False, 3)
    kw = dict(W.problem_kwargs(case))
    p = Q.make_problem(**dict(kw, max_seqlen_k=200))
    a = Q.make_attention(num_heads_q=64, num_heads_kv=8, head_dim=128)
    import torch
    out = torch.empty(304, 64, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(304, 64, device="cuda")
    Q.check(Q.sparse_attention(p, a, _dev(q, False), _dev(case.seq_lens_q), _dev(case.seq_lens_k), _dev(case.block_table),
                               _dev(idx), _dev(pool), out, lse), "sparse_attention")
    _check(case, (out.double().cpu().numpy(), lse.double().cpu().numpy(), 0), q, idx, pool, 8, True, False)


def _make(Q, case, **kw):
    return (Q.make_problem(**W.problem_kwargs(case)), Q.make_attention(num_heads_q=64, num_heads_kv=8, head_dim=128, **kw))


def test_offsets_past_32_bits(Q):
    """Entries on the last pages of a pool of over 4 GB."""
    import torch
    bs, nb, rows = 1024, 20, 304
    page = bs * 1152 + (1 << 28)
    case = _ragged([rows], [2 * bs], block_size=bs, sparse_count=512, seed=1)
    case.num_blocks = nb
    case.block_table = np.array([[nb - 1, nb - 2]], np.int32)
    small = cache(case, 8, 128, True, seed=1)
    pool = torch.zeros(nb * page, dtype=torch.uint8, device="cuda")
    for pg in (nb - 1, nb - 2):
        pool[pg * page:pg * page + bs * 1152] = _dev(small[pg].reshape(-1))
    idx = W.random_indices(case, seed=2)
    q = _query(rows, 64, 128, False, 3)
    p, a = _make(Q, case, kv_stride=page)
    out = torch.empty(rows, 64, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(rows, 64, device="cuda")
    Q.check(Q.sparse_attention(p, a, _dev(q, False), _dev(case.seq_lens_q), _dev(case.seq_lens_k), _dev(case.block_table),
                               _dev(idx), pool, out, lse), "sparse_attention")
    _check(case, (out.double().cpu().numpy(), lse.double().cpu().numpy(), 0), q, idx, small, 8, True, False)


def test_runs_on_its_stream_and_in_a_graph(Q):
    """Captured on a stream of its own, twice in a row, and replayed on new queries, lists and contents."""
    import torch
    rows = 304
    case = _ragged([rows], [300], block_size=16, sparse_count=512, seed=2)
    p, a = _make(Q, case)
    pool = torch.zeros(cache(case, 8, 128, True, seed=1).shape, dtype=torch.uint8, device="cuda")
    q = torch.zeros(rows, 64, 128, dtype=torch.bfloat16, device="cuda")
    idx = torch.full((rows, 512), -1, dtype=torch.int32, device="cuda")
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty(rows, 64, device="cuda")
    args = (_dev(case.seq_lens_q), _dev(case.seq_lens_k), _dev(case.block_table))
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            Q.check(Q.sparse_attention(p, a, q, *args, idx, pool, out, lse), "sparse_attention")
            Q.check(Q.sparse_attention(p, a, q, *args, idx, pool, out2), "sparse_attention")
    for seed in (1, 2):
        hp, hq, hi = cache(case, 8, 128, True, seed), _query(rows, 64, 128, False, seed), W.random_indices(case, seed)
        pool.copy_(_dev(hp))
        q.copy_(_dev(hq, False))
        idx.copy_(_dev(hi))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
        _check(case, (out.double().cpu().numpy(), lse.double().cpu().numpy(), 0), hq, hi, hp, 8, True, False)


CHILD = r"""
import sys
sys.path.insert(0, %r)
import torch
import sparse_attention_token_block_gb300 as Q
Q.use_testing_library()
Q.lib.qli_testing_set_stall(%d)
rows = 304
p = Q.make_problem(batch=1, max_q_tokens=rows, num_blocks=4, block_size=64, max_blocks_per_seq=4, sparse_count=512,
                   sparse_mode=0, cmp_ratio=1, max_seqlen_q=rows, max_seqlen_k=256)
a = Q.make_attention(num_heads_q=64, num_heads_kv=8, head_dim=128)
dev = dict(device="cuda")
pool = torch.zeros(4, 64, Q.kv_entry_bytes(a), dtype=torch.uint8, **dev)
q = torch.ones(rows, 64, 128, dtype=torch.bfloat16, **dev)
out = torch.ones_like(q)
table = torch.arange(4, dtype=torch.int32, **dev)[None]
idx = torch.full((rows, 512), -1, dtype=torch.int32, **dev)
idx[:, :64] = torch.arange(64, dtype=torch.int32, **dev)
lens = torch.full((1,), 256, dtype=torch.int32, **dev)
ws = torch.zeros(64, dtype=torch.int32, **dev)
Q.check(Q.sparse_attention(p, a, q, None, lens, table, idx, pool, out, None, ws), "sparse_attention")
st, bits = Q.get_device_error(ws)
print("STATUS", st, bits, int(torch.isnan(out.float()).all().item()), int((out == 0).all().item()))
print("AFTER", torch.ones(1024, **dev).sum().item())
"""


@pytest.mark.parametrize("stall", [0, 1])
def test_waits_run_out(Q, stall):
    """With the testing build's stall switch no tile is handed on: every bounded wait runs out, the call reports
    QLI_ERR_DEVICE_TIMEOUT and writes NaN, and the context stays usable."""
    out = subprocess.run([sys.executable, "-c", CHILD % (ROOT, stall)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stderr[-2000:]
    status = [x for x in out.stdout.splitlines() if x.startswith("STATUS")][0].split()[1:]
    assert status == (["6", "4", "1", "0"] if stall else ["0", "0", "0", "1"])
    assert "AFTER 1024.0" in out.stdout
