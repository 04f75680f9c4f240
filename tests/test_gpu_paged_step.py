"""A dense layer's step as it is used: new tokens appended, then their attention over the cache, first a prompt in
chunks and then tokens one at a time, captured and replayed; against the 64-bit oracle on the cache as it then is (needs
a GB300)."""
import numpy as np
import pytest

from attention_tools import cache_case, table
from oracle import attention as A
from paged_tools import check, dev, round_to, settings

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


@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
@pytest.mark.parametrize("e2m1,f16", [(True, False), (False, True)])
def test_prompt_in_chunks_then_tokens(Q, window, sinks, e2m1, f16):
    import torch
    hq, hkv, dim, chunks = 8, 2, 128, [70, 33, 1, 1, 1]
    batch, longest = 2, sum(chunks)
    rng = np.random.default_rng(1)
    case = cache_case(batch=batch, s1=1, seq_lens_k=[longest] * batch, block_size=16, sparse_count=1, sparse_mode=3, seed=1)
    r = Q.make_norm_rope(num_heads_q=hq, num_heads_k=hkv, head_dim=dim, rotary_dim=dim, max_positions=longest,
                         dtype=Q.ACT_F16 if f16 else Q.ACT_BF16)
    w = dev(round_to(1 + 0.2 * rng.normal(size=dim), f16), f16)
    cos_sin, bt = dev(table(longest, dim)), dev(case.block_table)
    pool = torch.full((case.num_blocks, 16, A.entry_bytes(hkv, dim)), 0x7F, dtype=torch.uint8, device="cuda")     # NaN scales
    ws = torch.zeros(64, dtype=torch.int32, device="cuda")
    done = 0
    for n in chunks:
        case.s1, case.seq_lens_k = n, np.full(batch, done + n, np.int32)
        p, a = settings(Q, case, hq, hkv, dim, e2m1, f16, max_seqlen_k=longest)
        qkv = dev(round_to(rng.normal(size=(batch * n, hq + 2 * hkv, dim)), f16), f16)
        tb = dev(np.repeat(np.arange(batch), n).astype(np.int32))
        tp = dev(np.tile(np.arange(done, done + n), batch).astype(np.int32))
        q, out = (torch.zeros(batch * n, hq, dim, dtype=qkv.dtype, device="cuda") for _ in range(2))
        lse = torch.zeros(batch * n, hq, device="cuda")
        lens = dev(case.seq_lens_k)

        def step():
            Q.check(Q.kv_append(p, a, r, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], w, w, tp, cos_sin, tb, tp, bt, q, pool, ws))
            Q.check(Q.paged_attention(p, a, q, None, lens, bt, pool, out, lse, ws, window=window, sinks=sinks))

        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            step()
        graph.replay()
        torch.cuda.synchronize()
        got = (out.double().cpu().numpy(), lse.double().cpu().numpy(), Q.get_device_error(ws)[1])
        check(case, got, q.float().cpu().numpy(), pool.cpu().numpy(), hkv, e2m1, f16, window=window, sinks=sinks,
              max_seqlen_k=longest)
        done += n


def test_two_streams_at_once(Q):
    """Calls on two streams of one device share nothing."""
    import torch
    from attention_tools import cache
    from paged_tools import attend, queries
    case = cache_case(batch=3, s1=40, seq_lens_k=[3000, 900, 1700], block_size=64, sparse_count=1, sparse_mode=3, seed=2)
    pool = cache(case, 8, 64, True, 1)
    q = [queries(case.rows, 32, 64, False, s) for s in (2, 3)]
    want = [attend(Q, case, x, pool, 8, True, False)[0] for x in q]
    p, a = settings(Q, case, 32, 8, 64, True, False)
    args = (None, dev(case.seq_lens_k), dev(case.block_table), dev(pool))
    qd = [dev(x, False) for x in q]
    out = [[torch.zeros_like(qd[0]) for _ in range(10)] for _ in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for i in range(10):
        for s, x, o in zip(streams, qd, out):
            Q.check(Q.paged_attention(p, a, x, *args, o[i], stream=s))
    torch.cuda.synchronize()
    for o, ref in zip(out, want):
        assert all(np.array_equal(x.double().cpu().numpy(), ref) for x in o)


def test_no_sequences(Q):
    """Rows without any sequence are zero; nothing else is looked at."""
    import torch
    p = Q.make_problem(batch=0, layout_q=Q.TND, total_q_tokens=5, num_blocks=1, block_size=16, max_blocks_per_seq=1, sparse_count=1,
                       sparse_mode=3, cmp_ratio=1, max_seqlen_q=5, max_seqlen_k=16)
    a = Q.make_attention(num_heads_q=4, num_heads_kv=2, head_dim=64)
    q = torch.ones(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.ones_like(q), torch.ones(5, 4, device="cuda")
    Q.check(Q.paged_attention(p, a, q, None, None, None, None, out, lse))
    assert not out.any() and torch.isneginf(lse).all()
