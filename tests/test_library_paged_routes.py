"""Which qli_paged_attention calls go to the kernel of many rows: the host's rule (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def route():
    from sparse_attention_token_block_gb300 import build as B
    B.build()
    import sparse_attention_token_block_gb300 as Q
    f = ctypes.CDLL(Q.TESTING_LIB_PATH).qli_testing_paged_chunks

    def call(batch, s1, positions, hq=64, hkv=8, dim=128, window=0, sinks=0, tnd=0, **kw):
        layout = dict(layout_q=Q.TND, total_q_tokens=tnd) if tnd else dict(max_q_tokens=s1)
        p = Q.make_problem(batch=batch, num_blocks=batch * -(-positions // 16), block_size=16, max_blocks_per_seq=-(-positions // 16),
                           sparse_count=1, sparse_mode=3, cmp_ratio=1, max_seqlen_q=s1, max_seqlen_k=positions, **layout, **kw)
        a = Q.make_attention(num_heads_q=hq, num_heads_kv=hkv, head_dim=dim)
        return f(ctypes.byref(p), ctypes.byref(a), window, sinks)
    return call


def test_by_what_both_cost(route):
    assert route(32, 1, 32768) == 0 and route(32, 2, 131072) == 0          # up to 16 rows read a KV head
    assert route(32, 4, 16384) == 1 and route(4, 8, 16384, hq=32) == 1
    assert route(24, 8, 512, hq=32) == 0 and route(24, 16, 512, hq=32) == 1
    assert route(4, 32, 512, hq=32) == 0
    assert route(1, 1, 100000, hq=128, hkv=1) == 1                          # one token of a wide group
    assert route(4, 8192, 8192, tnd=15360) == 1
    assert route(4, 8192, 8192, tnd=15360, window=1024, sinks=16) == 1
    assert route(3, 331, 2000, hq=15, hkv=5, dim=64, tnd=409, window=129, sinks=1) == 0


def test_refusals(route):
    assert route(2, 4, 512, window=-1) == -1 and route(2, 4, 512, sinks=-1) == -1 and route(2, 4, 512, hq=63) == -1
    assert route(0, 5, 16, tnd=5) == -1                                     # a pool has at least one page

