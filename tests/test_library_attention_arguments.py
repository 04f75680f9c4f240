"""The attention side's binding looks at every tensor before it hands on an address: types, sizes and
contiguity that would be misread, or read or written past their end, are refused (no GPU needed: a
refusal raises before any CUDA call)."""
import pytest

torch = pytest.importorskip("torch")

BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def Q():
    from sparse_attention_token_block_gb300 import build as B
    B.build()
    import sparse_attention_token_block_gb300 as Q
    return Q


def _refuses(call, good, bad):
    """`call` raises for each replacement of one good argument."""
    for name, value, error in bad:
        with pytest.raises(error, match=name):
            call(**dict(good, **{name: value}))


def _every_other(t):
    """The same values at twice the distance."""
    wide = torch.stack([t, t], -1)
    return wide[..., 0]


def test_norm_rope(Q):
    n, d = 3, 128
    r = Q.make_norm_rope(num_heads_q=4, num_heads_k=1, head_dim=d, rotary_dim=64, max_positions=100)
    good = dict(q=torch.zeros(n, 4, d, dtype=BF16), k=torch.zeros(n, 1, d, dtype=BF16), q_weight=torch.zeros(d, dtype=BF16),
                k_weight=torch.zeros(d, dtype=BF16), positions=torch.zeros(n, dtype=I32), cos_sin=torch.zeros(100, 64))
    good.update(q_out=good["q"].clone(), k_out=good["k"].clone())
    bad = [(w, x, e) for w in ("q_weight", "k_weight")
           for x, e in ((torch.zeros(d), TypeError), (torch.zeros(d).half(), TypeError),
                        (torch.zeros(d - 1, dtype=BF16), ValueError), (_every_other(good[w]), ValueError))]
    bad += [("positions", torch.zeros(n, dtype=torch.int64), TypeError), ("positions", _every_other(good["positions"]), ValueError),
            ("cos_sin", torch.zeros(100, 64, dtype=torch.float64), TypeError), ("cos_sin", torch.zeros(100, 64).half(), TypeError),
            ("cos_sin", torch.zeros(99, 64), ValueError), ("cos_sin", torch.zeros(100, 128)[:, :64], ValueError)]
    _refuses(lambda **kw: Q.norm_rope(r, *[kw[x] for x in ("q", "k", "q_weight", "k_weight", "positions", "cos_sin", "q_out",
                                                           "k_out")], stream=0), good, bad)


def _problem(Q, **kw):
    args = dict(batch=2, max_q_tokens=2, num_blocks=8, block_size=64, max_blocks_per_seq=4, sparse_count=64,
                sparse_mode=3, cmp_ratio=1, max_seqlen_q=2, max_seqlen_k=256)
    args.update(kw)
    return Q.make_problem(**args)


def _bad_pools(Q, p, a, stride=0):
    entry = Q.kv_entry_bytes(a)
    page = stride or p.block_size * entry
    u8 = torch.uint8
    short = (p.num_blocks - 1) * page + p.block_size * entry - 1
    bad = [("kv", torch.zeros(short, dtype=u8), ValueError), ("kv", torch.zeros(short + 1, dtype=u8).view(-1, 1).expand(-1, 2), ValueError)]
    wide = torch.zeros(p.num_blocks, page + 16, dtype=u8)
    return bad + [("kv", wide[:, :page], ValueError)]                                 # pages at another distance


@pytest.mark.parametrize("stride", [0, 64 * 288 + 16])
@pytest.mark.parametrize("write", [True, False])
def test_cache(Q, write, stride):
    n = 5
    p, a = _problem(Q), Q.make_attention(num_heads_q=2, num_heads_kv=2, head_dim=128, kv_stride=stride)
    i32 = torch.zeros(n, dtype=I32)
    good = dict(k=torch.zeros(n, 2, 128, dtype=BF16), v=torch.zeros(n, 2, 128, dtype=BF16), token_batch=i32, token_pos=i32,
                block_table=torch.zeros(2, 4, dtype=I32), kv=torch.zeros(8 * (stride or 64 * 288), dtype=torch.uint8))
    bad = [("token_batch", i32.long(), TypeError), ("token_batch", _every_other(i32), ValueError),
           ("token_pos", i32.long(), TypeError), ("token_pos", i32[:4], ValueError), ("token_pos", _every_other(i32), ValueError),
           ("block_table", torch.zeros(2, 4), TypeError), ("block_table", torch.zeros(2, 3, dtype=I32), ValueError),
           ("block_table", torch.zeros(2, 5, dtype=I32)[:, :4], ValueError)] + _bad_pools(Q, p, a, stride)
    order = ("k", "v", "token_batch", "token_pos", "block_table", "kv") if write else (
        "token_batch", "token_pos", "block_table", "kv", "k", "v")
    _refuses(lambda **kw: (Q.kv_write if write else Q.kv_read)(p, a, *[kw[x] for x in order], stream=0), good, bad)


@pytest.mark.parametrize("tnd", [True, False])
def test_sparse_attention(Q, tnd):
    rows = 4
    p = _problem(Q, **(dict(layout_q=Q.TND, max_q_tokens=0, total_q_tokens=rows) if tnd else {}))
    a = Q.make_attention(num_heads_q=4, num_heads_kv=2, head_dim=128)
    good = dict(query=torch.zeros(rows, 4, 128, dtype=BF16), seq_lens_q=torch.zeros(2, dtype=I32),
                seq_lens_k=torch.zeros(2, dtype=I32), block_table=torch.zeros(2, 4, dtype=I32),
                sparse_indices=torch.zeros(rows, 64, dtype=I32), kv=torch.zeros(8, 64, 288, dtype=torch.uint8),
                out=torch.zeros(rows, 4, 128, dtype=BF16), lse=torch.zeros(rows, 4))
    bad = [(x, good[x].long(), TypeError) for x in ("seq_lens_k", "block_table", "sparse_indices")]
    bad += [(x, _every_other(good[x]), ValueError) for x in ("seq_lens_k", "block_table", "sparse_indices", "lse")]
    bad += [(x, good[x].flatten()[:-1], ValueError) for x in ("seq_lens_k", "block_table", "sparse_indices", "lse")]
    bad += [("lse", good["lse"].to(BF16), TypeError), ("lse", good["lse"].double(), TypeError)] + _bad_pools(Q, p, a)
    if tnd:
        bad += [("seq_lens_q", good["seq_lens_q"].long(), TypeError), ("seq_lens_q", good["seq_lens_q"][:1], ValueError)]
    _refuses(lambda **kw: Q.sparse_attention(p, a, *[kw[x] for x in ("query", "seq_lens_q", "seq_lens_k", "block_table",
                                                                     "sparse_indices", "kv", "out", "lse")], stream=0), good, bad)


def test_tensors_that_fit_are_handed_on(Q):
    """Longer buffers, pages a view apart, other byte types, and plain addresses reach the library (which finds
    no device here, or a GPU that runs nothing: no tokens, no rows)."""
    p = _problem(Q, max_q_tokens=0)
    a = Q.make_attention(num_heads_q=4, num_heads_kv=2, head_dim=128, kv_stride=64 * 288 + 32)
    pool = torch.zeros(8, 64 * 288 + 32, dtype=torch.int8)
    none = torch.zeros(0, 4, 128, dtype=BF16)
    table = torch.zeros(3, 4, dtype=I32)
    for kv in (pool, pool[:, :64 * 288], pool.flatten(), 1 << 20):
        assert Q.sparse_attention(p, a, none, None, torch.zeros(9, dtype=I32), table, torch.zeros(0, 64, dtype=I32), kv, none,
                                  torch.zeros(0, 4), stream=0) == 0
        k = torch.zeros(0, 2, 128, dtype=BF16)
        i32 = torch.zeros(0, dtype=I32)
        assert Q.kv_write(p, a, k, k, i32, torch.zeros(7, dtype=I32), table, kv, stream=0) == 0
        assert Q.kv_read(p, a, i32, i32, table, kv, k, k, stream=0) == 0
    r = Q.make_norm_rope(num_heads_q=4, num_heads_k=0, head_dim=128, rotary_dim=0, max_positions=1, norm=False)
    assert Q.norm_rope(r, none, None, None, None, torch.zeros(0, dtype=I32), None, none, None, stream=0) == 0
