"""Refusals of qli_kv_append and qli_paged_attention, and of their binding: all before any CUDA call (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

BF16, I32 = torch.bfloat16, torch.int32
X = 1 << 20                                       # a 256-byte aligned stand-in address, never dereferenced


@pytest.fixture(scope="module")
def Q():
    from sparse_attention_token_block_gb300 import build as B
    B.build()
    import sparse_attention_token_block_gb300 as Q
    return Q


def _problem(Q, **kw):
    args = dict(batch=2, max_q_tokens=2, num_blocks=8, block_size=64, max_blocks_per_seq=4, sparse_count=1,
                sparse_mode=3, cmp_ratio=1, max_seqlen_q=2, max_seqlen_k=256)
    args.update(kw)
    return Q.make_problem(**args)


def _attention(Q, **kw):
    args = dict(num_heads_q=16, num_heads_kv=2, head_dim=128)
    args.update(kw)
    return Q.make_attention(**args)


def _rotation(Q, **kw):
    args = dict(num_heads_q=16, num_heads_k=2, head_dim=128, rotary_dim=64, max_positions=100)
    args.update(kw)
    return Q.make_norm_rope(**args)


PAGED = ["p", "a", "window", "sinks", "query", "q_stride", "seq_lens_q", "seq_lens_k", "block_table", "kv", "out", "lse",
         "workspace", "workspace_bytes", "stream"]
APPEND = ["p", "a", "r", "tokens", "q", "q_stride", "k", "k_stride", "v", "v_stride", "q_weight", "k_weight", "positions",
          "cos_sin", "token_batch", "token_pos", "block_table", "q_out", "q_out_stride", "kv", "workspace", "workspace_bytes",
          "stream"]


def _paged(Q, p=None, a=None, **kw):
    args = dict(p=p or _problem(Q), a=a or _attention(Q), window=0, sinks=0, query=X, q_stride=0, seq_lens_q=None, seq_lens_k=X,
                block_table=X, kv=X, out=X, lse=X, workspace=X, workspace_bytes=256, stream=None)
    args.update(kw)
    return Q.lib.qli_paged_attention(*[args[n] for n in PAGED])


def _append(Q, p=None, a=None, r=None, **kw):
    args = dict(p=p or _problem(Q), a=a or _attention(Q), r=r or _rotation(Q), tokens=3, workspace=X, workspace_bytes=256,
                stream=None, q_stride=0, k_stride=0, v_stride=0, q_out_stride=0)
    args.update({n: X for n in APPEND if n not in args})
    args.update(kw)
    return Q.lib.qli_kv_append(*[args[n] for n in APPEND])


@pytest.mark.parametrize("kw", [
    dict(window=-1), dict(sinks=-1), dict(query=None), dict(query=X + 8), dict(q_stride=15 * 128), dict(q_stride=16 * 128 + 4),
    dict(q_stride=-2048), dict(seq_lens_k=None), dict(block_table=None), dict(kv=None), dict(kv=X + 8), dict(out=None),
    dict(out=X + 8), dict(lse=X + 2), dict(workspace=X + 128), dict(workspace_bytes=255)])
def test_paged_attention_arguments(Q, kw):
    assert _paged(Q, **kw) == 1


def test_paged_attention_attributes(Q):
    assert _paged(Q, p=_problem(Q, block_size=24)) == 1
    assert _paged(Q, p=_problem(Q, max_blocks_per_seq=3)) == 1
    bad = _attention(Q)
    bad.head_dim = 96
    assert _paged(Q, a=bad) == 1
    assert _paged(Q, a=_attention(Q, kv_stride=64 * 288 - 16)) == 1
    tnd = _problem(Q, layout_q=Q.TND, total_q_tokens=4)
    assert _paged(Q, p=tnd) == 1                                            # prefix sums are required
    assert Q.lib.qli_paged_attention(None, _attention(Q), 0, 0, X, 0, None, X, X, X, X, None, None, 0, None) == 1
    assert Q.lib.qli_paged_attention(_problem(Q), None, 0, 0, X, 0, None, X, X, X, X, None, None, 0, None) == 1
    # nothing to do, nothing looked at
    assert _paged(Q, p=_problem(Q, max_q_tokens=0), query=None, out=None, kv=None) == 0
    assert _paged(Q, p=_problem(Q, batch=0), query=None, out=None) == 0
    many = _problem(Q, layout_q=Q.TND, total_q_tokens=1 << 25, max_seqlen_k=1)
    assert _paged(Q, p=many, seq_lens_q=X) == 2
    # positions that tiles would count past 2^31
    far = dict(block_size=1024, max_blocks_per_seq=1 << 21)
    assert _paged(Q, p=_problem(Q, max_seqlen_k=(1 << 31) - 1, **far)) == 2
    assert _paged(Q, p=_problem(Q, max_seqlen_k=(1 << 31) - 1023, **far)) == 2


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(q=None), dict(k=None), dict(v=None), dict(q=X + 8), dict(k=X + 8),
    dict(v=X + 8), dict(q_out=None), dict(q_out=X + 8), dict(q_stride=2040), dict(k_stride=252), dict(v_stride=260),
    dict(q_out_stride=2040), dict(q_weight=None), dict(k_weight=None), dict(k_weight=X + 2), dict(positions=None),
    dict(cos_sin=None), dict(cos_sin=X + 4), dict(token_batch=None), dict(token_pos=None), dict(block_table=None),
    dict(kv=None), dict(kv=X + 8), dict(workspace=X + 64), dict(workspace_bytes=128)])
def test_append_arguments(Q, kw):
    assert _append(Q, **kw) == 1


def test_append_attributes(Q):
    assert _append(Q, r=_rotation(Q, num_heads_k=1)) == 1
    assert _append(Q, r=_rotation(Q, head_dim=64, rotary_dim=64)) == 1
    assert _append(Q, r=_rotation(Q, dtype=Q.ACT_F16)) == 1
    assert _append(Q, r=_rotation(Q, rotary_dim=132)) == 1
    wide = _rotation(Q, head_dim=256)
    assert _append(Q, r=wide) == 1                                           # the cache has no heads of 256
    assert _append(Q, p=_problem(Q, block_size=8)) == 1
    assert _append(Q, tokens=0, q=None, k=None, v=None, q_out=None, kv=None) == 0
    assert Q.lib.qli_kv_append(_problem(Q), _attention(Q), None, 0, *[None, 0] * 3, *[None] * 7, None, 0, None, None, 0, None) == 1


def _refuses(call, good, bad):
    for name, value, error in bad:
        with pytest.raises(error, match=name):
            call(**dict(good, **{name: value}))


def test_binding_of_paged_attention(Q):
    p, a = _problem(Q), _attention(Q)
    good = dict(query=torch.zeros(4, 16, 128, dtype=BF16), seq_lens_q=None, seq_lens_k=torch.zeros(2, dtype=I32),
                block_table=torch.zeros(2, 4, dtype=I32), kv=torch.zeros(8 * 64 * 288, dtype=torch.uint8),
                out=torch.zeros(4, 16, 128, dtype=BF16), lse=torch.zeros(4, 16))
    call = lambda **kw: Q.paged_attention(p, a, *[kw[n] for n in good], stream=0)  # noqa: E731
    _refuses(call, good, [
        ("query", good["query"].half(), TypeError), ("query", torch.zeros(4, 16, 64, dtype=BF16), ValueError),
        ("query", torch.zeros(4, 32, 128, dtype=BF16)[:, ::2], ValueError), ("out", good["out"][:3], ValueError),
        ("out", torch.zeros(4, 20, 128, dtype=BF16)[:, :16], ValueError), ("seq_lens_q", torch.zeros(2), TypeError),
        ("seq_lens_q", torch.zeros(1, dtype=I32), ValueError), ("seq_lens_k", torch.zeros(1, dtype=I32), ValueError),
        ("seq_lens_k", torch.zeros(2, dtype=torch.int64), TypeError), ("block_table", torch.zeros(2, 3, dtype=I32), ValueError),
        ("kv", good["kv"][:-1], ValueError), ("lse", torch.zeros(4, 16).half(), TypeError), ("lse", torch.zeros(4, 15), ValueError)])


@pytest.mark.parametrize("window, sinks", [(1 << 32, 0), ((1 << 31), 4), (16, 1 << 32), (-(1 << 31) - 1, 0)])
def test_binding_keeps_the_whole_window(Q, window, sinks):
    q = torch.zeros(4, 16, 128, dtype=BF16)
    with pytest.raises(ValueError, match="32-bit"):
        Q.paged_attention(_problem(Q), _attention(Q), q, None, torch.zeros(2, dtype=I32), torch.zeros(2, 4, dtype=I32),
                          torch.zeros(8 * 64 * 288, dtype=torch.uint8), q.clone(), window=window, sinks=sinks, stream=0)


def test_binding_of_append(Q):
    p, a, r = _problem(Q), _attention(Q), _rotation(Q)
    n = 3
    good = dict(q=torch.zeros(n, 16, 128, dtype=BF16), k=torch.zeros(n, 2, 128, dtype=BF16), v=torch.zeros(n, 2, 128, dtype=BF16),
                q_weight=torch.zeros(128, dtype=BF16), k_weight=torch.zeros(128, dtype=BF16), positions=torch.zeros(n, dtype=I32),
                cos_sin=torch.zeros(100, 64), token_batch=torch.zeros(n, dtype=I32), token_pos=torch.zeros(n, dtype=I32),
                block_table=torch.zeros(2, 4, dtype=I32), q_out=torch.zeros(n, 16, 128, dtype=BF16),
                kv=torch.zeros(8 * 64 * 288, dtype=torch.uint8))
    call = lambda **kw: Q.kv_append(p, a, r, *[kw[x] for x in good], stream=0)  # noqa: E731
    _refuses(call, good, [
        ("q", good["q"].float(), TypeError), ("k", good["k"][:, :1], ValueError), ("v", good["v"].half(), TypeError),
        ("v", torch.zeros(n, 2, 256, dtype=BF16)[..., ::2], ValueError), ("q_weight", torch.zeros(128), TypeError),
        ("k_weight", torch.zeros(64, dtype=BF16), ValueError), ("positions", torch.zeros(2, dtype=I32), ValueError),
        ("cos_sin", torch.zeros(99, 64), ValueError), ("token_batch", torch.zeros(n, dtype=torch.int64), TypeError),
        ("token_pos", torch.zeros(2, dtype=I32), ValueError), ("block_table", torch.zeros(7, dtype=I32), ValueError),
        ("q_out", good["q_out"][:2], ValueError), ("kv", good["kv"][1:], ValueError)])


def test_binding_wants_one_device(Q, monkeypatch):
    """Tensors that are not on the current device are refused (host tensors here)."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    p, a = _problem(Q), _attention(Q)
    q = torch.zeros(4, 16, 128, dtype=BF16)
    with pytest.raises(ValueError, match="current device"):
        Q.paged_attention(p, a, q, None, torch.zeros(2, dtype=I32), torch.zeros(2, 4, dtype=I32),
                          torch.zeros(8 * 64 * 288, dtype=torch.uint8), q.clone(), stream=0)
