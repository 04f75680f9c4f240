"""Norm and rotation of queries and keys on the GPU (qli_norm_rope) against the 64-bit oracle (needs a
GB300)."""
import numpy as np
import pytest

from attention_tools import half_step, round_to, smallest_step, table
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
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if f16 is None else t.to(torch.float16 if f16 else torch.bfloat16)


def _check(got, x, w, pos, cs, rot, inter, eps, norm, f16):
    """|got - ref| within: fp32 sums and products (the mean square within (D / 8 + 8) 2^-24, the
    reciprocal root within 2^-22, four roundings, each product of the rotation) and one rounding."""
    ref = A.norm_rope(x, w, pos, cs, rot, inter, eps, norm)
    y = np.abs(A.norm_rope(x, w, np.zeros(len(pos), int), np.eye(1, max(rot, 1)).astype(np.float32), 0, inter, eps, norm))
    pair = y.copy()
    half = rot // 2
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, half), slice(half, rot))
    pair[..., a] += y[..., b]
    pair[..., b] += y[..., a]
    d = x.shape[-1]
    err = (d / 8 + 8 + 16) * 2.0 ** -24 * pair if norm else 4 * 2.0 ** -24 * pair
    if not norm:
        err[..., rot:] = 0
    tol = err + half_step(f16) * (np.abs(ref) + err) + smallest_step(f16)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])


# tokens, query heads, key heads, D, R
SHAPES = [(1, 64, 8, 128, 128), (1, 1, 1, 64, 64), (5, 3, 1, 256, 256), (33, 20, 5, 64, 32), (7, 9, 2, 128, 24),
          (130, 4, 4, 128, 64), (3, 0, 2, 128, 128), (3, 7, 0, 64, 8), (2, 5, 3, 256, 0), (257, 8, 1, 64, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("norm", [True, False])
def test_matches_the_oracle(Q, shape, inter, f16, norm):
    import torch
    t, hq, hk, d, rot = shape
    rng = np.random.default_rng(t * 7 + hq)
    packed = round_to(rng.normal(size=(t, hq + 2 * hk + 1, d)) * np.exp(rng.uniform(-4, 3, (t, hq + 2 * hk + 1, 1))), f16)
    w = [round_to(1 + 0.3 * rng.normal(size=d), f16) for _ in range(2)]
    cs = table(500, rot) if rot else np.zeros((500, 0), np.float32)
    pos = rng.integers(0, 500, t).astype(np.int32)
    x = _dev(packed, f16)
    q, k = x[:, :hq], x[:, hq:hq + hk]
    dt = torch.float16 if f16 else torch.bfloat16
    qo = torch.full((t, hq, d), 7, dtype=dt, device="cuda") if hq else None
    ko = torch.full((t, hk + 1, d), 7, dtype=dt, device="cuda")
    r = Q.make_norm_rope(num_heads_q=hq, num_heads_k=hk, head_dim=d, rotary_dim=rot, max_positions=500,
                         dtype=Q.ACT_F16 if f16 else Q.ACT_BF16, interleaved=inter, norm=norm, eps=1e-5)
    ws = torch.zeros(64, dtype=torch.int32, device="cuda")
    wd = [_dev(v, f16) if norm else None for v in w]
    Q.check(Q.norm_rope(r, q if hq else None, k if hk else None, wd[0], wd[1], _dev(pos), _dev(cs) if rot else None, qo,
                        ko[:, :hk] if hk else None, ws), "norm_rope")
    assert Q.get_device_error(ws) == (0, 0)
    if hq:
        _check(qo.double().cpu().numpy(), packed[:, :hq], w[0], pos, cs, rot, inter, 1e-5, norm, f16)
    if hk:
        _check(ko[:, :hk].double().cpu().numpy(), packed[:, hq:hq + hk], w[1], pos, cs, rot, inter, 1e-5, norm, f16)
    assert (ko[:, hk:] == 7).all()                          # what lies beside a strided output stays
    # in place, on the packed projection itself
    rest = x[:, hq + hk:].clone()
    Q.check(Q.norm_rope(r, q if hq else None, k if hk else None, wd[0], wd[1], _dev(pos), _dev(cs) if rot else None,
                        q if hq else None, k if hk else None, ws), "norm_rope in place")
    assert (hq == 0 or torch.equal(q, qo)) and torch.equal(k, ko[:, :hk]) and torch.equal(x[:, hq + hk:], rest)


# enough tokens that a lane takes several heads at a time
@pytest.mark.parametrize("shape", [(700, 40, 3, 128, 128), (500, 90, 7, 256, 64), (2600, 20, 5, 64, 24)])
@pytest.mark.parametrize("inter", [False, True])
def test_many_tokens(Q, shape, inter):
    test_matches_the_oracle(Q, shape, inter, False, True)


def test_zero_vectors_extreme_magnitudes_and_last_position(Q):
    import torch
    d = 128
    rows = np.zeros((4, 1, d), np.float32)
    rows[1] = 1e-18                                          # the mean square underflows beside eps
    rows[2] = round_to(np.full((1, d), 1e18), False)
    rows[3] = round_to(np.random.default_rng(0).normal(size=(1, d)), False)
    w = np.ones(d, np.float32)
    cs, pos = table(131072, d), np.array([0, 1, 131071, 131071], np.int32)
    r = Q.make_norm_rope(num_heads_q=1, num_heads_k=0, head_dim=d, rotary_dim=d, max_positions=131072)
    q = _dev(rows, False)
    out = torch.empty_like(q)
    Q.check(Q.norm_rope(r, q, None, _dev(w, False), None, _dev(pos), _dev(cs), out, None), "norm_rope")
    # the oracle takes the values that the tensor holds (1e-18 is not a bfloat16)
    _check(out.double().cpu().numpy(), q.float().cpu().numpy(), w, pos, cs, d, False, 1e-6, True, False)
    assert not out[0].any()


def test_bad_positions_write_zeros_and_set_the_bit(Q):
    import torch
    rng = np.random.default_rng(5)
    x = round_to(rng.normal(size=(6, 3, 64)), False)
    pos = np.array([0, -1, 9, 10, 2147483647, -2147483648], np.int32)
    w, cs = np.ones(64, np.float32), table(10, 64)
    r = Q.make_norm_rope(num_heads_q=2, num_heads_k=1, head_dim=64, rotary_dim=64, max_positions=10)
    d = _dev(x, False)
    qo = torch.full((6, 2, 64), 3, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((6, 1, 64), 3, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(64, dtype=torch.int32, device="cuda")
    Q.check(Q.norm_rope(r, d[:, :2], d[:, 2:], _dev(w, False), _dev(w, False), _dev(pos), _dev(cs), qo, ko, ws), "norm_rope")
    assert Q.get_device_error(ws) == (5, 1)
    got = np.concatenate([qo.double().cpu().numpy(), ko.double().cpu().numpy()], 1)
    assert not got[[1, 3, 4, 5]].any()
    _check(got, x, w, pos, cs, 64, False, 1e-6, True, False)


def test_runs_on_its_stream_and_in_a_graph(Q):
    import torch
    x = _dev(round_to(np.random.default_rng(6).normal(size=(40, 9, 128)), False), False)
    w, cs, pos = _dev(np.ones(128, np.float32), False), _dev(table(64, 128)), _dev(np.arange(40, dtype=np.int32))
    r = Q.make_norm_rope(num_heads_q=8, num_heads_k=1, head_dim=128, rotary_dim=128, max_positions=64)
    outs = [torch.empty(40, h, 128, dtype=torch.bfloat16, device="cuda") for h in (8, 1)]
    call = lambda st: Q.check(Q.norm_rope(r, x[:, :8], x[:, 8:], w, w, pos, cs, outs[0], outs[1], stream=st), "norm_rope")  # noqa: E731
    call(None)
    torch.cuda.synchronize()
    ref = [o.clone() for o in outs]
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            call(st)
    x.mul_(-1)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, -e) for o, e in zip(outs, ref))
