"""Norm, rotation and cache write of new tokens in one pass (qli_kv_append) against the 64-bit oracle (needs a
GB300)."""
import numpy as np
import pytest

from attention_tools import cache_case, table
from oracle import attention as A
from paged_tools import check_cached, dev, half_step, round_to, smallest_step, turn_bound

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


class Step:
    """Inputs of one call: packed projections of `n` tokens over three sequences."""

    def __init__(self, n, hq, hkv, dim, rotary, e2m1, f16, interleaved=False, norm=True, factors=(1.0, 1.0), seed=0,
                 max_pos=5000, block_size=16, gap=48):
        rng = np.random.default_rng(seed)
        self.n, self.hq, self.hkv, self.dim, self.rotary, self.e2m1, self.f16 = n, hq, hkv, dim, rotary, e2m1, f16
        self.interleaved, self.norm, self.factors = interleaved, norm, factors
        lens = [max(16, n), max(70, n), 33]
        self.case = cache_case(batch=3, s1=1, seq_lens_k=lens, block_size=block_size, sparse_count=1, seed=seed, extra_pages=1)
        places = [(b, j) for b in range(3) for j in range(lens[b])]
        pick = rng.permutation(len(places))[:n]
        self.tb, self.tp = (np.array([places[i][x] for i in pick], np.int32) for x in (0, 1))
        self.positions = rng.integers(0, max_pos, n).astype(np.int32)
        mag = np.exp(rng.uniform(-6, 5, size=(n, hq + 2 * hkv, 1)))
        self.qkv = round_to(rng.normal(size=(n, hq + 2 * hkv, dim)) * mag, f16)
        if n > 2:
            self.qkv[2, -1] = 0.0                              # a vector of zeros
        self.q, self.k, self.v = self.qkv[:, :hq], self.qkv[:, hq:hq + hkv], self.qkv[:, hq + hkv:]
        self.qw, self.kw = (round_to(1 + 0.3 * rng.normal(size=dim), f16) for _ in range(2))
        self.cos_sin = table(max_pos, rotary) if rotary else np.zeros((max_pos, 0), np.float32)
        eb = A.entry_bytes(hkv, dim)
        self.stride = block_size * eb + gap
        self.raw = rng.integers(0, 256, (self.case.num_blocks, self.stride), dtype=np.uint8)

    def pool(self, raw):
        eb, c = A.entry_bytes(self.hkv, self.dim), self.case
        return raw[:, :c.block_size * eb].reshape(c.num_blocks, c.block_size, eb)

    def settings(self, Q):
        c = self.case
        p = Q.make_problem(batch=c.batch, max_q_tokens=1, num_blocks=c.num_blocks, block_size=c.block_size,
                           max_blocks_per_seq=c.max_blocks_per_seq, sparse_count=1, sparse_mode=0, cmp_ratio=1, max_seqlen_q=1,
                           max_seqlen_k=int(c.seq_lens_k.max()))
        act = Q.ACT_F16 if self.f16 else Q.ACT_BF16
        a = Q.make_attention(num_heads_q=max(self.hq, self.hkv) // self.hkv * self.hkv, num_heads_kv=self.hkv, head_dim=self.dim,
                             dtype=act, kv_dtype=Q.KV_E2M1 if self.e2m1 else Q.KV_INT4, k_scale=self.factors[0],
                             v_scale=self.factors[1], kv_stride=self.stride)
        r = Q.make_norm_rope(num_heads_q=self.hq, num_heads_k=self.hkv, head_dim=self.dim, rotary_dim=self.rotary,
                             max_positions=len(self.cos_sin), dtype=act, interleaved=self.interleaved, norm=self.norm, eps=1e-5)
        return p, a, r

    def run(self, Q, packed=True, in_place=False):
        """(q out, pool bytes, error bits)"""
        import torch
        x = dev(self.qkv, self.f16)
        q, k, v = x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]
        if not packed:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        out = q if in_place else torch.full((self.n, self.hq, self.dim), 7.0, dtype=x.dtype, device="cuda")
        raw, ws = dev(self.raw), torch.zeros(64, dtype=torch.int32, device="cuda")
        w = (dev(self.qw, self.f16), dev(self.kw, self.f16)) if self.norm else (None, None)
        st = Q.kv_append(*self.settings(Q), q, k, v, *w, dev(self.positions), dev(self.cos_sin), dev(self.tb), dev(self.tp),
                         dev(self.case.block_table), out, raw, ws)
        Q.check(st, "kv_append")
        bits = Q.get_device_error(ws)[1]
        assert torch.equal(x[:, self.hq:].float(), dev(self.qkv, self.f16)[:, self.hq:].float())      # inputs stay
        return out.double().cpu().numpy(), raw.cpu().numpy(), bits

    def check(self, got):
        out, raw, bits = got
        want = self.raw.copy()
        q, k, err = A.append(self.case, self.pool(want), self.q, self.k, self.v, self.qw, self.kw, self.positions, self.cos_sin,
                             self.rotary, self.interleaved, 1e-5, self.tb, self.tp, self.e2m1, *self.factors, norm=self.norm)
        assert bits == err
        args = (self.positions, self.cos_sin, self.rotary, self.interleaved, np.float64(np.float32(1e-5)), self.norm)
        dq = turn_bound(self.q, self.qw, *args)
        assert (np.abs(out - q) <= dq + half_step(self.f16) * (np.abs(q) + dq) + smallest_step(self.f16)).all()
        # values, what was not written and the gaps: the same bytes; keys: codes between those of the ends of what
        # the turned key may be
        dk = turn_bound(self.k, self.kw, *args)
        eb, unit = A.entry_bytes(self.hkv, self.dim), A.unit_bytes(self.dim)
        key = np.zeros(eb, bool)
        for h in range(self.hkv):
            key[h * unit:h * unit + self.dim // 2] = key[h * unit + self.dim:h * unit + self.dim + self.dim // 16] = True
        g, w = self.pool(raw), self.pool(want)
        assert np.array_equal(g[..., ~key], w[..., ~key])
        assert np.array_equal(raw[:, self.case.block_size * eb:], self.raw[:, self.case.block_size * eb:])
        written = np.zeros(g.shape[:2], bool)
        for t in range(self.n):
            where, _ = A.entry_of(self.case, int(self.tb[t]), int(self.tp[t]), self.case.max_blocks_per_seq * self.case.block_size)
            if where and 0 <= self.positions[t] < len(self.cos_sin):
                written[where] = True
                for h in range(self.hkv):
                    check_cached(g[where][None, h * unit:(h + 1) * unit], k[t, h][None], dk[t, h][None], self.e2m1, self.factors[0],
                                 False)
        assert np.array_equal(g[~written], self.pool(self.raw)[~written])


LAYOUTS = [(4, 1, 128, 128), (0, 3, 64, 32), (64, 8, 128, 128), (7, 7, 64, 24), (20, 5, 64, 64), (9, 3, 128, 0), (5, 1, 128, 24),
           (128, 64, 128, 64)]


@pytest.mark.parametrize("hq,hkv,dim,rotary", LAYOUTS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("e2m1,f16", [(True, False), (False, True), (True, True), (False, False)])
@pytest.mark.parametrize("norm,factors", [(True, (1.0, 1.0)), (False, (0.3, 5.0)), (True, (0.25, 2.0 ** -7))])
def test_against_the_oracle(Q, hq, hkv, dim, rotary, interleaved, e2m1, f16, norm, factors):
    s = Step(9, hq, hkv, dim, rotary, e2m1, f16, interleaved, norm, factors, seed=hq + rotary)
    s.check(s.run(Q, packed=interleaved, in_place=norm))


@pytest.mark.parametrize("n", [1, 2, 33, 300, 3000])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (64, 8)])
def test_numbers_of_tokens(Q, n, hq, hkv):
    if n == 3000 and hq == 64:
        n = 1500
    s = Step(n, hq, hkv, 128, 128, True, False, seed=n, block_size=64)
    s.check(s.run(Q))


def test_bad_tokens(Q):
    s = Step(12, 8, 2, 128, 64, True, False, seed=3)
    s.tb[1], s.tb[4] = -1, 3
    s.tp[2], s.tp[5] = -1, s.case.max_blocks_per_seq * s.case.block_size
    s.positions[3], s.positions[6] = -1, 5000
    s.check(s.run(Q))
    out = s.run(Q)[0]
    assert not out[[3, 6]].any() and out[[1, 2, 4, 5]].any((1, 2)).all()
    s = Step(12, 8, 2, 128, 64, True, False, seed=4)
    s.case.block_table[s.tb[0], s.tp[0] // 16] = s.case.num_blocks
    s.check(s.run(Q))


def test_same_values_as_the_two_calls(Q):
    """Against qli_norm_rope and qli_kv_write: the queries' and the values' bits, the keys where rounding them
    first changes nothing (float16 keys that are exact: no norm, no rotation)."""
    import torch
    s = Step(40, 16, 4, 128, 128, False, True, seed=5, gap=0)
    out, raw, _ = s.run(Q)
    p, a, r = s.settings(Q)
    x = dev(s.qkv, True)
    q, k = torch.empty(40, 16, 128, dtype=torch.float16, device="cuda"), torch.empty(40, 4, 128, dtype=torch.float16, device="cuda")
    Q.check(Q.norm_rope(r, x[:, :16], x[:, 16:20], dev(s.qw, True), dev(s.kw, True), dev(s.positions), dev(s.cos_sin), q, k))
    assert np.array_equal(out, q.double().cpu().numpy())
    s = Step(40, 16, 4, 128, 0, False, True, seed=6, norm=False)
    out, raw, _ = s.run(Q)
    p, a, r = s.settings(Q)
    x, pool = dev(s.qkv, True), dev(s.raw)
    Q.check(Q.kv_write(p, a, x[:, 16:20], x[:, 20:], dev(s.tb), dev(s.tp), dev(s.case.block_table), pool))
    assert np.array_equal(raw, pool.cpu().numpy()) and np.array_equal(out, s.q.astype(np.float64))


def test_graph(Q):
    import torch
    s = Step(20, 8, 2, 128, 128, True, False, seed=7)
    want = s.run(Q)
    x, raw = dev(s.qkv, False), dev(s.raw)
    out = torch.zeros(20, 8, 128, dtype=torch.bfloat16, device="cuda")
    rest = (dev(s.qw, False), dev(s.kw, False), dev(s.positions), dev(s.cos_sin), dev(s.tb), dev(s.tp), dev(s.case.block_table))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        Q.check(Q.kv_append(*s.settings(Q), x[:, :8], x[:, 8:10], x[:, 10:], *rest, out, raw))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want[0]) and np.array_equal(raw.cpu().numpy(), want[1])
