"""The 4-bit paged KV cache on the GPU (qli_kv_write, qli_kv_read) against the oracle: written bytes
identical, read values within their one rounding (needs a GB300)."""
import numpy as np
import pytest

from attention_tools import cache, cache_case, half_step, round_to, smallest_step
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


def _problem(Q, case):
    return Q.make_problem(batch=case.batch, max_q_tokens=1, num_blocks=case.num_blocks, block_size=case.block_size,
                          max_blocks_per_seq=case.max_blocks_per_seq, sparse_count=1, sparse_mode=0,
                          cmp_ratio=case.cmp_ratio, max_seqlen_q=1, max_seqlen_k=int(case.seq_lens_k.max()))


def _vectors(shape, f16, seed, e2m1, factor):
    """Normal vectors over a wide range of magnitudes; degenerate blocks first: zeros and signed zeros,
    quotients exactly halfway between codes, scales below and above e4m3's range, the types' extremes."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=shape) * np.exp(rng.uniform(-8, 6, size=shape[:-1] + (1,)))
    flat = x.reshape(-1, 16)
    top = 6.0 if e2m1 else 7.0
    mids = (A.E2M1[1:] + A.E2M1[:-1]) / 2 if e2m1 else np.arange(7) + 0.5
    ties = lambda s: np.append(np.resize(mids, 15) * rng.choice([-1, 1], 15), top) * s  # noqa: E731
    special = [np.zeros(16), np.resize([0.0, -0.0], 16), ties(1.0), ties(0.375), ties(2.0 ** -6), np.full(16, 2.0 ** -11),
               np.full(16, -3e-5), ties(448.0), np.resize([6e4, -6e4, 1.0], 16), np.append(np.full(15, -1e-4), 50.0)]
    # a scale halfway between two e4m3 values: max / Q = 1.0625 (ties to 1.0) and 1.1875 (to 1.25)
    special += [np.append(rng.normal(size=15), top * 1.0625), np.append(rng.normal(size=15), top * 1.1875)]
    for i, s in enumerate(special[:len(flat)]):
        flat[i] = s * (factor if i not in (6, 8) else 1.0)
    return round_to(x, f16)


LAYOUTS = [(1, 64), (1, 128), (3, 64), (8, 128), (5, 128), (16, 64), (64, 128)]


@pytest.mark.parametrize("heads,dim", LAYOUTS)
@pytest.mark.parametrize("e2m1", [True, False])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("factors", [(1.0, 1.0), (0.3, 5.0), (0.25, 2.0 ** -7)])
def test_write_is_bit_exact_and_read_back(Q, heads, dim, e2m1, f16, factors):
    import torch
    case = cache_case(batch=3, s1=1, seq_lens_k=[70, 33, 1], block_size=16, sparse_count=1, seed=heads, extra_pages=2)
    rng = np.random.default_rng(dim)
    tb = np.concatenate([np.full(20, 0), np.full(9, 1), [2]]).astype(np.int32)
    tp = np.concatenate([rng.permutation(70)[:20], rng.permutation(33)[:9], [0]]).astype(np.int32)
    n = len(tb)
    k, v = (_vectors((n, heads, dim), f16, s, e2m1, g) for s, g in zip((1, 2), factors))
    eb = A.entry_bytes(heads, dim)
    stride = case.block_size * eb + 48                                         # pages with a gap after them
    raw = rng.integers(0, 256, (case.num_blocks, stride), dtype=np.uint8)
    pool = raw[:, :case.block_size * eb].reshape(case.num_blocks, case.block_size, eb)
    ref = pool.copy()
    assert A.cache_write(case, ref, k, v, tb, tp, e2m1, *factors) == 0
    a = Q.make_attention(num_heads_q=heads, num_heads_kv=heads, head_dim=dim, dtype=Q.ACT_F16 if f16 else Q.ACT_BF16,
                         kv_dtype=Q.KV_E2M1 if e2m1 else Q.KV_INT4, k_scale=factors[0], v_scale=factors[1], kv_stride=stride)
    assert Q.kv_entry_bytes(a) == eb
    p = _problem(Q, case)
    packed = _dev(np.concatenate([k, v, k[:, :1]], 1), f16)                    # strided views of one projection
    d = _dev(raw)
    ws = torch.zeros(64, dtype=torch.int32, device="cuda")
    Q.check(Q.kv_write(p, a, packed[:, :heads], packed[:, heads:2 * heads], _dev(tb), _dev(tp), _dev(case.block_table), d,
                       ws), "kv_write")
    got = d.cpu().numpy()
    assert np.array_equal(got[:, :case.block_size * eb].reshape(ref.shape), ref)
    assert np.array_equal(got[:, case.block_size * eb:], raw[:, case.block_size * eb:])
    out = torch.full((n, 2 * heads + 1, dim), 9, dtype=packed.dtype, device="cuda")
    Q.check(Q.kv_read(p, a, _dev(tb), _dev(tp), _dev(case.block_table), d, out[:, :heads], out[:, heads:2 * heads], ws),
            "kv_read")
    assert Q.get_device_error(ws) == (0, 0)
    rk, rv, _ = A.cache_read(case, ref, heads, dim, tb, tp, e2m1, *factors)
    want = np.concatenate([rk, rv], 1)
    o = out[:, :2 * heads].double().cpu().numpy()
    limit = 65504.0 if f16 else 3e38
    inside = np.abs(want) <= limit
    # code * scale is exact in fp32 (at most 6 significant bits), the factor rounds once, the type once
    tol = np.abs(want) * (half_step(f16) + 2.0 ** -23) + smallest_step(f16)
    assert np.all(np.abs(o - want)[inside] <= tol[inside]) and (out[:, 2 * heads:] == 9).all()
    assert np.array_equal(np.sign(o[~inside]), np.sign(want[~inside]))


def test_invalid_tokens(Q):
    import torch
    case = cache_case(batch=2, s1=1, seq_lens_k=[100, 40], block_size=32, sparse_count=1, seed=5)
    case.block_table[0, 3] = case.num_blocks + 2
    case.block_table[1, 3] = -7
    pool = cache(case, 2, 64, True, seed=1)
    #             ok  batch  batch  pos  pos    page  page  beyond the table, ok
    tb = np.array([0, 2, -1, 0, 1, 0, 1, 1, 1], np.int32)
    tp = np.array([5, 0, 3, -1, 2147483647, 99, 127, 128, 39], np.int32)
    k = round_to(np.random.default_rng(0).normal(size=(9, 2, 64)), False)
    ref = pool.copy()
    err = A.cache_write(case, ref, k, -k, tb, tp, True)
    assert err == 3
    a, p = Q.make_attention(num_heads_q=2, num_heads_kv=2, head_dim=64), _problem(Q, case)
    d, kd = _dev(pool), _dev(k, False)
    ws = torch.zeros(64, dtype=torch.int32, device="cuda")
    args = (_dev(tb), _dev(tp), _dev(case.block_table))
    Q.check(Q.kv_write(p, a, kd, -kd, *args, d, ws), "kv_write")
    assert Q.get_device_error(ws) == (5, err)
    assert np.array_equal(d.cpu().numpy(), ref)
    ko, vo = torch.full_like(kd, 3), torch.full_like(kd, 3)
    Q.check(Q.kv_read(p, a, *args, d, ko, vo, ws), "kv_read")
    assert Q.get_device_error(ws) == (5, err)
    rk, rv, _ = A.cache_read(case, ref, 2, 64, tb, tp, True)
    assert np.array_equal(ko.double().cpu().numpy(), rk) and np.array_equal(vo.double().cpu().numpy(), rv)
    # without a workspace the same tokens are skipped
    Q.check(Q.kv_write(p, a, kd, -kd, *args, d), "kv_write")
    assert np.array_equal(d.cpu().numpy(), ref)


def test_offsets_past_32_bits(Q):
    """A pool of 5 GB: entries on its last pages are found (page * stride needs 64 bits)."""
    import torch
    heads, dim, bs = 64, 128, 1024
    a = Q.make_attention(num_heads_q=64, num_heads_kv=heads, head_dim=dim, kv_stride=1024 * 9216 + (1 << 28))
    nb = 20
    page = a.kv_stride
    p = Q.make_problem(batch=1, max_q_tokens=1, num_blocks=nb, block_size=bs, max_blocks_per_seq=2, sparse_count=1,
                       sparse_mode=0, cmp_ratio=1, max_seqlen_q=1, max_seqlen_k=2 * bs)
    pool = torch.zeros(nb * page, dtype=torch.uint8, device="cuda")
    table = _dev(np.array([[nb - 1, nb - 2]], np.int32))
    k = round_to(np.random.default_rng(1).normal(size=(2, heads, dim)), False)
    tb, tp = np.zeros(2, np.int32), np.array([bs - 1, 2 * bs - 1], np.int32)
    kd = _dev(k, False)
    Q.check(Q.kv_write(p, a, kd, kd, _dev(tb), _dev(tp), table, pool), "kv_write")
    ref = A.encode(k, k, True)
    for i, pg in enumerate((nb - 1, nb - 2)):
        at = pg * page + (bs - 1) * 9216
        assert np.array_equal(pool[at:at + 9216].cpu().numpy(), ref[i])
    ko, vo = torch.empty_like(kd), torch.empty_like(kd)
    Q.check(Q.kv_read(p, a, _dev(tb), _dev(tp), table, pool, ko, vo), "kv_read")
    assert np.array_equal(ko.double().cpu().numpy(), A.decode(ref, heads, dim, True)[0])
    del pool


def test_write_then_read_in_a_graph(Q):
    import torch
    case = cache_case(batch=4, s1=1, seq_lens_k=[64] * 4, block_size=16, sparse_count=1, seed=2)
    a, p = Q.make_attention(num_heads_q=2, num_heads_kv=2, head_dim=128, kv_dtype=Q.KV_INT4), _problem(Q, case)
    pool = torch.zeros(case.num_blocks, 16, Q.kv_entry_bytes(a), dtype=torch.uint8, device="cuda")
    tb, tp, bt = _dev(np.arange(4, dtype=np.int32)), _dev(np.array([0, 17, 34, 63], np.int32)), _dev(case.block_table)
    x = torch.zeros(4, 4, 128, dtype=torch.bfloat16, device="cuda")
    k, v = torch.empty(4, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            Q.check(Q.kv_write(p, a, x[:, :2], x[:, 2:], tb, tp, bt, pool), "kv_write")
            Q.check(Q.kv_read(p, a, tb, tp, bt, pool, k, v), "kv_read")
    for seed in (1, 2):
        new = round_to(np.random.default_rng(seed).normal(size=(4, 4, 128)), False)
        x.copy_(_dev(new, False))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        dk, dv = A.decode(A.encode(new[:, :2], new[:, 2:], False), 2, 128, False)
        assert np.array_equal(k.double().cpu().numpy(), dk) and np.array_equal(v.double().cpu().numpy(), dv)
