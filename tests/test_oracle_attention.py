"""Pins of the 64-bit oracle of the attention side, independent of the CUDA code: values worked by
hand, torch's float8 cast, grids searched by brute force, and invariants."""
import numpy as np
import pytest

from attention_tools import cache, cache_case, round_to, table
from oracle import ERR_LENGTH, ERR_PAGE
from oracle import attention as A


def test_e4m3_table_and_rounding_match_torch():
    torch = pytest.importorskip("torch")
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).float().numpy(), A.E4M3)
    mids = (A.E4M3[1:] + A.E4M3[:-1]) / 2
    a = np.concatenate([A.E4M3, mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9),
                        np.random.default_rng(0).uniform(0, 448, 2000)]).astype(np.float32)
    ref = torch.from_numpy(a).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(A._nearest(A.E4M3, a.astype(np.float64)), ref)


def test_block_worked_by_hand():
    # largest magnitude 12: E2M1 scale 2, int4 scale e4m3(12 / 7 = 1.714) = 1.75
    x = np.array([12, -12, 1, 3, 0.5, -0.5, 0, 5, 6, 7, -7, 8, 2.5, -1, 10, 11], np.float32)[None]
    code, s = A.quantize(x, True, 1.0)
    assert A.E4M3[s[0, 0]] == 2.0
    #    quotients  6  -6 .5 1.5 .25 -.25 0 2.5  3 3.5 -3.5  4 1.25 -.5  5 5.5
    assert code[0].tolist() == [7, 15, 1, 3, 0, 8, 0, 4, 5, 6, 14, 6, 2, 9, 6, 7]
    code, s = A.quantize(x, False, 1.0)
    assert A.E4M3[s[0, 0]] == 1.75
    want = [7, -7, 1, 2, 0, 0, 0, 3, 3, 4, -4, 5, 1, -1, 6, 6]
    assert code[0].tolist() == [c & 15 for c in want]


def test_codes_are_the_nearest_values():
    rng = np.random.default_rng(1)
    for e2m1 in (True, False):
        grid = np.concatenate([-A.E2M1, A.E2M1]) if e2m1 else np.arange(-7, 8)
        x = rng.normal(size=(200, 32)).astype(np.float32)
        code, s = A.quantize(x, e2m1, 1.0)
        sf = np.repeat(A.E4M3[s], 16, -1)
        c = code.astype(int)
        val = np.where(c >= 8, -A.E2M1[c & 7], A.E2M1[c & 7]) if e2m1 else np.where(c >= 8, c - 16, c)
        best = np.abs(x[..., None] - grid * sf[..., None]).min(-1)
        assert np.allclose(np.abs(x - val * sf), best, rtol=0, atol=1e-7 * np.abs(x).max())


def test_zero_and_tiny_blocks_have_zero_codes_and_scale():
    for e2m1 in (True, False):
        for x in (np.zeros((1, 16), np.float32), np.full((1, 16), -1e-6, np.float32)):
            code, s = A.quantize(x, e2m1, 1.0)
            assert not code.any() and not s.any()
        code, s = A.quantize(np.full((1, 16), 1e30, np.float32), e2m1, 1.0)
        assert A.E4M3[s[0, 0]] == 448 and (code == 7).all()


@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 64), (2, 128)])
@pytest.mark.parametrize("e2m1", [True, False])
def test_encode_decode_layout(heads, dim, e2m1):
    """Values on the grid survive exactly, at the documented bytes."""
    rng = np.random.default_rng(2)
    top = 6.0 if e2m1 else 7.0
    grid = A.E2M1 if e2m1 else np.arange(8)
    x = [grid[rng.integers(0, 8, (4, heads, dim))] * rng.choice([-1, 1], (4, heads, dim)) for _ in range(2)]
    for y in x:
        y[..., ::16] = top                                   # every block's scale is the factor
    k, v = (x[0] * 0.25).astype(np.float32), (x[1] * 8).astype(np.float32)
    e = A.encode(k, v, e2m1, k_scale=0.5, v_scale=2.0)
    assert e.shape[1] % 16 == 0 and e.shape[1] - heads * (dim + dim // 8) < 16
    dk, dv = A.decode(e, heads, dim, e2m1, 0.5, 2.0)
    assert np.array_equal(dk, k) and np.array_equal(dv, v)
    h = heads - 1
    unit = e[2, h * A.unit_bytes(dim):]
    assert np.all(A.E4M3[unit[dim:dim + dim // 16]] == 0.5) and np.all(A.E4M3[unit[dim + dim // 16:dim + dim // 8]] == 4.0)
    i = 7                                                    # element 7 of V: high nibble of byte 3
    nib = int(unit[dim // 2 + 3]) >> 4
    val = (-A.E2M1[nib & 7] if nib >= 8 else A.E2M1[nib & 7]) if e2m1 else (nib - 16 if nib >= 8 else nib)
    assert val * 4.0 * 2.0 == v[2, h, i]


def test_rotation_worked_by_hand_and_keeps_lengths():
    cs = np.array([[1, 1, 0, 0], [0, 0.6, 1, 0.8]], np.float32)              # R = 4: cosines, sines
    x = np.arange(1.0, 9.0)[None, None, :]
    got = A.norm_rope(x, None, [1], cs, 4, False, 0.0, norm=False)[0, 0]
    # pairs (0, 2) by 90 degrees, (1, 3) by (0.6, 0.8)
    assert np.allclose(got, [-3, 2 * 0.6 - 4 * 0.8, 1, 4 * 0.6 + 2 * 0.8, 5, 6, 7, 8], atol=1e-6)
    got = A.norm_rope(x, None, [1], cs, 4, True, 0.0, norm=False)[0, 0]
    assert np.allclose(got, [-2, 1, 3 * 0.6 - 4 * 0.8, 4 * 0.6 + 3 * 0.8, 5, 6, 7, 8], atol=1e-6)
    x = np.random.default_rng(3).normal(size=(5, 3, 64))
    for inter in (False, True):
        y = A.norm_rope(x, np.ones(64), [0, 1, 7, 30, 63], table(64, 32), 32, inter, 0.0)
        assert np.allclose((y * y).mean(-1), 1.0, atol=1e-5)
    assert not A.norm_rope(x, np.ones(64), [-1, 64, 0, 0, 0], table(64, 32), 32, False, 0.0)[:2].any()


def test_attention_with_one_entry_returns_its_value_and_equal_logits_average():
    case = cache_case(batch=2, s1=1, seq_lens_k=[40, 20], block_size=16, sparse_count=4, seed=1)
    pool = cache(case, 2, 64, True, seed=2)
    q = np.random.default_rng(3).normal(size=(2, 4, 64))
    idx = np.array([[33, -1, -1, -1], [-1, 3, 5, 3]], np.int32)
    out, lse, err, _ = A.sparse_attention(case, q, idx, pool, 2, True, 0.125)
    entry = pool[case.block_table[0, 2], 1][None]
    k, v = A.decode(entry, 2, 64, True)
    assert err == 0
    for h in range(4):
        assert np.allclose(out[0, h], v[0, h // 2]) and np.isclose(lse[0, h], 0.125 * k[0, h // 2] @ q[0, h])
    out, lse, _, _ = A.sparse_attention(case, np.zeros_like(q), idx, pool, 2, True, 0.125)
    e = np.stack([pool[case.block_table[1, 0], s] for s in (3, 5, 3)])
    assert np.allclose(out[1, 0], A.decode(e, 2, 64, True)[1][:, 0].mean(0)) and np.allclose(lse[1], np.log(3))


def test_attention_padding_and_error_conventions():
    case = cache_case(batch=2, s1=1, seq_lens_k=[40, 20], block_size=16, sparse_count=3, seed=1)
    pool = cache(case, 1, 64, False, seed=2)
    q = np.ones((2, 1, 64))
    out, lse, err, _ = A.sparse_attention(case, q, np.full((2, 3), -1, np.int32), pool, 1, False, 1.0)
    assert err == 0 and not out.any() and np.all(lse == -np.inf)
    idx = np.array([[40, 39, -2], [20, -1, -1]], np.int32)
    out, lse, err, spread = A.sparse_attention(case, q, idx, pool, 1, False, 1.0)
    assert err == ERR_LENGTH and spread["n"].tolist() == [1, 0] and np.isinf(lse[1, 0])
    case.block_table[0, 2] = case.num_blocks
    assert A.sparse_attention(case, q, idx, pool, 1, False, 1.0)[2] == ERR_LENGTH | ERR_PAGE


def test_cache_write_touches_only_its_entries():
    case = cache_case(batch=2, s1=1, seq_lens_k=[40, 20], block_size=16, sparse_count=3, seed=1)
    pool = np.random.default_rng(0).integers(0, 256, (case.num_blocks, 16, A.entry_bytes(1, 64)), dtype=np.uint8)
    before = pool.copy()
    k = round_to(np.random.default_rng(1).normal(size=(3, 1, 64)), False)
    err = A.cache_write(case, pool, k, k, [0, 1, 5], [17, 19, 0], True)
    assert err == ERR_LENGTH
    changed = np.argwhere((pool != before).any(-1)).tolist()
    assert sorted(changed) == sorted([[case.block_table[0, 1], 1], [case.block_table[1, 1], 3]])
    assert np.array_equal(pool[..., 72:], before[..., 72:])                  # padding bytes stay
    rk, rv, err = A.cache_read(case, pool, 1, 64, [0, 1, 0], [17, 19, 9999], True)
    assert err == ERR_LENGTH and np.array_equal(rk, rv) and not rk[2].any()
    assert np.abs(rk[:2] - k[:2]).max() < 0.5
