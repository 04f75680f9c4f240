"""The probabilities of the dense paged attention, through both of its kernels, against the 64-bit oracle (needs a
GB300): with float16 activations they enter the products with the bits that fp16 drops of them, and those far below a
row's largest count whatever the number of positions."""
import math

import numpy as np
import pytest

from attention_tools import cache, cache_case, half_step, round_to, smallest_step
from oracle import attention as A
from paged_tools import attend, check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", params=[1, 2], ids=["few", "many"])
def Q(request):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_token_block_gb300 import build as B
    B.build()
    import sparse_attention_token_block_gb300 as Q
    saved = Q._lib_handle, Q._lib_path
    Q._lib_handle, Q._lib_path = None, Q.TESTING_LIB_PATH
    Q.lib.qli_testing_set_paged(request.param)
    yield Q
    Q.lib.qli_testing_set_paged(0)
    Q._lib_handle, Q._lib_path = saved


def _bounds(ref, spread, f16, terms, depth=25):
    """Bound of |out - ref| for exact queries (powers of two times integers below 2^11) of which `terms` elements are not
    zero, the other products adding nothing:
      * logits: `terms` - 1 additions of a product's sum (each within 2^-23 of the sum of magnitudes, truncation allowed), the
        factor's three roundings and the fused multiply-add's one (2^-24 each): (2 terms + 4) 2^-24 of the magnitudes, in
        numerator and denominator;
      * exponentials 2^-20 (the function 2^-22, and the rounding of its argument, below 32 in magnitude, 2^-20 ln 2), in both too:
        2^-19;
      * n + 64 additions of a sum and of an output, 2^-23 each;
      * a probability within 2^-22 of itself (float16: fp16's half step of a remainder of at most 2^-11) or 2^-11 (bfloat16:
        one rounding to fp16), and within 2^-`depth` of a row's sum: 2^-25 is fp16's half step below its normal range, of
        numbers among which the largest stands at 2^0 at least (in the kernels a row's sum stands at 2^6 at least, the lower of 2^11
        and 2^6: depth 31);
      * the output's own rounding."""
    n = np.maximum(spread["n"], 1)[:, None]
    dz = spread["qk"] * (2 * terms + 4) * 2.0 ** -24
    rel = (2.0 ** -22 if f16 else 2.0 ** -11) + 2 * dz + 2.0 ** -19 + (n + 64) * 2.0 ** -23
    err = rel[..., None] * (spread["wv"] + np.abs(ref)) + (n * 2.0 ** -depth * spread["vmax"])[..., None]
    return err + half_step(f16) * (np.abs(ref) + err) + smallest_step(f16)


def _check(case, got, q, pool, hkv, e2m1, f16, scale, terms, depth=25, **kw):
    out, lse, bits = got
    ref, rl, err, spread = A.paged_attention(case, q, pool, hkv, e2m1, scale, **kw)
    assert bits == err == 0
    bad = ~(np.abs(out - ref) <= _bounds(ref, spread, f16, terms, depth))
    assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[:3], out[bad][:3], ref[bad][:3])
    n = np.maximum(spread["n"], 1)[:, None]
    ltol = spread["qk"] * (2 * terms + 4) * 2.0 ** -24 + 2.0 ** -19 + n * 2.0 ** -23 + 2.0 ** -22 * np.abs(rl)
    assert np.all(np.abs(lse - rl) <= ltol)


# few positions a row, so that the probabilities' errors do not average out
@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 128), (16, 2, 64), (5, 1, 128), (3, 3, 64)])
@pytest.mark.parametrize("e2m1", [True, False])
@pytest.mark.parametrize("terms", [4, 1])
def test_float16_outputs_are_off_by_their_rounding(Q, hq, hkv, dim, e2m1, terms):
    rows = 300
    case = cache_case(layout_q="TND", q_lens=[rows], seq_lens_k=[700], block_size=16, sparse_count=1, sparse_mode=3, seed=3)
    pool = cache(case, hkv, dim, e2m1, seed=1)
    rng = np.random.default_rng(4)
    q = np.zeros((rows, hq, dim), np.float32)
    q[..., rng.permutation(dim)[:terms]] = rng.normal(size=(rows, hq, terms))
    q = round_to(q, True)
    # (sharp: rows raise their maximum in the middle of a tile)
    for scale, window, sinks in ((1 / math.sqrt(terms), 8, 0), (1 / math.sqrt(terms), 6, 2), (20.0, 40, 3)):
        got = attend(Q, case, q, pool, hkv, e2m1, True, window=window, sinks=sinks, scale=scale)
        _check(case, got, q, pool, hkv, e2m1, True, scale, terms, window=window, sinks=sinks)


def _one_far_above(n, dim, gap, spread, e2m1, seed):
    """A case and a pool of one KV head: position 0 has a logit of 0 and a value of zeros, the n others logits about `gap` bits
    lower, spread over about `spread` bits, and values about 1."""
    case = cache_case(batch=1, s1=1, seq_lens_k=[n + 1], block_size=64, sparse_count=1, sparse_mode=3, seed=seed, permute=False)
    slots = case.num_blocks * case.block_size
    rng = np.random.default_rng(seed)
    k, v = np.zeros((slots, 1, dim), np.float32), np.zeros((slots, 1, dim), np.float32)
    at = (case.block_table[0][:, None] * 64 + np.arange(64)).reshape(-1)[:n + 1]
    k[at[1:], 0, 0] = -gap * math.log(2.0)
    k[at[1:], 0, 16] = rng.uniform(-0.5, 0.5, n) * spread * math.log(2.0)
    v[at[1:]] = 1 + 0.25 * rng.normal(size=(n, 1, dim))
    return case, A.encode(k, v, e2m1).reshape(case.num_blocks, 64, -1)


@pytest.mark.parametrize("gap", [20, 22, 24, 25, 26, 27])
@pytest.mark.parametrize("spread", [1, 0])
@pytest.mark.parametrize("f16", [False, True])
def test_one_position_far_above_many(Q, gap, spread, f16):
    dim, e2m1 = (64, True) if gap % 2 else (128, False)
    case, pool = _one_far_above(100000, dim, gap, spread, e2m1, gap)
    q = np.zeros((1, 2, dim), np.float32)
    q[:, :, 0] = 1
    q[:, 1, 16] = 1
    _check(case, attend(Q, case, q, pool, 1, e2m1, f16, scale=1.0), q, pool, 1, e2m1, f16, 1.0, 2, depth=31)


@pytest.mark.parametrize("gap", [24, 27])
@pytest.mark.parametrize("f16", [False, True])
def test_one_position_far_above_many_in_one_warp(Q, gap, f16):
    """The same where a warp carries all positions of a sequence: more sequences than the GPU holds CTAs, of the same pages."""
    dim, hkv, sequences = 64, 8, 640
    case, one = _one_far_above(50000, dim, gap, 1, True, gap)
    unit = A.unit_bytes(dim)
    pool = np.tile(one[..., :unit], hkv)
    q = np.zeros((sequences, hkv, dim), np.float32)
    q[:, :, 0] = 1
    q[sequences // 2:, :, 16] = 1
    many = cache_case(batch=sequences, s1=1, seq_lens_k=[1] * sequences, block_size=64, sparse_count=1, sparse_mode=3, seed=1)
    many.seq_lens_k = np.repeat(case.seq_lens_k, sequences)
    many.block_table = np.repeat(case.block_table, sequences, 0)
    many.num_blocks, many.max_blocks_per_seq = case.num_blocks, case.max_blocks_per_seq
    out, lse, bits = attend(Q, many, q, pool, hkv, True, f16, scale=1.0)
    for b in (0, sequences - 1):
        got = out[b:b + 1, :1], lse[b:b + 1, :1], bits
        _check(case, got, q[b:b + 1, :1], one, 1, True, f16, 1.0, 2, depth=31)
    for half in (slice(0, sequences // 2), slice(sequences // 2, None)):         # every head and sequence the same
        assert (out[half] == out[half][:1, :1]).all() and (lse[half] == lse[half][:1, :1]).all()


@pytest.mark.parametrize("factor", [2.0 ** -124, 2.0 ** 100])
def test_factors_near_the_ends_of_the_range(Q, factor):
    case = cache_case(layout_q="TND", q_lens=[150, 1], seq_lens_k=[900, 5000], block_size=64, sparse_count=1, sparse_mode=3, seed=2)
    pool, q = cache(case, 2, 64, True, 1, 1.0, factor), queries(case.rows, 8, 64, False, 2)
    got = attend(Q, case, q, pool, 2, True, False, factors=(1.0, factor))
    check(case, got, q, pool, 2, True, False, factors=(1.0, factor))


@pytest.mark.parametrize("std", [3.0, 10.0])
@pytest.mark.parametrize("e2m1,f16", [(True, False), (False, True)])
def test_logits_that_spread_widely(Q, std, e2m1, f16):
    """Rows whose maximum rises again and again, in first and second halves of tiles, beside others whose does not."""
    case = cache_case(layout_q="TND", q_lens=[260, 40], seq_lens_k=[2500, 1200], block_size=64, sparse_count=1, sparse_mode=3, seed=2)
    pool, q = cache(case, 2, 64, e2m1, 1), queries(case.rows, 4, 64, f16, 2)
    q[::3] *= np.float32(std)
    q = round_to(q, f16)
    for window, sinks in ((0, 0), (200, 3)):
        got = attend(Q, case, q, pool, 2, e2m1, f16, window=window, sinks=sinks)
        check(case, got, q, pool, 2, e2m1, f16, window=window, sinks=sinks)


def _sized_logits(scale, f16):
    """Queries with one element that is not zero, of 0.7 to 1.3: equal codes and scales give equal logits, others differ by more
    than any rounding, and a row's largest is 2.1 to 7.8 times `scale`."""
    dim, hkv, hq, rows = 64, 2, 4, 150
    case = cache_case(layout_q="TND", q_lens=[rows, 1], seq_lens_k=[700, 333], block_size=16, sparse_count=1, sparse_mode=3, seed=3)
    rng = np.random.default_rng(5)
    n = case.num_blocks * case.block_size
    k = rng.choice([-3.0, -1.0, 0.5, 1.0, 2.0, 6.0], size=(n, hkv, dim)).astype(np.float32)
    k[..., ::16] = 6.0                                      # (every block's scale is 1)
    pool = A.encode(k, rng.normal(size=(n, hkv, dim)).astype(np.float32), True).reshape(case.num_blocks, 16, -1)
    q = np.zeros((case.rows, hq, dim), np.float32)
    q[..., 5] = round_to(rng.uniform(0.7, 1.3, size=(case.rows, hq)) * rng.choice([-1, 1], size=(case.rows, hq)), f16)
    return case, q, pool, hkv


@pytest.mark.parametrize("scale", [2.0 ** e for e in (8, 16, 20, 22, 24)])
@pytest.mark.parametrize("f16", [False, True])
def test_large_logits(Q, scale, f16):
    """Up to 2^27, of which fp32 holds every 16th: the positions of the largest share the weight."""
    case, q, pool, hkv = _sized_logits(scale, f16)
    out, lse, bits = attend(Q, case, q, pool, hkv, True, f16, scale=scale)
    ref, rl, err, spread = A.paged_attention(case, q, pool, hkv, True, scale)
    assert bits == err == 0
    spread["qk"] = np.zeros_like(spread["qk"])              # (equal logits have equal errors)
    assert (np.abs(out - ref) <= _bounds(ref, spread, f16, 1)).all()
    # (the factor's three roundings, the product's and those of the way to the natural logarithm: 2^-24 each)
    assert (np.abs(lse - rl) <= 7 * 2.0 ** -24 * np.abs(rl) + 2.0 ** -10).all()


@pytest.mark.parametrize("scale", [2.0 ** e for e in (28, 30, 40, 60, 120)])
@pytest.mark.parametrize("f16", [False, True])
def test_logits_beyond_the_range_are_no_numbers(Q, scale, f16):
    case, q, pool, hkv = _sized_logits(scale, f16)
    out, lse, bits = attend(Q, case, q, pool, hkv, True, f16, scale=scale)
    assert bits == 0 and np.isnan(out).all() and np.isnan(lse).all()
