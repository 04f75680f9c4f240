"""The probabilities of the dense paged attention, through both of its kernels, against the 64-bit oracle (needs a
GB300): with float16 activations they enter the products with the bits that fp16 drops of them."""
import math

import numpy as np
import pytest

from attention_tools import cache, cache_case, half_step, round_to, smallest_step
from oracle import attention as A
from paged_tools import attend

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


def _bounds(ref, spread, f16, terms):
    """Bound of |out - ref| for exact queries (powers of two times integers below 2^11) of which `terms` elements are not
    zero, the other products adding nothing:
      * logits: `terms` - 1 additions of a product's sum (each within 2^-23 of the sum of magnitudes, truncation allowed), the
        factor's three roundings and the fused multiply-add's one (2^-24 each): (2 terms + 4) 2^-24 of the magnitudes, in
        numerator and denominator;
      * exponentials 2^-20 (the function 2^-22, and the rounding of its argument, below 32 in magnitude, 2^-20 ln 2), in both too:
        2^-19;
      * n + 64 additions of a sum and of an output, 2^-23 each;
      * a probability within 2^-22 of itself (float16: fp16's half step of a remainder of at most 2^-11) or 2^-11 (bfloat16:
        one rounding to fp16), 2^-25 below fp16's normal range;
      * the output's own rounding."""
    n = np.maximum(spread["n"], 1)[:, None]
    dz = spread["qk"] * (2 * terms + 4) * 2.0 ** -24
    rel = (2.0 ** -22 if f16 else 2.0 ** -11) + 2 * dz + 2.0 ** -19 + (n + 64) * 2.0 ** -23
    err = rel[..., None] * (spread["wv"] + np.abs(ref)) + (n * 2.0 ** -25 * spread["vmax"])[..., None]
    return err + half_step(f16) * (np.abs(ref) + err) + smallest_step(f16)


def _check(case, got, q, pool, hkv, e2m1, f16, scale, terms, **kw):
    out, lse, bits = got
    ref, rl, err, spread = A.paged_attention(case, q, pool, hkv, e2m1, scale, **kw)
    assert bits == err == 0
    bad = ~(np.abs(out - ref) <= _bounds(ref, spread, f16, terms))
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
