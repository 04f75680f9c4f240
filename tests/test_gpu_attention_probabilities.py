"""With float16 activations the attention's probabilities enter the products with the bits that fp16 drops of
them: the output is off by its own rounding and the fp32 sums', no more (both kernels, against the 64-bit
oracle; needs a GB300)."""
import math

import numpy as np
import pytest

from attention_tools import cache, cache_case, half_step, round_to, smallest_step
from oracle import attention as A
from test_gpu_attention_ranges import _lists, _sample, _sms
from test_gpu_sparse_attention import Q, _run  # noqa: F401 (Q is a fixture)

pytestmark = pytest.mark.gpu

USED = 4                                                     # elements of a query that are not zero


def _bounds(ref, spread):
    """As attention_bounds, for exact queries of which USED elements are not zero (the other products add
    nothing), and probabilities within 2^-22 of themselves (fp16's half step of a remainder of at most 2^-11),
    2^-25 below its normal range."""
    n = spread["n"][:, None]
    dz = spread["qk"] * (USED + 16) * 2.0 ** -23 * 2
    rel = 2.0 ** -22 + 2 * dz + (n + 64) * 2.0 ** -23 + 2.0 ** -20
    err = rel[..., None] * (spread["wv"] + np.abs(ref)) + (n * 2.0 ** -25 * spread["vmax"])[..., None]
    return err + half_step(True) * (np.abs(ref) + err) + smallest_step(True)


@pytest.mark.parametrize("hq,hkv,dim,blocks", [(64, 8, 64, False), (32, 2, 64, False), (64, 8, 128, False), (64, 8, 128, True),
                                               (32, 8, 128, True)])
@pytest.mark.parametrize("e2m1", [True, False])
def test_outputs_are_off_by_their_rounding(Q, hq, hkv, dim, blocks, e2m1):  # noqa: F811
    per = 128 * hkv // hq
    rows = per * -(-_sms() // hkv) if blocks else 40
    case = cache_case(layout_q="TND", q_lens=[rows], seq_lens_k=[600], block_size=16, sparse_count=512, seed=3)
    pool = cache(case, hkv, dim, e2m1, seed=1)
    idx = _lists(case, 2)
    idx[:, 8:] = -1
    q = np.zeros((rows, hq, dim), np.float32)
    rng = np.random.default_rng(4)
    q[..., rng.permutation(dim)[:USED]] = rng.normal(size=(rows, hq, USED))
    q = round_to(q, True)
    scale = 1 / math.sqrt(USED)
    got = _run(Q, case, q, idx, pool, hkv, e2m1, True, scale)
    case, (out, lse, bits), q, idx = _sample(case, got, q, idx, np.arange(0, rows, max(1, rows // 40)))
    ref, rl, err, spread = A.sparse_attention(case, q, idx, pool, hkv, e2m1, scale)
    assert bits == err == 0
    bad = ~(np.abs(out - ref) <= _bounds(ref, spread))
    assert not bad.any(), (int(bad.sum()), bad.size)
