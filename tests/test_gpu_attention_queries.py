"""float16 queries enter the attention's products as they are: a head's small elements count beside a
large one, however far apart (both kernels, against the 64-bit oracle; needs a GB300)."""
import numpy as np
import pytest

from attention_tools import attention_bounds, cache_case, round_to
from oracle import attention as A
from test_gpu_attention_ranges import _lists, _sample, _sms
from test_gpu_sparse_attention import Q, _run  # noqa: F401 (Q is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,blocks", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("e2m1", [True, False])
def test_small_elements_beside_a_large_one(Q, dim, blocks, e2m1):
    """Element 0 of a query is 2^15 and meets keys that are zero there; the logits come from the others, of about
    2^-10 and down to float16's subnormals."""
    hq, hkv, keys = 64, 8, 600
    rows = 16 * -(-_sms() // hkv) if blocks else 5
    case = cache_case(layout_q="TND", q_lens=[rows], seq_lens_k=[keys], block_size=16, sparse_count=512, seed=3)
    rng = np.random.default_rng(1)
    n = case.num_blocks * 16
    k, v = (rng.normal(size=(n, hkv, dim)).astype(np.float32) for _ in range(2))
    k *= 200
    k[..., 0] = 0
    pool = A.encode(k, v, e2m1).reshape(case.num_blocks, 16, -1)
    q = rng.normal(size=(rows, hq, dim)) * 2.0 ** -10 * np.exp(rng.uniform(-6, 0, (rows, hq, dim)))
    q[..., 0] = np.where(rng.random((rows, hq)) < 0.5, 32768, -32768)
    q = round_to(q, True)
    idx = _lists(case, 2)
    got = _run(Q, case, q, idx, pool, hkv, e2m1, True, 1.0)
    case, (out, lse, bits), q, idx = _sample(case, got, q, idx, np.array([0, 1, rows // 2, rows - 2, rows - 1]))
    ref, rl, err, spread = A.sparse_attention(case, q, idx, pool, hkv, e2m1, 1.0)
    spread["kq"][:] = 0                                      # nothing is lost of a query
    tol, ltol = attention_bounds(ref, rl, spread, dim, True)
    assert bits == err == 0
    assert np.all(np.abs(out - ref) <= tol) and np.all(np.abs(lse - rl) <= ltol)
