"""The example's layers without an indexer on the GPU, against the 64-bit oracle (needs a GB300)."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("kv", ["KV_E2M1", "KV_INT4"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_layer_step(kv, window, sinks):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_token_block_gb300 import build as B
    B.build()
    import sparse_attention_token_block_gb300 as Q
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    from sparse_layer_step import LayerStep
    step = LayerStep(np.array([700, 130, 64]), getattr(Q, kv), window=window, sinks=sinks)
    first = step().clone()
    assert step.device_error() == (0, 0)
    off, off_lse = step.check()
    # bfloat16's half step on the largest value, and one more for the fp16 probabilities and fp32 sums
    assert off < 2.0 ** -7 and off_lse < 1e-4
    assert torch.equal(step(), first)
