"""The cache write's divisions on the GPU: every scale against operands around every code's border, bit
for bit against the oracle's fp32 divisions (needs a GB300)."""
import numpy as np
import pytest

from oracle import attention as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e2m1", [True, False])
@pytest.mark.parametrize("factor", [1.0, 0.7, 3.0e-4])
def test_every_scale_at_every_border(e2m1, factor):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_token_block_gb300 import build as B
    B.build()
    import sparse_attention_token_block_gb300 as Q
    top = 6.0 if e2m1 else 7.0
    mids = (A.E2M1[1:] + A.E2M1[:-1]) / 2 if e2m1 else np.arange(7) + 0.5
    blocks = []
    for s in A.E4M3[1:]:
        for m in mids:
            # the block's largest element sets the scale; the others are halves around the border m * s
            near = np.float16(min(m * s * factor, 6e4))
            bits = near.view(np.uint16).astype(int) + np.arange(-7, 8)
            v = np.clip(bits, 0, 0x7BFF).astype(np.uint16).view(np.float16)
            v = np.minimum(v, np.float16(min(top * s * factor, 6e4))) * np.where(np.arange(15) % 2, 1, -1)
            blocks.append(np.append(v, np.float16(min(top * s * factor, 6e4))))
    x = np.array(blocks, np.float16)
    x = np.concatenate([x, np.zeros((-len(x) % 4, 16), np.float16)]).reshape(-1, 1, 64).astype(np.float32)
    n = len(x)
    p = Q.make_problem(batch=1, max_q_tokens=1, num_blocks=-(-n // 64), block_size=64, max_blocks_per_seq=-(-n // 64),
                       sparse_count=1, sparse_mode=0, cmp_ratio=1, max_seqlen_q=1, max_seqlen_k=n)
    a = Q.make_attention(num_heads_q=1, num_heads_kv=1, head_dim=64, dtype=Q.ACT_F16, kv_dtype=Q.KV_E2M1 if e2m1 else Q.KV_INT4,
                         k_scale=factor, v_scale=factor)
    pool = torch.zeros(p.num_blocks, 64, Q.kv_entry_bytes(a), dtype=torch.uint8, device="cuda")
    d = torch.from_numpy(x).half().cuda()
    i32 = lambda v: torch.from_numpy(np.asarray(v, np.int32)).cuda()  # noqa: E731
    Q.check(Q.kv_write(p, a, d, -d, i32(np.zeros(n)), i32(np.arange(n)), i32(np.arange(p.num_blocks)[None]), pool), "kv_write")
    ref = A.encode(x, -x, e2m1, factor, factor)
    assert np.array_equal(pool.cpu().numpy().reshape(-1, ref.shape[1])[:n], ref)
