"""Failure detection of the dense paged attention: with the testing build's stall switch nothing is copied or handed
on, so every bounded wait runs out; both kernels must report QLI_ERR_DEVICE_TIMEOUT, write NaN and leave the context
usable (needs a GB300)."""
import os
import subprocess
import sys

import pytest

from test_gpu_attention_faults import built  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
sys.path.insert(0, %r)
import torch
import sparse_attention_token_block_gb300 as Q
Q.use_testing_library()
Q.lib.qli_testing_set_stall(%d)
Q.lib.qli_testing_set_paged(%d)
batch, s1, heads, dim = %d, %d, %d, 128
p = Q.make_problem(batch=batch, max_q_tokens=s1, num_blocks=16, block_size=64, max_blocks_per_seq=16, sparse_count=1,
                   sparse_mode=0, cmp_ratio=1, max_seqlen_q=s1, max_seqlen_k=1024)
a = Q.make_attention(num_heads_q=heads, num_heads_kv=heads, head_dim=dim)
dev = dict(device="cuda")
pool = torch.zeros(16, 64, Q.kv_entry_bytes(a), dtype=torch.uint8, **dev)
q = torch.ones(batch * s1, heads, dim, dtype=torch.bfloat16, **dev)
out, lse = torch.ones_like(q), torch.ones(batch * s1, heads, **dev)
table = torch.arange(16, dtype=torch.int32, **dev).repeat(batch, 1)
lens = torch.full((batch,), 1024, dtype=torch.int32, **dev)
ws = torch.zeros(64, dtype=torch.int32, **dev)
Q.check(Q.paged_attention(p, a, q, None, lens, table, pool, out, lse, ws), "paged_attention")
st, bits = Q.get_device_error(ws)
nan = torch.isnan(out.float()).all() and torch.isnan(lse).all()
print("STATUS", st, bits, int(nan.item()), int((out == 0).all().item()))
print("AFTER", torch.ones(1024, **dev).sum().item())
"""


# one CTA a block, clusters that share one, and more blocks than the GPU holds at a time
@pytest.mark.parametrize("kernel,batch,s1,heads", [(1, 2, 1, 8), (1, 1, 1, 1), (2, 20, 130, 8), (2, 1, 130, 2), (2, 60, 130, 4)])
@pytest.mark.parametrize("stall", [1, 0])
def test_waits_run_out(built, kernel, batch, s1, heads, stall):  # noqa: F811
    out = subprocess.run([sys.executable, "-c", CHILD % (ROOT, stall, kernel, batch, s1, heads)], capture_output=True, text=True,
                         timeout=120)
    assert out.returncode == 0, out.stderr[-2000:]
    status = [x for x in out.stdout.splitlines() if x.startswith("STATUS")][0].split()[1:]
    assert status == (["6", "4", "1", "0"] if stall else ["0", "0", "0", "1"])
    assert "AFTER 1024.0" in out.stdout
