"""Failure detection of the sparse attention where the pages of the cache lie no whole number of entries apart
(16-byte copies instead of row gathers): with the testing build's stall switch nothing is copied, so every
bounded wait runs out; the kernel must report QLI_ERR_DEVICE_TIMEOUT, write NaN and leave the context usable."""
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
rows, dim = %d, %d
p = Q.make_problem(batch=rows, max_q_tokens=1, num_blocks=4, block_size=64, max_blocks_per_seq=4, sparse_count=64,
                   sparse_mode=0, cmp_ratio=1, max_seqlen_q=1, max_seqlen_k=256)
a = Q.make_attention(num_heads_q=8, num_heads_kv=8, head_dim=dim)
a.kv_stride = 64 * Q.kv_entry_bytes(a) + 16
dev = dict(device="cuda")
pool = torch.zeros(4, a.kv_stride, dtype=torch.uint8, **dev)
q = torch.ones(rows, 8, dim, dtype=torch.bfloat16, **dev)
out = torch.ones_like(q)
table = torch.arange(4, dtype=torch.int32, **dev).repeat(rows, 1)
idx = torch.arange(64, dtype=torch.int32, **dev).repeat(rows, 1)
lens = torch.full((rows,), 256, dtype=torch.int32, **dev)
ws = torch.zeros(64, dtype=torch.int32, **dev)
Q.check(Q.sparse_attention(p, a, q, None, lens, table, idx, pool, out, None, ws), "sparse_attention")
st, bits = Q.get_device_error(ws)
print("STATUS", st, bits, int(torch.isnan(out.float()).all().item()), int((out == 0).all().item()))
print("AFTER", torch.ones(1024, **dev).sum().item())
"""


@pytest.mark.parametrize("rows,dim", [(2, 64), (460, 128)])
@pytest.mark.parametrize("stall", [1, 0])
def test_waits_run_out(built, rows, dim, stall):  # noqa: F811
    out = subprocess.run([sys.executable, "-c", CHILD % (ROOT, stall, rows, dim)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stderr[-2000:]
    status = [x for x in out.stdout.splitlines() if x.startswith("STATUS")][0].split()[1:]
    assert status == (["6", "4", "1", "0"] if stall else ["0", "0", "0", "1"])
    assert "AFTER 1024.0" in out.stdout
