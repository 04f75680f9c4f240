"""One decode step of an attention layer, from the packed projections to the attention's output.

    python examples/sparse_layer_step.py [--batch 32] [--kv-dtype e2m1|int4] [--window N [--sinks N]] [--check]

Per step: norm and rotate the new token's queries and keys, its key and value going straight into the
4-bit cache (one pass), quantise the indexer's query and key, select 2048 cached positions per sequence,
attend to them.  With ``--window`` the layer is one without an indexer: its tokens attend to the last N
cached positions and the first few (``--sinks``), with 0 to all of them.  Every call only enqueues, so the
step is captured once into a CUDA graph and replayed.  ``--check`` compares the last step with the 64-bit
oracle (on the host).
"""
import argparse
import math
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import sparse_attention_token_block_gb300 as Q  # noqa: E402

HQ, HKV, DIM, INDEX_HEADS, BLOCK, TOP = 64, 8, 128, 64, 64, 2048


class LayerStep:
    """Buffers of one layer for `lens` cached tokens per sequence (the new token included); `window` None: the
    indexer selects `top` positions."""

    def __init__(self, lens, kv_dtype=Q.KV_E2M1, seed=0, top=TOP, window=None, sinks=0):
        self.window, self.sinks = window, sinks
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
        i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
        self.lens, b = np.asarray(lens), len(lens)
        need = -(-self.lens // BLOCK)
        order = np.random.default_rng(seed).permutation(int(need.sum()))
        table = np.full((b, int(need.max())), -1, np.int32)
        for i, n in enumerate(need):
            table[i, :n] = order[need[:i].sum():need[:i].sum() + n]
        self.p = Q.make_problem(batch=b, max_q_tokens=1, num_blocks=len(order), block_size=BLOCK,
                                max_blocks_per_seq=table.shape[1], sparse_count=top, sparse_mode=3, cmp_ratio=1,
                                max_seqlen_q=1, max_seqlen_k=int(self.lens.max()))
        self.a = Q.make_attention(num_heads_q=HQ, num_heads_kv=HKV, head_dim=DIM, kv_dtype=kv_dtype)
        self.r = Q.make_norm_rope(num_heads_q=HQ, num_heads_k=HKV, head_dim=DIM, rotary_dim=DIM,
                                  max_positions=int(self.lens.max()))
        self.indexer = Q.Indexer(self.p)
        self.table, self.seq_lens_k = i32(table), i32(self.lens)
        self.token_batch, self.token_pos = i32(np.arange(b)), i32(self.lens - 1)
        angle = np.arange(self.lens.max())[:, None] * 10000.0 ** (-np.arange(0, DIM, 2) / DIM)[None, :]
        self.cos_sin = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
        # this step's projections: packed queries, keys and values, and the indexer's query and key
        self.qkv = rand(b, HQ + 2 * HKV, DIM).bfloat16()
        self.index_q, self.index_k = rand(b, INDEX_HEADS, DIM).bfloat16(), rand(b, DIM).bfloat16()
        self.index_w = rand(b, INDEX_HEADS).abs().mul_(0.01).half()
        self.q_weight, self.k_weight = (1 + 0.1 * rand(DIM)).bfloat16(), (1 + 0.1 * rand(DIM)).bfloat16()
        # the caches, filled as a prefill leaves them
        n = len(order) * BLOCK
        self.index_pool = torch.empty(len(order), BLOCK, 1, DIM, dtype=torch.int8, device="cuda")
        self.index_scale = torch.empty(len(order), BLOCK, 1, dtype=torch.float16, device="cuda")
        self.kv_pool = torch.zeros(len(order), BLOCK, Q.kv_entry_bytes(self.a), dtype=torch.uint8, device="cuda")
        Q.check(Q.quantize(Q.INT8, Q.F16, rand(n, DIM).bfloat16(), self.index_pool, self.index_scale), "quantize")
        for i in range(b):
            pos = torch.arange(self.lens[i], dtype=torch.int32, device="cuda")
            kv = rand(len(pos), 2 * HKV, DIM).bfloat16()
            Q.check(Q.kv_write(self.p, self.a, kv[:, :HKV], kv[:, HKV:], torch.full_like(pos, i), pos, self.table, self.kv_pool),
                    "kv_write")
        # what the step writes
        self.q = torch.empty(b, HQ, DIM, dtype=torch.bfloat16, device="cuda")
        self.index_q8 = torch.empty(b, INDEX_HEADS, DIM, dtype=torch.int8, device="cuda")
        self.index_q_scale = torch.empty(b, INDEX_HEADS, dtype=torch.float16, device="cuda")
        self.out = torch.empty_like(self.q)
        self.lse = torch.empty(b, HQ, dtype=torch.float32, device="cuda")

    def __call__(self):
        p, a, ws = self.p, self.a, self.indexer.workspace
        Q.check(Q.kv_append(p, a, self.r, self.qkv[:, :HQ], self.qkv[:, HQ:HQ + HKV], self.qkv[:, HQ + HKV:], self.q_weight,
                            self.k_weight, self.token_pos, self.cos_sin, self.token_batch, self.token_pos, self.table, self.q,
                            self.kv_pool, ws), "kv_append")
        if self.window is not None:
            Q.check(Q.paged_attention(p, a, self.q, None, self.seq_lens_k, self.table, self.kv_pool, self.out, self.lse, ws,
                                      window=self.window, sinks=self.sinks), "paged_attention")
            return self.out
        Q.check(Q.quantize(Q.INT8, Q.F16, self.index_q, self.index_q8, self.index_q_scale), "quantize")
        Q.check(Q.quantize_keys(p, self.index_k, self.token_batch, self.token_pos, self.table, self.index_pool,
                                self.index_scale, ws), "quantize_keys")
        self.indices = self.indexer.run(self.index_q8, self.index_pool, self.index_w, self.index_q_scale, self.index_scale,
                                        None, self.seq_lens_k, self.table)
        Q.check(Q.sparse_attention(p, a, self.q, None, self.seq_lens_k, self.table, self.indices, self.kv_pool, self.out,
                                   self.lse, ws), "sparse_attention")
        return self.out

    def device_error(self):
        return self.indexer.device_error()

    def check(self):
        """The attention of the step as it ran (its rotated queries, indices and cache) in 64 bits."""
        from types import SimpleNamespace

        from oracle import attention as A
        case = SimpleNamespace(layout_q="BSND", s1=1, batch=len(self.lens), cmp_ratio=1, block_size=BLOCK,
                               num_blocks=self.p.num_blocks, max_blocks_per_seq=self.p.max_blocks_per_seq,
                               block_table=self.table.cpu().numpy(), seq_lens_q=None, seq_lens_k=self.lens, sparse_mode=3,
                               max_seqlen_k=self.p.max_seqlen_k)
        q, pool, e2m1 = self.q.float().cpu().numpy(), self.kv_pool.cpu().numpy(), self.a.kv_dtype == Q.KV_E2M1
        if self.window is None:
            ref, lse, err, _ = A.sparse_attention(case, q, self.indices.cpu().numpy(), pool, HKV, e2m1, 1 / math.sqrt(DIM))
        else:
            ref, lse, err, _ = A.paged_attention(case, q, pool, HKV, e2m1, 1 / math.sqrt(DIM), window=self.window,
                                                 sinks=self.sinks)
        assert err == 0
        off = np.abs(self.out.double().cpu().numpy() - ref).max() / np.abs(ref).max()
        off_lse = np.abs(self.lse.double().cpu().numpy() - lse).max()
        return off, off_lse


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--kv-dtype", default="e2m1", choices=["e2m1", "int4"])
    ap.add_argument("--window", type=int, default=None, help="no indexer: attend to the last N positions (0: all)")
    ap.add_argument("--sinks", type=int, default=0, help="and to the first N")
    ap.add_argument("--check", action="store_true")
    args = ap.parse_args()
    lens = np.random.default_rng(3).integers(8192, 32768, size=args.batch, endpoint=True)
    step = LayerStep(lens, Q.KV_E2M1 if args.kv_dtype == "e2m1" else Q.KV_INT4, window=args.window, sinks=args.sinks)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        step()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for _ in range(5):
            graph.replay()
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(50):
            graph.replay()
        stop.record()
    torch.cuda.synchronize()
    st, bits = step.device_error()
    Q.check(st, "device error (bits %d)" % bits)
    print("%d sequences of %d-%d tokens, %s cache: %.1f us per layer step" % (
        args.batch, lens.min(), lens.max(), args.kv_dtype, start.elapsed_time(stop) * 1e3 / 50))
    if args.check:
        off, off_lse = step.check()
        print("against 64 bits: out %.1e of its largest value, lse %.1e" % (off, off_lse))
        assert off < 2.0 ** -7 and off_lse < 1e-3


if __name__ == "__main__":
    main()
