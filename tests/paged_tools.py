"""Calls, inputs and tolerances shared by the tests of the dense paged attention and of the append."""
import math

import numpy as np

import workloads as W
from attention_tools import attention_bounds, half_step, round_to, smallest_step
from oracle import attention as A

U = 2.0 ** -24                                             # half a step of fp32


def dev(a, f16=None):
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if f16 is None else t.to(torch.float16 if f16 else torch.bfloat16)


def queries(rows, hq, dim, f16, seed, std=1.0):
    return round_to(np.random.default_rng(seed).normal(size=(rows, hq, dim)) * std, f16)


def settings(Q, case, hq, hkv, dim, e2m1, f16, complete=False, max_seqlen_k=None, **kw):
    args = dict(W.problem_kwargs(case), mask_complete_blocks=int(complete))
    if max_seqlen_k is not None:
        args["max_seqlen_k"] = max_seqlen_k
    return (Q.make_problem(**args),
            Q.make_attention(num_heads_q=hq, num_heads_kv=hkv, head_dim=dim, dtype=Q.ACT_F16 if f16 else Q.ACT_BF16,
                             kv_dtype=Q.KV_E2M1 if e2m1 else Q.KV_INT4, **kw))


def attend(Q, case, query, pool, hkv, e2m1, f16, window=0, sinks=0, scale=0.0, factors=(1.0, 1.0), kv_stride=0, q_pad=0,
           complete=False, max_seqlen_k=None):
    """paged_attention on fresh buffers: (out, lse, error bits); called twice, and the results are the same."""
    import torch
    rows, hq, dim = query.shape
    p, a = settings(Q, case, hq, hkv, dim, e2m1, f16, complete, max_seqlen_k, softmax_scale=scale, k_scale=factors[0],
                    v_scale=factors[1], kv_stride=kv_stride)
    qd = dev(np.concatenate([query, np.ones((rows, q_pad, dim), np.float32)], 1), f16)[:, :hq]
    out = torch.full((rows, hq, dim), 5.0, dtype=qd.dtype, device="cuda")
    lse = torch.full((rows, hq), 5.0, dtype=torch.float32, device="cuda")
    ws = torch.zeros(64, dtype=torch.int32, device="cuda")
    args = (dev(case.seq_lens_q), dev(case.seq_lens_k), dev(case.block_table), dev(pool))
    Q.check(Q.paged_attention(p, a, qd, *args, out, lse, ws, window=window, sinks=sinks), "paged_attention")
    bits = Q.get_device_error(ws)[1]
    again = torch.full_like(out, 7.0)
    Q.check(Q.paged_attention(p, a, qd, *args, again, window=window, sinks=sinks), "paged_attention")
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), bits


def check(case, got, query, pool, hkv, e2m1, f16, window=0, sinks=0, scale=0.0, factors=(1.0, 1.0), complete=False,
          max_seqlen_k=None):
    out, lse, bits = got
    d = query.shape[2]
    ref, rl, err, spread = A.paged_attention(case, query, pool, hkv, e2m1, scale or 1 / math.sqrt(d), *factors, window=window,
                                             sinks=sinks, complete=complete, max_seqlen_k=max_seqlen_k)
    assert bits == err
    tol, ltol = attention_bounds(ref, rl, spread, d, f16)
    bad = ~(np.abs(out - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], out[bad][:3], ref[bad][:3], tol[bad][:3])
    empty = np.isinf(rl)
    assert np.array_equal(np.isinf(lse), empty) and (lse[empty] < 0).all()
    assert np.all(np.abs(lse[~empty] - rl[~empty]) <= ltol[~empty])
    assert not out[empty].any()


def turn_bound(x, weight, positions, cos_sin, rotary, interleaved, eps, norm):
    """Bound of an fp32 norm and rotation's error against 64 bits, [T, H, D]: the sum of squares (rounded at most 16
    times on the way of any term), mean, eps and root stay within 16 U of the factor (rsqrt: 2 ulp), the two
    factors round twice, and the rotation's two products and sum at most three times each part: 24 U of
    |a c| + |b s|, every magnitude of the normalised vector."""
    y = np.abs(x.astype(np.float64))
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.abs(weight.astype(np.float64))
    table = np.abs(cos_sin)
    mags = A.norm_rope(y, None, positions, np.concatenate([table[:, :rotary // 2], -table[:, rotary // 2:]], 1), rotary,
                       interleaved, 0.0, norm=False)
    # a c - b (-s) and b c + a (-s): the second has to be a sum too
    other = A.norm_rope(y, None, positions, table, rotary, interleaved, 0.0, norm=False)
    return 24 * U * np.maximum(mags, other)


def check_cached(raw, y, dy, e2m1, factor, values):
    """Codes and scales of one KV head's K (values False) or V in entries' bytes `raw` [T, unit] against the real
    numbers y [T, D] known within dy: each lies between those of the ends of what y may be."""
    d = y.shape[1]
    at, sat = (d // 2, d + d // 16) if values else (0, d)
    b = raw[:, at:at + d // 2]
    code = np.stack([b & 15, b >> 4], -1).reshape(-1, d).astype(np.int64)
    scale = raw[:, sat:sat + d // 16].astype(np.int64)
    f = np.float64(np.float32(factor))
    top = 6.0 if e2m1 else 7.0
    mag, dq = np.abs(y) / f, (dy + 2 * U * np.abs(y)) / f
    blocks = lambda x: x.reshape(len(x), -1, 16)  # noqa: E731
    small = lambda a: A._nearest(A.E4M3, np.minimum(np.maximum(a, 0) / top, 448.0))  # noqa: E731
    low, high = (blocks(np.maximum(mag - dq, 0)).max(-1) * (1 - 2 * U), blocks(mag + dq).max(-1) * (1 + 2 * U))
    assert ((small(low) <= scale) & (scale <= small(high))).all()
    s = np.repeat(A.E4M3[scale], 16, -1)
    val = np.where(code >= 8, -A.E2M1[code & 7], A.E2M1[code & 7]) if e2m1 else np.where(code >= 8, code - 16, code)
    grid = np.concatenate([-A.E2M1[:0:-1], A.E2M1]) if e2m1 else np.arange(-7.0, 8.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        q0, q1 = ((y / f - dq) / s, (y / f + dq) / s)
    room = lambda x, way: np.clip(x + way * 4 * U * np.abs(x), -top, top)  # noqa: E731
    def nearest(x, up):                                    # the larger or smaller neighbour of a tie
        i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
        lo, hi = grid[i - 1], grid[i]
        return np.where((x - lo > hi - x) | ((x - lo == hi - x) & up), hi, lo)
    live = s > 0
    assert (val[~live] == 0).all()
    assert (nearest(room(q0, -1), False)[live] <= val[live]).all() and (val[live] <= nearest(room(q1, 1), True)[live]).all()


__all__ = ["dev", "queries", "settings", "attend", "check", "turn_bound", "check_cached", "half_step", "smallest_step", "round_to"]
