"""The attention side in 64 bits: per-head norm and rotation, the 4-bit KV cache, and attention over
listed entries.  Plain numpy, shares no code with the CUDA library.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  bfloat16 and float16 inputs arrive as
float32 arrays that hold exactly representable values.
"""
from __future__ import annotations

import numpy as np

from . import ERR_LENGTH, ERR_PAGE

BLOCK = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the 127 finite non-negative float8_e4m3fn values, by code
E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def norm_rope(x, weight, positions, cos_sin, rotary, interleaved, eps, norm=True):
    """x float [T, H, D] -> float64 [T, H, D]; rows at positions outside the table are zero."""
    y = x.astype(np.float64)
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * weight.astype(np.float64)
    out = y.copy()
    half = rotary // 2
    for t, pos in enumerate(positions):
        if not 0 <= pos < cos_sin.shape[0]:
            out[t] = 0.0
            continue
        for i in range(half):
            c, s = float(cos_sin[pos, i]), float(cos_sin[pos, half + i])
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
    return out


def _nearest(grid, a):
    """Codes of the grid value nearest to a >= 0, ties to the even code, at most the last."""
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    mid = (grid[lo] + grid[hi]) / 2
    return np.where((a > mid) | ((a == mid) & (hi % 2 == 0)), hi, lo)


def quantize(x, e2m1, factor):
    """x float32 [..., D] -> (codes uint8 of 4 bits [..., D], scale bytes uint8 [..., D / 16])."""
    f32 = np.float32
    y = (x.astype(f32) / f32(factor)).reshape(*x.shape[:-1], -1, BLOCK)
    top = f32(6.0 if e2m1 else 7.0)
    scale = _nearest(E4M3, np.minimum(np.abs(y).max(-1) / top, f32(448)).astype(np.float64)).astype(np.uint8)
    s = E4M3[scale].astype(f32)[..., None]
    q = np.divide(y, s, out=np.zeros_like(y), where=s > 0).astype(f32)
    if e2m1:
        code = _nearest(E2M1, np.abs(q).astype(np.float64)) + 8 * (np.signbit(q) & (s > 0))
    else:
        code = np.clip(np.rint(q), -7, 7).astype(np.int64) & 15
    return code.astype(np.uint8).reshape(x.shape), scale


def unit_bytes(dim):
    return dim + dim // 8


def entry_bytes(heads, dim):
    return -(-heads * unit_bytes(dim) // 16) * 16


def encode(k, v, e2m1, k_scale=1.0, v_scale=1.0, into=None):
    """Entries uint8 [T, entry_bytes] of k, v [T, H, D]; padding bytes come from ``into`` (zeros)."""
    t, h, d = k.shape
    out = np.zeros((t, entry_bytes(h, d)), np.uint8) if into is None else into.copy()
    ck, sk = quantize(k, e2m1, k_scale)
    cv, sv = quantize(v, e2m1, v_scale)
    for i in range(h):
        at = i * unit_bytes(d)
        for part in (ck[:, i, 0::2] | (ck[:, i, 1::2] << 4), cv[:, i, 0::2] | (cv[:, i, 1::2] << 4), sk[:, i], sv[:, i]):
            out[:, at:at + part.shape[1]] = part
            at += part.shape[1]
    return out


def decode(entries, heads, dim, e2m1, k_scale=1.0, v_scale=1.0):
    """float64 (k, v) [T, H, D] of entries uint8 [T, entry_bytes]."""
    res = []
    for at, sat, f in ((0, dim, k_scale), (dim // 2, dim + dim // BLOCK, v_scale)):
        x = np.zeros((entries.shape[0], heads, dim))
        for i in range(heads):
            u = entries[:, i * unit_bytes(dim):]
            b = u[:, at:at + dim // 2]
            code = np.stack([b & 15, b >> 4], -1).reshape(-1, dim).astype(np.int64)
            val = np.where(code >= 8, -E2M1[code & 7], E2M1[code & 7]) if e2m1 else np.where(code >= 8, code - 16, code)
            byte = u[:, sat:sat + dim // BLOCK]
            s = np.where(byte >= 128, -1.0, 1.0) * np.append(E4M3, np.nan)[byte & 127]
            x[:, i] = val * np.repeat(s, BLOCK, -1) * np.float64(np.float32(f))
        res.append(x)
    return res


def entry_of(case, b, pos, limit):
    """((page, slot), 0) of a compressed position, or (None, error bit)."""
    if not (0 <= b < case.batch) or pos < 0 or pos >= limit:
        return None, ERR_LENGTH
    page = int(case.block_table[b, pos // case.block_size])
    if not 0 <= page < case.num_blocks:
        return None, ERR_PAGE
    return (page, pos % case.block_size), 0


def cache_write(case, pool, k, v, token_batch, token_pos, e2m1, k_scale=1.0, v_scale=1.0):
    """Write into ``pool`` (uint8 [num_blocks, block_size, entry_bytes]) in place; returns the error bits."""
    err = 0
    for t in range(len(token_batch)):
        where, e = entry_of(case, int(token_batch[t]), int(token_pos[t]), case.max_blocks_per_seq * case.block_size)
        err |= e
        if where:
            pool[where] = encode(k[t:t + 1], v[t:t + 1], e2m1, k_scale, v_scale, into=pool[where][None])[0]
    return err


def cache_read(case, pool, heads, dim, token_batch, token_pos, e2m1, k_scale=1.0, v_scale=1.0):
    """float64 (k, v, error bits); tokens with an invalid place are zero."""
    k = np.zeros((len(token_batch), heads, dim))
    v = np.zeros_like(k)
    err = 0
    for t in range(len(token_batch)):
        where, e = entry_of(case, int(token_batch[t]), int(token_pos[t]), case.max_blocks_per_seq * case.block_size)
        err |= e
        if where:
            k[t:t + 1], v[t:t + 1] = decode(pool[where][None], heads, dim, e2m1, k_scale, v_scale)
    return k, v, err


def row_batch(case, r):
    if case.layout_q == "BSND":
        return r // case.s1
    b = int(np.searchsorted(case.seq_lens_q, r, side="right"))
    return b if b < case.batch else -1


def sparse_attention(case, query, idx, pool, heads_kv, e2m1, scale, k_scale=1.0, v_scale=1.0, use_seq_lens_k=True):
    """(out, lse, error bits, spread): query float [rows, Hq, D]; out float64 [rows, Hq, D], lse [rows, Hq];
    ``spread`` holds what the tolerances need: wv = sum_i w_i |V_i| [rows, Hq, D], vmax = max |V|, qk = the
    largest sum_d |q_d K_d| * scale, kq = the largest max |q| * sum_d |K_d| * scale, n = entries used."""
    rows, hq, d = query.shape
    g = hq // heads_kv
    out = np.zeros((rows, hq, d))
    lse = np.full((rows, hq), -np.inf)
    spread = dict(wv=np.zeros((rows, hq, d)), vmax=np.zeros((rows, hq)), qk=np.zeros((rows, hq)), kq=np.zeros((rows, hq)),
                  n=np.zeros(rows, int))
    err = 0
    for r in range(rows):
        b = row_batch(case, r)
        limit = -1
        if 0 <= b < case.batch:
            limit = case.max_blocks_per_seq * case.block_size
            if use_seq_lens_k:
                limit = min(limit, -(-int(case.seq_lens_k[b]) // case.cmp_ratio))
        found = []
        for j in idx[r]:
            if j == -1:
                continue
            where, e = entry_of(case, b, int(j), limit)
            err |= e
            if where:
                found.append(pool[where])
        if not found:
            continue
        k, v = decode(np.stack(found), heads_kv, d, e2m1, k_scale, v_scale)
        spread["n"][r] = len(found)
        for h in range(hq):
            kk, vv, q = k[:, h // g], v[:, h // g], query[r, h].astype(np.float64)
            z = kk @ q * scale
            top = z.max()
            w = np.exp(z - top)
            lse[r, h] = top + np.log(w.sum())
            w = w / w.sum()
            out[r, h] = w @ vv
            spread["wv"][r, h] = w @ np.abs(vv)
            spread["vmax"][r, h] = np.abs(vv).max()
            spread["qk"][r, h] = (np.abs(kk) @ np.abs(q)).max() * scale
            spread["kq"][r, h] = np.abs(kk).sum(-1).max() * np.abs(q).max() * scale
    return out, lse, err, spread
